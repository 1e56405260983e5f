"""8-bit cache pages: the append that writes them, reading them back, and attention over them,
against the fp64 definitions.

Tolerances.  A kept number is the nearest of e4m3's to y / 2^e: off by at most 2^-4 of |y| (half a
step of three mantissa bits) or 2^-10 2^e (half a step of the subnormals), and a key's y in fp32 by
E = 2^-24 (D + 24) of the largest magnitude that its norm and rotation handle: r is off by at most
(D + 4) 2^-24 relative (D squares summed, mean, square root), each product and sum of the rotation by
2^-24 of its terms, whose magnitudes are at most sqrt(2) of the pair's.  Values are scaled by powers
of two and rounded once, so their bytes are the definition's.  Attention: what the rows stand for is
exact in bf16 and fp32, so its tolerances are those of attention over such a cache
(test_gpu_paged_attention.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import q8_ref  # noqa: E402
import serving_ref as ref  # noqa: E402
import test_gpu_paged_attention as pa  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
host = pa.host


def e4m3(b):
    return torch.from_numpy(np.ascontiguousarray(b)).cuda().view(torch.float8_e4m3fn)


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def read(kb, vb, ks, vs, slots, dt, page):
    T, Hkv, D = len(slots), kb.shape[1], kb.shape[3]
    k = torch.full((T, Hkv, D), 5.0, dtype=DT[dt], device="cuda")
    v = torch.full_like(k, 5.0)
    kda.kda_paged_cache_read_q8(kb, vb, ks, vs, slots, k, v, T, Hkv, D, kb.shape[0], page)
    return k, v


# ------------------------------------------------------------------------------- reading back

@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_every_number_under_every_scale(dt, D):
    """All 256 bytes of numbers under all 256 scales.  (bf16 has no steps below 2^-133, and numbers
    under the scale bytes 0 to 2, which no append writes, are multiples of 2^-136 to 2^-134: there
    the nearest bf16 is what comes back.)"""
    ensure_built()
    H = 256 // D
    nums = np.broadcast_to(np.arange(256, dtype=np.uint8).reshape(1, H, 1, D), (16, H, 16, D))
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8).reshape(16, 1, 16), (16, H, 16))
    kb, ks = e4m3(nums), torch.from_numpy(scales.copy()).cuda()
    vb, vs = e4m3(nums[:, :, :, ::-1]), torch.from_numpy(scales[::-1].copy()).cuda()
    slots = torch.arange(256, device="cuda")
    k, v = read(kb, vb, ks, vs, slots, dt, 16)
    with np.errstate(over="ignore", invalid="ignore"):
        for got, b, s in ((k, raw(kb), scales), (v, raw(vb), scales[::-1])):
            want = q8_ref.value(b, s).astype(np.float32).transpose(0, 2, 1, 3).reshape(256, H, D)
            got = host(got)
            if dt == "bf16":
                assert (b.shape, s.min()) == (nums.shape, 0)
                near = host(torch.from_numpy(want).to(torch.bfloat16).float())
                assert (near == want)[np.broadcast_to(
                    (s > 2).transpose(0, 2, 1).reshape(256, H, 1), want.shape) &
                    np.isfinite(want)].all()
                want = near
            fine = np.isfinite(want) & (np.abs(want) <= 2.0 ** 127.9)
            assert (got[fine] == want[fine]).all()
            assert (np.isnan(got) == np.isnan(want)).all()
            assert not np.isfinite(got[np.isinf(want)]).any()


def test_read_slots_outside_and_order():
    ensure_built()
    rng = np.random.default_rng(0)
    nums, scales = q8_ref.quantise(rng.standard_normal((5, 3, 32, 64)))
    kb, ks = e4m3(nums), torch.from_numpy(scales).cuda()
    slots = torch.tensor([159, 3, -1, 160, 3, 2 ** 40, 64, -2 ** 60, 0], device="cuda")
    k, v = read(kb, kb, ks, ks, slots, "f32", 32)
    x = q8_ref.value(nums, scales).transpose(0, 2, 1, 3).reshape(160, 3, 64)
    for t, s in enumerate(slots.tolist()):
        want = x[s] if 0 <= s < 160 else np.zeros((3, 64))
        assert (host(k)[t] == want).all() and (host(v)[t] == want).all()
    # no tokens, no pages
    kda.kda_paged_cache_read_q8(kb, kb, ks, ks, slots[:0], k[:0], v[:0], 0, 3, 64, 5, 32)
    kda.kda_paged_cache_read_q8(None, None, None, None, slots, k, v, 9, 3, 64, 0, 32)
    assert (host(k) == 0).all() and (host(v) == 0).all()


# ----------------------------------------------------------------------------------- appending

def append(T, Hq, Hkv, D, R, page, dt, interleaved, seed=0, v=None, k=None, std=1.0):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    qkv = (rn(T, (Hq + 2 * Hkv + 1) * D) * std).to(DT[dt])
    q = qkv[:, :Hq * D].view(T, Hq, D)
    kk = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    vv = qkv[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    if v is not None:
        vv.copy_(v)
    if k is not None:
        kk.copy_(k)
    pages, maxp = -(-T // page) + 2, 500
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].clone()
    if T > 3:
        slots[1], slots[T - 1] = -1, pages * page
    wq, wk = 1 + 0.3 * rn(D), 1 + 0.3 * rn(D)
    pos = torch.randint(-3, maxp + 3, (T,), generator=g, device="cuda", dtype=torch.int32)
    ang = torch.arange(maxp, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (
        -torch.arange(0, max(R, 2), 2, device="cuda", dtype=torch.float64) / max(R, 2))
    cos, sin = ang.cos().float(), ang.sin().float()
    fill = torch.full((pages, Hkv, page, D), 0x5A, dtype=torch.uint8, device="cuda")
    kb, vb = (fill.clone().view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv, page), 0xA5, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    qo = torch.empty(T, Hq, D, dtype=DT[dt], device="cuda")
    kw = dict(eps=1e-5, interleaved=interleaved)
    head = (q, kk, vv, wq, wk, cos, sin, pos, slots)
    tail = (T, Hq, Hkv, D, R, maxp, pages, page)
    kda.kda_qk_norm_rope_append_q8(*head, qo, kb, vb, ks, vs, *tail, **kw)
    return dict(head=head, tail=tail, kw=kw, q=q, k=kk, v=vv, wk=wk, cos=cos, sin=sin, pos=pos,
                slots=slots, kb=kb, vb=vb, ks=ks, vs=vs, qo=qo, pages=pages, page=page, D=D, R=R,
                T=T, Hkv=Hkv, maxp=maxp, interleaved=interleaved, dt=dt)


def check_append(a):
    T, Hkv, D, page, pages = a["T"], a["Hkv"], a["D"], a["page"], a["pages"]
    slots = a["slots"].cpu().numpy()
    kept = (slots >= 0) & (slots < pages * page)

    def flat(x):
        x = raw(x)
        return np.moveaxis(x, 2, 1).reshape(pages * page, Hkv, *x.shape[3:])

    # values: the definition's bytes
    b, s = q8_ref.quantise(host(a["v"]))
    assert (flat(a["vs"])[slots[kept]] == s[kept]).all()
    assert (q8_ref.E4M3[flat(a["vb"])[slots[kept]]] == q8_ref.E4M3[b][kept]).all()
    # keys
    p = np.clip(a["pos"].cpu().numpy(), 0, a["maxp"] - 1)
    with np.errstate(invalid="ignore"):
        y = ref.norm_rope(host(a["k"]), host(a["wk"]), host(a["cos"])[p], host(a["sin"])[p],
                          a["R"], 1e-5, a["interleaved"])
    fine = np.isfinite(y).all(-1)
    y = np.where(fine[..., None], y, 0.0)
    err = 2.0 ** -24 * (D + 24) * 2 ** 0.5 * np.abs(y).max(-1, keepdims=True)
    sb, nb = flat(a["ks"]), flat(a["kb"])
    got_s = np.zeros(y.shape[:2], int)
    got_s[kept] = sb[slots[kept]]
    assert ((got_s == 255) == ~fine)[kept].all()
    e = got_s - 127
    lo = q8_ref.exponents(np.maximum(np.abs(y) - err, 0))
    hi = q8_ref.exponents(np.abs(y) + err)
    ok = kept[:, None] & fine
    assert ((lo <= e) & (e <= hi))[ok].all()
    got = np.zeros(y.shape)
    got[kept] = q8_ref.E4M3[nb[slots[kept]]]
    got = got * 2.0 ** e[..., None].astype(float)
    lim = err + np.maximum(2.0 ** -4 * (np.abs(y) + err), 2.0 ** (e[..., None] - 10.0))
    assert (np.abs(got - y) <= lim)[ok].all()
    # other places are as they were
    other = np.ones(pages * page, bool)
    other[slots[kept]] = False
    for x, f in ((a["kb"], 0x5A), (a["vb"], 0x5A), (a["ks"], 0xA5), (a["vs"], 0xA5)):
        assert (flat(x)[other] == f).all()
    # queries: those of the other appending call
    qo = torch.empty_like(a["qo"])
    kc, vc = (torch.empty(pages, Hkv, page, D, dtype=DT[a["dt"]], device="cuda") for _ in range(2))
    kda.kda_qk_norm_rope_append(*a["head"], qo, kc, vc, *a["tail"], **a["kw"])
    assert torch.equal(qo, a["qo"])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,R", [(32, 32), (32, 0), (64, 16), (64, 64), (128, 64), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,page", [(1, 4, 1, 16), (7, 3, 3, 128), (130, 6, 2, 64)])
def test_append(dt, D, R, interleaved, T, Hq, Hkv, page):
    check_append(append(T, Hq, Hkv, D, R, page, dt, interleaved, seed=T + D + R))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1215, 1216, 1301])
@pytest.mark.parametrize("Hkv,D", [(20, 32), (5, 64), (8, 128)])
def test_append_of_many_tokens(dt, T, Hkv, D):
    """Where a warp begins to take all heads of a kind."""
    check_append(append(T, Hkv, Hkv, D, D, 32, dt, False, seed=T))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_of_any_magnitude(dt):
    """Zeros, the smallest and largest magnitudes, borders of the scale and of the rounding, numbers
    that are halfway, infinities and NaNs, each in a row of its own."""
    D = 64
    rng = np.random.default_rng(3)
    rows = [np.zeros(D), np.full(D, 1e-38), np.full(D, 3.3e38), np.full(D, -3e38),
            rng.standard_normal(D) * 1e-30, rng.standard_normal(D) * 1e30]
    for k in range(-130, 120, 7):
        for top in (448.0, 449.0, 256.0, 447.0):  # (449 becomes 448 or 450 in bf16)
            x = rng.standard_normal(D)
            x = x / np.abs(x).max() * top * 2.0 ** k
            rows.append(x)
    half = (q8_ref.E4M3[:126] + q8_ref.E4M3[1:127]) / 2  # halves, both signs
    for k in (0, -20, 30):
        for part in (half[:62], half[62:124], -half[:62], -half[64:126]):
            rows.append(np.concatenate([part, [448.0, 0.0]]) * 2.0 ** k)
    for bad in (np.nan, np.inf, -np.inf):
        x = rng.standard_normal(D)
        x[rng.integers(D)] = bad
        rows.append(x)
    x = np.stack(rows)[:, None]
    v = torch.from_numpy(x).to("cuda", DT[dt])
    a = append(len(rows), 2, 1, D, 32, 16, dt, False, v=v, seed=9)
    check_append(a)
    k, vv = read(a["kb"], a["vb"], a["ks"], a["vs"], a["slots"], dt, 16)
    slots = a["slots"].cpu().numpy()
    kept = (slots >= 0) & (slots < a["pages"] * 16)
    b, s = q8_ref.quantise(host(a["v"]))
    want = q8_ref.value(b, s)
    assert (np.isnan(host(vv)) == np.isnan(want))[kept].all()
    fine = np.isfinite(want) & kept[:, None, None]
    assert (host(vv)[fine] == want[fine]).all()
    assert (host(vv)[~kept] == 0).all()
    # the same among the keys: rows with an infinity or a NaN are kept as NaNs
    a = append(len(rows), 2, 1, D, 0, 16, dt, False, k=v, seed=10)
    odd = ~np.isfinite(host(a["k"])).all(-1)
    huge = np.abs(host(a["k"])).max(-1) > 1e17  # (whose squares may leave fp32)
    sb = np.moveaxis(raw(a["ks"]), 2, 1).reshape(-1, 1)
    for t, sl in enumerate(a["slots"].tolist()):
        if 0 <= sl < a["pages"] * 16 and not huge[t, 0]:
            assert (sb[sl, 0] == 255) == odd[t, 0]


def test_append_stream_and_replay():
    a = append(33, 4, 2, 64, 64, 16, "bf16", False, seed=4)
    want = [raw(a[n]).copy() for n in ("kb", "vb", "ks", "vs")]
    gr = torch.cuda.CUDAGraph()
    out = (a["qo"], a["kb"], a["vb"], a["ks"], a["vs"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gr, stream=s):
        kda.kda_qk_norm_rope_append_q8(*a["head"], *out, *a["tail"], **a["kw"])
    for n in ("kb", "vb"):
        a[n].view(torch.uint8).fill_(0x5A)
    for n in ("ks", "vs"):
        a[n].fill_(0xA5)
    gr.replay()
    torch.cuda.synchronize()
    assert all((raw(a[n]) == w).all() for n, w in zip(("kb", "vb", "ks", "vs"), want))


# ----------------------------------------------------------------------------------- attention

def make(seqs, Hq, Hkv, D, page, dt, seed=0, fill=None, std=1.0, **kw):
    """test_gpu_paged_attention.make with its caches in 8 bits (kb, vb, ks, vs); kc and vc hold what
    they stand for.  fill: the pages of nobody, and places behind the keys, hold NaNs."""
    d = pa.make(seqs, Hq, Hkv, D, page, "f32", seed=seed, fill=None if fill is None else 1e9,
                std=std, **kw)
    rng = np.random.default_rng(seed)
    for n in "kv":
        x = host(d[n + "c"])
        odd = x == 1e9
        x = np.where(odd, 0.0, x) * np.exp(rng.standard_normal(x.shape[:3]))[..., None]
        b, s = q8_ref.quantise(x)
        d[n + "c"] = torch.from_numpy(q8_ref.value(b, s)).cuda()
        if fill == "scale":
            s[odd.all(-1)] = 255
        elif fill == "numbers":
            b[odd] = 0x7F
            s[odd.all(-1)] = 200
        d[n + "b"], d[n + "s"] = e4m3(b), torch.from_numpy(s).cuda()
    d["q"], d["out"], d["dt"] = d["q"].to(DT[dt]), d["out"].to(DT[dt]), dt
    if dt == "bf16":
        x = torch.zeros(d["T"], Hq + 1, D, dtype=DT[dt], device="cuda")
        x[:, :Hq] = d["q"]
        d["q"] = x[:, :Hq]
    return d


def call(d, ws=None, **kw):
    n = kda.kda_paged_attention_q8_fwd_workspace_size(
        d["N"], d["T"], d["Hq"], d["Hkv"], d["D"],
        dtype=kda.KDA_F32 if d["dt"] == "f32" else kda.KDA_BF16)
    if ws is None and n:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    kda.kda_paged_attention_q8_fwd(
        d["q"], d["kb"], d["vb"], d["ks"], d["vs"], d["table"], d["cu"], d["kv"], d["out"],
        d["N"], d["T"], d["Hq"], d["Hkv"], d["D"], d["kb"].shape[0], d["page"],
        d["table"].shape[1], lse=d["lse"], workspace=ws, **kw)


KINDS = pa.KINDS


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_mixed_batch(dt, D, page):
    d = make([(1, 1), (1, 77), (5, 5), (20, 150), (0, 40), (3, 129)], 4, 2, D, page, dt, pad=3)
    call(d)
    pa.check(d)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_one_key_is_read_exactly(dt, D):
    """A token that sees one key returns its value: every number under every scale that the append
    writes."""
    ensure_built()
    H, N = 256 // D, 239
    nums = np.broadcast_to(np.arange(256, dtype=np.uint8).reshape(1, H, 1, D), (N, H, 16, D)).copy()
    nums[nums == 127], nums[nums == 255] = 0, 128
    scales = np.full((N, H, 16), 255, np.uint8)
    scales[:, :, 0] = np.arange(8, 247, dtype=np.uint8)[:, None]
    vb, vs = e4m3(nums), torch.from_numpy(scales).cuda()
    kb = torch.zeros_like(vb.view(torch.uint8)).view(torch.float8_e4m3fn)
    q = torch.ones(N, H, D, dtype=DT[dt], device="cuda")
    out = torch.empty_like(q)
    table = torch.arange(N, dtype=torch.int32, device="cuda")[:, None].contiguous()
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    kv = torch.ones(N, dtype=torch.int32, device="cuda")
    n = kda.kda_paged_attention_q8_fwd_workspace_size(
        N, N, H, H, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    zero = torch.full_like(vs, 127)
    kda.kda_paged_attention_q8_fwd(q, kb, vb, zero, vs, table, cu, kv, out, N, N, H, H, D, N, 16,
                                   1, workspace=ws)
    assert (host(out) == q8_ref.value(nums, scales)[:, :, 0]).all()
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (40, 0), (40, 4), (128, 300), (7, 2)])
def test_window_and_sinks(dt, D, window, sinks):
    d = make([(1, 300), (60, 333), (9, 9), (33, 50)], 6, 2, D, 32, dt, seed=window)
    call(d, window=window, sinks=sinks)
    pa.check(d, window=window, sinks=sinks)


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257])
def test_single_token_lengths(dt, D, kv):
    d = make([(1, kv)], 2, 1, D, 16, dt, seed=kv)
    call(d)
    pa.check(d)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("q,kv,Hq,Hkv", [(127, 127, 1, 1), (128, 128, 2, 2), (129, 300, 1, 1),
                                         (256, 256, 1, 1), (257, 257, 1, 1), (31, 500, 8, 1),
                                         (32, 500, 8, 1), (33, 500, 8, 1), (65, 200, 4, 2),
                                         (100, 100, 5, 1), (43, 640, 3, 1), (2, 700, 64, 1)])
def test_chunk_edges(D, q, kv, Hq, Hkv):
    d = make([(q, kv)], Hq, Hkv, D, 64, "bf16", seed=q)
    call(d)
    pa.check(d)


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("fill", ["scale", "numbers"])
def test_what_lies_outside_the_keys_never_counts(dt, D, page, fill):
    d = make([(1, 130), (4, 67), (70, 201), (1, 1)], 4, 2, D, page, dt, fill=fill)
    call(d)
    pa.check(d)


@pytest.mark.parametrize("dt,D", KINDS)
def test_more_tokens_than_keys_and_no_keys(dt, D):
    d = make([(10, 4), (3, 0), (200, 150)], 2, 2, D, 16, dt, seed=6)
    call(d)
    pa.check(d)
    assert (host(d["out"])[:6] == 0).all()


@pytest.mark.parametrize("dt,D", KINDS)
def test_a_row_of_nan_reaches_what_sees_it(dt, D):
    d = make([(3, 40), (1, 30)], 2, 1, D, 16, dt, seed=8)
    d["vs"][int(d["table_h"][0, 2]), 0, 7] = 255  # key 39, the last token's own
    call(d)
    assert torch.isnan(d["out"][2]).all() and not torch.isnan(d["out"][3]).any()


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_long_and_many(dt, D):
    d = make([(1, 5000), (1, 3), (2, 2501), (1, 1)], 4, 2, D, 64, dt, seed=14)
    call(d)
    pa.check(d)
    d = make([(1, int(k)) for k in np.random.default_rng(1).integers(1, 400, 97)], 8, 2, D, 16, dt)
    call(d)
    pa.check(d)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window", [0, 300])
def test_neighbours_of_any_length(D, window):
    rng = np.random.default_rng(11)
    kv = np.concatenate([rng.integers(1, 400, 350), rng.integers(1, 1600, 350)])
    rng.shuffle(kv)
    d = make([(int(min(k, rng.integers(1, 4))), int(k)) for k in kv], 4, 1, D, 32, "bf16", seed=50)
    call(d, window=window, sinks=2 if window else 0)
    a = d["out"].clone()
    pa.check(d, window=window, sinks=2 if window else 0)
    for _ in range(10):
        call(d, window=window, sinks=2 if window else 0)
        assert torch.equal(a, d["out"])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5)])
def test_chunks_of_several_items_over_long_caches(D, window, sinks):
    for Hq, Hkv, page in ((2, 1, 64), (5, 1, 16), (2, 2, 128)):
        d = make([(300, 2100), (1, 900), (411, 1300), (140, 140)], Hq, Hkv, D, page, "bf16",
                 seed=D + Hq, pad=1)
        call(d, window=window, sinks=sinks)
        pa.check(d, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [32, 64, 128])
def test_chunks_in_fp32(D):
    for Hq, Hkv, page in ((4, 2, 64), (5, 1, 16)):
        d = make([(100, 100), (1, 700), (16, 16), (0, 9), (17, 300), (64, 64), (65, 900)], Hq, Hkv,
                 D, page, "f32", seed=3, pad=2, fill="scale")
        call(d)
        pa.check(d)


@pytest.mark.parametrize("dt,D", KINDS)
def test_more_sequences_than_threads(dt, D):
    rng = np.random.default_rng(7)
    for N, most in ((1000, 4), (1500, 21)):
        d = make([(int(q), int(q + k)) for q, k in zip(rng.integers(0, most, N),
                                                       rng.integers(0, 40, N))], 2, 1, D, 16, dt)
        call(d)
        pa.check(d)


@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (10, 2), (64, 1), (160, 1), (7, 7)])
def test_head_groups(Hq, Hkv):
    for dt, D in (("bf16", 64), ("bf16", 128), ("f32", 32)):
        d = make([(1, 70), (40, 140), (3, 3)], Hq, Hkv, D, 32, dt, seed=Hq)
        call(d)
        pa.check(d)


@pytest.mark.parametrize("dt,D", KINDS)
def test_sixteen_byte_alignment(dt, D):
    d = make([(1, 200), (50, 180)], 4, 2, D, 16, dt, seed=40)
    for n in ("q", "kb", "vb", "ks", "vs", "out", "lse", "table", "cu", "kv"):
        x = d[n].contiguous()
        pad = 16 // x.element_size()
        flat = torch.empty(x.numel() + pad, dtype=x.dtype, device="cuda")
        y = flat[pad:].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        d[n] = y
    call(d)
    pa.check(d)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f32", 64)])
def test_cache_beyond_32_bit_offsets(dt, D):
    """A cache of more than 2^32 numbers whose far pages are the ones in use."""
    d = make([(1, 600), (40, 300)], 4, 2, D, 64, dt, seed=16)
    near = d["kb"].shape[0]
    pages = (1 << 32) // (2 * 64 * D) + near
    shift = pages - near
    for n in ("kb", "vb", "ks", "vs"):
        big = torch.empty(pages, *d[n].shape[1:], dtype=torch.uint8, device="cuda")
        big[shift:] = d[n].view(torch.uint8)
        d[n] = big.view(d[n].dtype)
    d["table"] += shift
    call(d)
    pa.check(d)
    slots = torch.tensor([shift * 64 + 5, pages * 64 - 1], device="cuda")
    k, _ = read(d["kb"], d["vb"], d["ks"], d["vs"], slots, "f32", 64)
    flat = host(d["kc"]).transpose(0, 2, 1, 3).reshape(-1, 2, D)
    assert (host(k) == flat[[5, -1]]).all()


@pytest.mark.parametrize("dt,D", [("bf16", 32), ("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_bad_pages_and_lengths_are_clamped(dt, D):
    d = make([(2, 100), (1, 40), (1, 64)], 2, 1, D, 16, dt, pad=2, seed=90)
    maxp = d["table"].shape[1]
    d["table"][0, 1], d["table"][0, 2] = 2 ** 31 - 1, -2 ** 31
    d["kv"][1], d["kv"][2] = 2 ** 31 - 1, -5
    d["table_h"] = np.clip(d["table"].cpu().numpy().astype(np.int64), 0, d["kb"].shape[0] - 1)
    d["kv_h"] = np.array([100, 16 * maxp, 0])
    call(d)
    pa.check(d)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_repeat_stream_and_replay_give_the_same_bits(dt, D):
    d = make([(1, 3000), (90, 800), (1, 20), (5, 1200)], 8, 2, D, 32, dt, seed=15)
    call(d)
    a, l = d["out"].clone(), d["lse"].clone()
    s = torch.cuda.Stream()
    d["out"].fill_(1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(d)
    s.synchronize()
    assert torch.equal(a, d["out"]) and torch.equal(l, d["lse"])
    n = kda.kda_paged_attention_q8_fwd_workspace_size(
        d["N"], d["T"], 8, 2, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(d, ws=ws)
    ws.fill_(0xFF)
    for _ in range(2):
        d["out"].fill_(1)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, d["out"]) and torch.equal(l, d["lse"])
    d["kv"].sub_(torch.tensor([1500, 0, 5, 0], dtype=torch.int32, device="cuda"))
    d["kv_h"] = host(d["kv"]).astype(np.int32)
    gr.replay()
    torch.cuda.synchronize()
    pa.check(d)


def test_two_calls_at_once():
    ds = [make([(1, 700), (130, 900), (1, 64), (7, 2000)], 8, 2, 128, 64, "bf16", seed=70),
          make([(1, int(k)) for k in range(40, 1500, 23)], 8, 2, 64, 32, "bf16", seed=71)]
    want, ws = [], []
    for d in ds:
        call(d)
        want.append(d["out"].clone())
        n = kda.kda_paged_attention_q8_fwd_workspace_size(d["N"], d["T"], 8, 2, d["D"])
        ws.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for d in ds:
            d["out"].fill_(5)
        torch.cuda.synchronize()
        for d, w, s in zip(ds, ws, streams):
            with torch.cuda.stream(s):
                call(d, ws=w)
        torch.cuda.synchronize()
        assert all(torch.equal(x, d["out"]) for x, d in zip(want, ds))
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_empty_calls(dt):
    d = make([(2, 5)], 2, 1, 64, 16, dt)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    kda.kda_paged_attention_q8_fwd(d["q"], d["kb"], d["vb"], d["ks"], d["vs"], d["table"], d["cu"],
                                   d["kv"], d["out"], 0, 0, 2, 1, 64, d["kb"].shape[0], 16,
                                   d["table"].shape[1])
    kda.kda_paged_attention_q8_fwd(d["q"], None, None, None, None, None, d["cu"], d["kv"],
                                   d["out"], 1, 2, 2, 1, 64, 0, 16, 0, workspace=ws)
    torch.cuda.synchronize()
    assert (d["out"] == 0).all()


# --------------------------------------------------------------------------- few rows, odd queries

@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (3, 1), (4, 2), (5, 1), (8, 1), (9, 1), (12, 1),
                                   (16, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5), (1, 200)])
@pytest.mark.parametrize("D", [128, 64])
def test_few_rows(G, Hkv, window, sinks, D):
    """Up to 16 rows of a sequence, items of 16 where some have more; none, fewer keys than tokens,
    many tiles, several items in a block and cut ones."""
    d = make([(1, 1), (1, 129), (2, 300), (1, 0), (3, 1), (0, 7), (2, 2000), (1, 128), (1, 5000)] +
             [(0, 3)] * 6, G * Hkv, Hkv, D, 64, "bf16", seed=G + window, pad=2, fill="scale")
    assert d["T"] * G <= 16 * d["N"]  # (16 rows a sequence on average, or fewer)
    call(d, window=window, sinks=sinks)
    pa.check(d, window=window, sinks=sinks)


@pytest.mark.parametrize("G,Hkv,few", [(1, 2, 32), (4, 2, 8), (5, 1, 6), (8, 1, 4), (9, 1, 3),
                                       (16, 2, 2), (17, 1, 1), (32, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5), (1, 200)])
@pytest.mark.parametrize("D", [128, 64])
def test_up_to_32_rows(G, Hkv, few, window, sinks, D):
    """Items of 32 rows, full ones, those of a row more than a half and less; none, fewer keys than
    tokens, many tiles, several items in a block and cut ones.  (few: tokens of 32 rows.)"""
    seqs = [(few, 1), (few, 129), (few // 2 + 1, 300), (few, 0), (few + 1, 1), (few, 7), (1, 2000),
            (few, 128), (few, 5000), (0, 3), (few + 2, 700)] + [(few, 60)] * 4
    T = sum(q for q, _ in seqs)
    seqs += [(0, 3)] * max(0, (T * G + 31) // 32 - len(seqs))
    d = make(seqs, G * Hkv, Hkv, D, 64, "bf16", seed=G + window, pad=2, fill="scale")
    assert 16 * d["N"] < T * G <= 32 * d["N"]  # (17 to 32 rows a sequence on average)
    call(d, window=window, sinks=sinks)
    pa.check(d, window=window, sinks=sinks)


def test_few_rows_of_a_batch_whose_tables_are_near_the_limit():
    """Block tables so wide that items of 16 rows could pass the 31 bits of the line, while those of
    256 rows, which the limit is about, could not."""
    d = make([(1, 70), (1, 0), (1, 300)], 64, 4, 128, 128, "bf16", seed=3)
    N, pages = 65535, 6000
    assert (N * 16 / 16 + N) * 4 * (pages + 4) > 2 ** 31 > (N * 16 / 256 + N) * 4 * (pages + 5)
    table = d["table"].new_zeros((N, pages))
    table[:3, :d["table"].shape[1]] = d["table"]
    cu = torch.full((N + 1,), 3, dtype=torch.int32, device="cuda")
    cu[:4] = d["cu"]
    kv = torch.zeros(N, dtype=torch.int32, device="cuda")
    kv[:3] = d["kv"]
    q = torch.zeros((N, 64, 128), dtype=torch.bfloat16, device="cuda")
    q[:3] = d["q"]
    out, lse = torch.empty_like(q), torch.empty((N, 64), device="cuda")
    ws = torch.empty(kda.kda_paged_attention_q8_fwd_workspace_size(N, N, 64, 4, 128),
                     dtype=torch.uint8, device="cuda")
    kda.kda_paged_attention_q8_fwd(q, d["kb"], d["vb"], d["ks"], d["vs"], table, cu, kv, out, N, N,
                                   64, 4, 128, d["kb"].shape[0], 128, pages, lse=lse, workspace=ws)
    d["out"], d["lse"] = out[:3].contiguous(), lse[:3].contiguous()
    pa.check(d)


@pytest.mark.parametrize("slope", [20.0, 150.0, 600.0, -300.0])
@pytest.mark.parametrize("D", [128, 64])
def test_rising_scores_of_few_rows_and_of_chunks(slope, D):
    """Scores that grow along the keys: the standing maximum moves, by less and more than what is
    taken without scaling anew."""
    for seqs in ([(1, 1500), (2, 1500), (1, 130)], [(15, 1500), (12, 130), (16, 1500)],
                 [(200, 1500), (130, 130), (1, 1500)]):
        d = make(seqs, 2, 1, D, 64, "bf16", seed=13)
        k = np.zeros(tuple(d["kb"].shape))
        for n in range(3):
            for j in range(int(d["kv_h"][n])):
                k[int(d["table_h"][n, j // 64]), :, j % 64] = slope * j / 1500 / D
        b, s = q8_ref.quantise(k)
        d["kb"], d["ks"] = e4m3(b), torch.from_numpy(s).cuda()
        d["kc"] = torch.from_numpy(q8_ref.value(b, s)).cuda()
        d["q"].copy_(torch.rand_like(d["q"].float()) + 0.5)
        call(d, softmax_scale=1.0)
        pa.check(d, scale=1.0)


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("tokens", [1, 7, 150])
def test_queries_of_all_magnitudes(dt, D, tokens):
    """Rows of zeros, of the smallest and of large numbers, and of numbers of very different sizes;
    an infinity or a NaN in one row stays in it.  Scores of e^+-87 at most, so that nothing overflows."""
    d = make([(tokens, 400), (tokens, 300), (tokens, 200)], 4, 1, D, 64, dt, seed=5)
    q = d["q"].float().clone()
    q[0, 0] = 0
    q[0, 1] *= 1e-30
    q[0, 2] *= 3.0
    q[0, 3, ::2] *= 2.0 ** -9
    d["q"].copy_(q)
    call(d)
    pa.check(d)
    # next to no scale: all keys alike
    call(d, softmax_scale=1e-30)
    pa.check(d, scale=1e-30)
    a = d["out"].clone()
    d["q"][tokens, 2, 3] = float("inf")
    d["q"][tokens, 1, 0] = float("nan")
    call(d, softmax_scale=1e-30)
    same = torch.ones(d["T"], 4, dtype=torch.bool, device="cuda")
    same[tokens, 1:3] = False
    assert torch.equal(a[same], d["out"][same])
    assert torch.isnan(d["out"][tokens, 1]).all() and not torch.isfinite(d["out"][tokens, 2]).any()


@pytest.mark.parametrize("tokens", [1, 5, 100])
@pytest.mark.parametrize("D", [128, 64])
def test_graphs_that_share_a_workspace(tokens, D):
    """Two captured calls with one buffer, replayed in turn."""
    ds = [make([(tokens, 700), (tokens, 900), (1, 64)], 8, 2, D, 64, "bf16", seed=70),
          make([(tokens, int(k)) for k in range(140, 1500, 99)], 8, 2, D, 32, "bf16", seed=71)]
    n = max(kda.kda_paged_attention_q8_fwd_workspace_size(d["N"], d["T"], 8, 2, D) for d in ds)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, want = [], []
    for d in ds:
        call(d)
        want.append(d["out"].clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(d, ws=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        ds[i]["out"].fill_(3)
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(ds[i]["out"], want[i])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("R", [0, 32])
def test_keys_whose_squares_leave_fp32(dt, D, R):
    """Finite keys whose sum of squares overflows: 1 / rms is zero, so they become rows of zeros, as
    kda_qk_norm_rope_append makes them; 255 is for rows that hold an infinity or a NaN.  A row of
    1e18 at the head's last element alone, whose square does not overflow, is normed."""
    rng = np.random.default_rng(3)
    rows = [np.full(D, 3.3e38), np.full(D, -3e38), rng.standard_normal(D) * 1e30,
            np.r_[np.zeros(D - 1), 3e19], np.r_[-2e38, np.ones(D - 1)],
            np.r_[np.zeros(D - 1), 1e18],
            np.r_[np.full(D - 1, 3e38), np.inf], np.r_[np.nan, np.full(D - 1, 3e38)],
            np.full(D, -np.inf), rng.standard_normal(D)]
    k = torch.from_numpy(np.stack(rows)[:, None]).to("cuda", DT[dt])
    T = len(rows)
    a = append(T, 2, 1, D, R, 16, dt, False, k=k, seed=11)
    kc, vc = (torch.full((a["pages"], 1, 16, D), 7.0, dtype=DT[dt], device="cuda")
              for _ in range(2))
    kda.kda_qk_norm_rope_append(*a["head"], torch.empty_like(a["qo"]), kc, vc, *a["tail"],
                                **a["kw"])
    want = host(kc)[:, 0].reshape(-1, D)
    got = q8_ref.value(raw(a["kb"]), raw(a["ks"]))[:, 0].reshape(-1, D)
    byte = raw(a["ks"])[:, 0].reshape(-1)
    slots = a["slots"].tolist()
    assert sum(0 <= s < a["pages"] * 16 for s in slots) == T - 2
    for t, s in enumerate(slots):
        if not 0 <= s < a["pages"] * 16:
            continue
        if t < 5:
            assert (want[s] == 0).all() and (got[s] == 0).all() and byte[s] == q8_ref.LO + 127
        elif t in (6, 7, 8):
            assert byte[s] == 255 and not np.isfinite(want[s]).all()
        else:
            # one rounding to e4m3 (2^-4), one to bf16 (2^-8), and fp32's of norm and rotation
            lim = (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -15) * np.abs(want[s]) + 2.0 ** -9 * \
                2.0 ** (int(byte[s]) - 127) + (D + 24) * 2.0 ** -24 * np.abs(want[s]).max()
            assert byte[s] != 255 and np.abs(want[s]).max() > 0.1
            assert (np.abs(got[s] - want[s]) <= lim).all()


EXTREMES = [(2.0 ** 114, 2.0 ** -102), (2.98e38, 2.0 ** -102), (2.0 ** 100, 2.0 ** -90),
            (2.0 ** -110, 2.0 ** 122)]


def keys_of_one_magnitude(shape, k, seed):
    """Rows of one number, k or -k, in 8 bits: (numbers, scale bytes, signs [pages, Hkv, page])."""
    sign = np.where(np.random.default_rng(seed).random(shape[:3]) < 0.5, -1.0, 1.0)
    b, s = q8_ref.quantise(np.broadcast_to(sign[..., None] * k, shape))
    return b, s, sign


def check_one_magnitude(out, lse, k, q, sign, V, D):
    """One query row of elements q against keys of k sign_j: scores are +-S, S = q k sqrt(D) of 2^13
    or more, so the result is the mean of the values of the visible keys with the larger score.  A
    score in log2 has an error of up to 8 roundings (products, maxima, joined parts): the weights of
    equal ones differ by that at most, and a mean of any weights lies between its values."""
    S = q * k * D ** 0.5
    best = sign == sign.max()
    v, err = V[best], 2.0 ** -21 * S * 1.4427
    A = np.abs(v).mean(0)
    slack = 2.0 ** -7 * (A + np.abs(v).max(0) * 2.0 ** -8)
    assert np.isfinite(out).all()
    assert (out >= v.min(0) - slack).all() and (out <= v.max(0) + slack).all()
    if err < 0.1:
        assert (np.abs(out - v.mean(0)) <= 2 * err * A + 2.0 ** -8 * (A + np.abs(v.mean(0)))).all()
    want = sign.max() * S + np.log(best.sum())
    assert abs(lse - want) <= 2.0 ** -19 * S + 1e-3


@pytest.mark.parametrize("k,q", EXTREMES)
@pytest.mark.parametrize("tokens", [1, 6, 150])
@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 128)])
def test_keys_of_all_magnitudes(dt, D, tokens, k, q):
    """Keys up to the largest that a row can hold beside small queries, and the other way round:
    their products are in range, so no way to them may leave it."""
    d = make([(tokens, 700), (tokens, tokens), (tokens, 300)], 4, 1, D, 64, dt, seed=21)
    b, s, sign = keys_of_one_magnitude(d["kb"].shape, k, 5)
    k = float(q8_ref.value(b, s).max())
    d["kb"], d["ks"] = e4m3(b), torch.from_numpy(s).cuda()
    d["q"].fill_(q)
    call(d)
    out, lse, V = host(d["out"]), host(d["lse"]), host(d["vc"])
    for n in range(3):
        kv, t0 = int(d["kv_h"][n]), int(d["cu_h"][n])
        sg = q8_ref.rows_of(sign, d["table_h"][n], kv, 64)[:, 0]
        v = q8_ref.rows_of(V, d["table_h"][n], kv, 64)[:, 0]
        for i in range(tokens):
            m = kv - tokens + i + 1
            for h in range(4):
                check_one_magnitude(out[t0 + i, h], lse[t0 + i, h], k, q, sg[:m], v[:m], D)
    assert kda.kda_device_error() == 0


RISES = [15.0, 30.0, 36.0, 44.0, 48.0, 52.0, 56.0, 60.0, 72.0]
LN2 = float(np.float32(np.log(2)))


class Rise:
    """Lists of keys in pages of 64 whose scores, in log2, are 0 and from key `at` of each list on
    `top`, the same for every query, and whose values are `large` times 1/2 to 1: the largest sums
    that values can have.  In 8 bits, or (q8 False) in bf16."""

    def __init__(self, lists, Hkv, D, top, at, large, q8=True):
        ensure_built()
        need, rng = [-(-n // 64) for n in lists], np.random.default_rng(7)
        self.lists, self.Hkv, self.D, self.pages = lists, Hkv, D, sum(need)
        self.table = np.zeros((len(lists), max(need)), np.int32)
        k = np.zeros((self.pages, Hkv, 64, 1))
        for i, m in enumerate(need):
            self.table[i, :m] = sum(need[:i]) + np.arange(m)
            j = np.arange(64 * m).reshape(m, 1, 64, 1)
            k[self.table[i, :m]] = np.where(j < at, 0.0, top)
        x = {"k": k, "v": rng.uniform(0.5, 1.0, k.shape) * large}
        for n in "kv":
            shape = (*k.shape[:3], D)
            if q8:
                b, s = q8_ref.quantise(x[n])
                x[n] = q8_ref.value(b, s)
                full, s = torch.zeros(shape, dtype=torch.uint8), torch.from_numpy(s).cuda()
                b = torch.from_numpy(b)
            else:
                b, s = torch.from_numpy(x[n]).to(torch.bfloat16), None
                x[n] = host(b)
                full = torch.zeros(shape, dtype=torch.bfloat16)
            full[..., :1 if n == "k" else D] = b  # keys: all in the first column
            setattr(self, n + "c", full.cuda().view(torch.float8_e4m3fn) if q8 else full.cuda())
            setattr(self, n + "s", s)
        self.x = x

    def of(self, i):
        """Scores and values [keys, Hkv] of a list."""
        return [q8_ref.rows_of(self.x[n], self.table[i], self.lists[i], 64)[..., 0] for n in "kv"]

    def queries(self, tokens, G):
        """Queries whose score is a key's first element, offsets, and places for the results."""
        cu = np.concatenate([[0], np.cumsum(tokens)])
        q = torch.zeros(cu[-1], G * self.Hkv, self.D, dtype=torch.bfloat16, device="cuda")
        q[:, :, 0] = 1
        return q, cu, torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")


def check_rise(out, lse, k, v, D):
    """A sequence's tokens, [tokens, Hq, D], against sums along its scores and values.  Tolerances
    as test_gpu_paged_attention.compare's."""
    k, v, tokens = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda(), out.shape[0]
    out = out.double().view(tokens, k.shape[1], -1, D)  # [tokens, Hkv, G, D]
    p = torch.exp2(k - k.max())
    l, o = (x.cumsum(0)[-tokens:] for x in (p, p * v))
    want = (o / l)[:, :, None, None]
    dl = (D + 8) * 2.0 ** -24 * float(k.max()) * LN2
    lim = 2 * dl + (len(k) + 64) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -7
    bad = ~((out - want).abs() <= lim * want)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:3], out[bad][:3])
    want = (float(k.max()) * LN2 + l.log())[:, :, None]
    lse = lse.double().view(tokens, k.shape[1], -1)
    assert ((lse - want).abs() <= dl + 2.0 ** -22 * (want.abs() + 3 + len(k) / 16)).all()


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).cuda()


@pytest.mark.parametrize("at,top,large",
                         [(at, top, 2.0 ** 84) for at in (40, 700) for top in RISES] +
                         [(40, top, 2.0 ** -107) for top in (0.0, 15.0, 60.0)])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_large_values_under_rising_scores(D, at, top, large):
    """Scores that rise by 2^top at once, up to what the standing maximum absorbs and beyond, over
    1500 (less than 2^11) values of up to 2^84: nothing overflows on the way.  Many heads, so that
    one block has most of a row's keys.  And over the smallest values."""
    for tokens, Hkv in (([1, 2], 100), ([12, 16], 100), ([130, 200], 50)):
        r = Rise([1500, 1400], Hkv, D, top, at, large)
        q, cu, out, lse = r.queries(tokens, 2)
        ws = torch.empty(kda.kda_paged_attention_q8_fwd_workspace_size(2, len(q), 2 * Hkv, Hkv, D),
                         dtype=torch.uint8, device="cuda")
        kda.kda_paged_attention_q8_fwd(
            q, r.kc, r.vc, r.ks, r.vs, i32(r.table), i32(cu), i32(r.lists), out, 2, len(q),
            2 * Hkv, Hkv, D, r.pages, 64, r.table.shape[1], lse=lse, softmax_scale=LN2,
            workspace=ws)
        for n in range(2):
            check_rise(out[cu[n]:cu[n + 1]], lse[cu[n]:cu[n + 1]], *r.of(n), D)
    assert kda.kda_device_error() == 0
