"""kda_paged_attention_fwd against the fp64 definition.

Tolerances, per element.  A score is a sum of D products in fp32, scaled: off by at most
d = (D + 8) 2^-24 Z with Z the largest sum |q k| scale of the row; every softmax weight is then
off by at most 2 d + (n + 64) 2^-24 relative (numerator and denominator, n keys summed), so the
output by that times A = sum p |v|.  bf16 weights of the tensor-core path add 2^-8 A (half a
step on each weight) and the output's own rounding 2^-8 |o|.  lse: d + 2^-22 (|lse| + 1 + n 2^-4)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import serving_ref as ref  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(x):
    return x.detach().double().cpu().numpy()


def make(seqs, Hq, Hkv, D, page, dt, seed=0, spare=3, pad=0, fill=None, std=1.0):
    """seqs: (new tokens, keys in all).  Keys and pages that no sequence has hold `fill`."""
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum([q for q, _ in seqs])]).astype(np.int32)
    T = int(cu[-1]) + pad
    kv = np.array([k for _, k in seqs], np.int32)
    need = [-(-int(k) // page) for k in kv]
    pages, maxp = sum(need) + spare, max(need + [1]) + 1
    table = np.full((len(seqs), maxp), -7 if fill is not None else 0, np.int32)
    perm = np.random.default_rng(seed).permutation(pages)
    at = 0
    for n, m in enumerate(need):
        table[n, :m] = perm[at:at + m]
        at += m
    kc, vc = (torch.randn(pages, Hkv, page, D, generator=g, device="cuda") for _ in range(2))
    kc *= std
    if fill is not None:
        own = torch.zeros(pages, 1, page, 1, dtype=torch.bool, device="cuda")
        for n, m in enumerate(need):
            for i in range(m):
                own[int(table[n, i]), 0, :min(page, int(kv[n]) - i * page)] = True
        kc, vc = (torch.where(own, x, torch.full_like(x, fill)) for x in (kc, vc))
    q = torch.randn(T, Hq + 1, D, generator=g, device="cuda").to(DT[dt])[:, :Hq]
    return dict(q=q, kc=kc.to(DT[dt]), vc=vc.to(DT[dt]), table=torch.from_numpy(table).cuda(),
                cu=torch.from_numpy(cu).cuda(), kv=torch.from_numpy(kv).cuda(), cu_h=cu, kv_h=kv,
                table_h=table, page=page, D=D, Hq=Hq, Hkv=Hkv, N=len(seqs), T=T, dt=dt,
                out=torch.full((T, Hq, D), 7.0, dtype=DT[dt], device="cuda"),
                lse=torch.full((T, Hq), 7.0, device="cuda"), live=int(cu[-1]))


def call(d, ws=None, **kw):
    n = kda.kda_paged_attention_fwd_workspace_size(
        d["N"], d["T"], d["Hq"], d["Hkv"], d["D"],
        dtype=kda.KDA_F32 if d["dt"] == "f32" else kda.KDA_BF16)
    if ws is None and n:
        ws = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
    kda.kda_paged_attention_fwd(d["q"], d["kc"], d["vc"], d["table"], d["cu"], d["kv"], d["out"],
                                d["N"], d["T"], d["Hq"], d["Hkv"], d["D"], d["kc"].shape[0],
                                d["page"], d["table"].shape[1], lse=d["lse"], workspace=ws, **kw)


def check(d, **kw):
    r = ref.paged_attention(host(d["q"])[:d["live"]], host(d["kc"]), host(d["vc"]), d["table_h"],
                            d["cu_h"], d["kv_h"], d["page"], **kw)
    compare(d, r)
    assert (host(d["out"])[d["live"]:] == 7.0).all()
    assert (host(d["lse"])[d["live"]:] == 7.0).all()


def compare(d, r):
    out, lse, A, Z = r
    n = int(max(d["kv_h"], default=0))
    dl = (d["D"] + 8) * 2.0 ** -24 * Z
    lim = (2 * dl + (n + 64) * 2.0 ** -24)[..., None] * A
    if d["dt"] == "bf16":
        lim = lim + 2.0 ** -8 * (A + np.abs(out))
    got = host(d["out"])[:d["live"]]
    bad = ~(np.abs(got - out) <= lim)
    assert not bad.any(), (np.abs(got - out)[bad].max(), int(bad.sum()), np.argwhere(bad)[:5])
    gl = host(d["lse"])[:d["live"]]
    empty = np.isneginf(lse)
    assert (np.isneginf(gl) == empty).all()
    ok = ~empty
    assert (np.abs(gl[ok] - lse[ok]) <= dl[ok] + 2.0 ** -22 * (np.abs(lse[ok]) + 1 + n / 16)).all()
    assert kda.kda_device_error() == 0


KINDS = [("f32", 32), ("f32", 64), ("f32", 128), ("bf16", 32), ("bf16", 64), ("bf16", 128)]


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("page", [16, 128])
def test_mixed_batch(dt, D, page):
    d = make([(1, 1), (1, 77), (5, 5), (20, 150), (0, 40), (3, 129)], 4, 2, D, page, dt, pad=3)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 32), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (40, 0), (40, 4), (128, 300), (7, 2)])
def test_window_and_sinks(dt, D, window, sinks):
    d = make([(1, 300), (60, 333), (9, 9), (33, 50)], 6, 2, D, 32, dt, seed=window)
    call(d, window=window, sinks=sinks)
    check(d, window=window, sinks=sinks)


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("kv", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257])
def test_single_token_lengths(dt, D, kv):
    d = make([(1, kv)], 2, 1, D, 16, dt, seed=kv)
    call(d)
    check(d)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q,kv,Hq,Hkv", [(127, 127, 1, 1), (128, 128, 2, 2), (129, 300, 1, 1),
                                         (256, 256, 1, 1), (257, 257, 1, 1), (31, 500, 8, 1),
                                         (32, 500, 8, 1), (33, 500, 8, 1), (65, 200, 4, 2),
                                         (100, 100, 5, 1), (43, 640, 3, 1), (2, 700, 64, 1)])
def test_chunk_edges(D, q, kv, Hq, Hkv):
    d = make([(q, kv)], Hq, Hkv, D, 64, "bf16", seed=q)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D", [("f32", 64), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
def test_what_lies_outside_the_keys_never_counts(dt, D, page, fill):
    d = make([(1, 130), (4, 67), (70, 201), (1, 1)], 4, 2, D, page, dt, fill=fill)
    call(d)
    check(d)


@pytest.mark.parametrize("D", [64, 128])
def test_keys_behind_the_window_may_hold_anything(D):
    """Single tokens: the pages that left the window are free, whatever they hold by now."""
    d = make([(1, 500), (1, 90), (1, 700)], 4, 2, D, 32, "bf16", seed=4)
    w, s = 100, 5
    r = ref.paged_attention(host(d["q"]), host(d["kc"]), host(d["vc"]), d["table_h"], d["cu_h"],
                            d["kv_h"], 32, window=w, sinks=s)
    for n, kv in enumerate(d["kv_h"]):
        for j in range(s, max(s, int(kv) - w)):
            p = int(d["table_h"][n, j // 32])
            d["kc"][p, :, j % 32] = float("nan")
            d["vc"][p, :, j % 32] = float("nan")
    call(d, window=w, sinks=s)
    compare(d, r)


def test_more_tokens_than_keys_and_no_keys():
    for dt, D in (("f32", 64), ("bf16", 128)):
        d = make([(10, 4), (3, 0), (200, 150)], 2, 2, D, 16, dt, seed=6)
        call(d)
        check(d)
        assert (host(d["out"])[:6] == 0).all()


def test_bad_pages_and_lengths_stay_inside_the_cache():
    """Entries outside the cache are clamped: wrong numbers, no fault, no other row touched."""
    for dt, D in (("f32", 64), ("bf16", 64), ("bf16", 128)):
        d = make([(2, 100), (1, 40), (1, 64)], 2, 1, D, 16, dt, pad=2)
        d["table"][0, 1] = 2 ** 31 - 1
        d["table"][0, 2] = -2 ** 31
        d["kv"][1] = 2 ** 31 - 1
        d["kv"][2] = -5
        d["cu"][3] = 2 ** 30
        call(d)
        torch.cuda.synchronize()
        assert kda.kda_device_error() == 0


def test_scale_and_sharp_softmax():
    """Large scores of both signs: one key takes all."""
    for dt, D in (("f32", 128), ("bf16", 64), ("bf16", 128)):
        d = make([(3, 400), (40, 300)], 4, 4, D, 64, dt, std=30.0, seed=12)
        call(d, softmax_scale=0.7)
        check(d, scale=0.7)


def test_rising_scores():
    """Keys whose scores grow along the sequence: the running maximum moves at every tile."""
    for D in (64, 128):
        d = make([(1, 1500), (64, 1500)], 2, 1, D, 64, "bf16", seed=13)
        ramp = {}
        for n in range(2):
            for j in range(1500):
                ramp[int(d["table_h"][n, j // 64]), j % 64] = j / 1500 * 20
        for (p, o), x in ramp.items():
            d["kc"][p, :, o] = x / D
        d["q"].copy_(torch.rand_like(d["q"]) + 0.5)
        call(d, softmax_scale=1.0)
        check(d, scale=1.0)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_long_and_many(dt, D):
    """Few rows over long caches (cut along the keys) beside short ones."""
    d = make([(1, 5000), (1, 3), (2, 2501), (1, 1)], 4, 2, D, 64, dt, seed=14)
    call(d)
    check(d)
    d = make([(1, int(k)) for k in np.random.default_rng(1).integers(1, 400, 97)], 8, 2, D, 16, dt)
    call(d)
    check(d)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [0, 700])
def test_many_tiles_of_single_tokens(D, window):
    """Enough single tokens over long caches that every block walks many tiles and items."""
    kv = np.random.default_rng(3).integers(300, 3500, 36)
    d = make([(1, int(k)) for k in kv], 32, 16, D, 64, "bf16", seed=30)
    call(d, window=window, sinks=3 if window else 0)
    a = d["out"].clone()
    check(d, window=window, sinks=3 if window else 0)
    for _ in range(20):
        call(d, window=window, sinks=3 if window else 0)
        assert torch.equal(a, d["out"])


@pytest.mark.parametrize("D", [64, 128])
def test_repeat_stream_and_replay_give_the_same_bits(D):
    d = make([(1, 3000), (90, 800), (1, 20), (5, 1200)], 8, 2, D, 32, "bf16", seed=15)
    call(d)
    a, l = d["out"].clone(), d["lse"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    d["out"].fill_(1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(d)
    s.synchronize()
    assert torch.equal(a, d["out"]) and torch.equal(l, d["lse"])
    n = kda.kda_paged_attention_fwd_workspace_size(d["N"], d["T"], 8, 2, D)
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
    # new lengths under the same graph
    d["kv"].sub_(torch.tensor([1500, 0, 5, 0], dtype=torch.int32, device="cuda"))
    d["kv_h"] = host(d["kv"]).astype(np.int32)
    gr.replay()
    torch.cuda.synchronize()
    check(d)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f32", 64)])
def test_cache_beyond_32_bit_offsets(dt, D):
    """A cache of more than 2^32 elements whose far pages are the ones in use."""
    d = make([(1, 600), (40, 300)], 4, 2, D, 64, dt, seed=16)
    near = d["kc"].shape[0]
    per = 2 * 64 * D
    pages = (1 << 32) // per + near
    shift = pages - near
    for n in ("kc", "vc"):
        big = torch.empty(pages, 2, 64, D, dtype=DT[dt], device="cuda")
        big[shift:] = d[n]
        d[n + "0"], d[n] = d[n], big
    d["table"] += shift
    call(d)
    d["kc"], d["vc"] = d["kc0"], d["vc0"]
    check(d)


@pytest.mark.parametrize("dt,D", KINDS)
def test_more_sequences_than_threads(dt, D):
    """1000 and 1500 sequences of 0 to 20 tokens: several rounds of the kernels' search for their
    rows, and no search."""
    rng = np.random.default_rng(7)
    for N, most in ((1000, 4), (1500, 21)):
        d = make([(int(q), int(q + k)) for q, k in zip(rng.integers(0, most, N),
                                                       rng.integers(0, 40, N))], 2, 1, D, 16, dt)
        call(d)
        check(d)


@pytest.mark.parametrize("Hq,Hkv", [(3, 1), (10, 2), (64, 1), (128, 1), (160, 1), (7, 7)])
def test_head_groups(Hq, Hkv):
    for dt, D in (("bf16", 64), ("bf16", 128), ("f32", 32)):
        d = make([(1, 70), (40, 140), (3, 3)], Hq, Hkv, D, 32, dt, seed=Hq)
        call(d)
        check(d)


@pytest.mark.parametrize("dt,D", KINDS)
def test_sixteen_byte_alignment(dt, D):
    """Buffers on 16-byte boundaries that are no 32-byte ones."""
    d = make([(1, 200), (50, 180)], 4, 2, D, 16, dt, seed=40)
    for n in ("q", "kc", "vc", "out", "lse", "table", "cu", "kv"):
        x = d[n]
        pad = 16 // x.element_size()
        flat = torch.empty(x.numel() + pad, dtype=x.dtype, device="cuda")
        y = flat[pad:].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        d[n] = y
    call(d)
    check(d)


def test_empty_calls():
    d = make([(1, 5)], 2, 1, 64, 16, "f32")
    kda.kda_paged_attention_fwd(d["q"], d["kc"], d["vc"], d["table"], d["cu"], d["kv"], d["out"],
                                0, 0, 2, 1, 64, d["kc"].shape[0], 16, d["table"].shape[1])
    # a cache without pages: nothing to see
    for dt, D in (("f32", 64), ("bf16", 128)):
        d = make([(2, 5)], 2, 1, D, 16, dt)
        n = kda.kda_paged_attention_fwd_workspace_size(
            1, 2, 2, 1, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        kda.kda_paged_attention_fwd(d["q"], None, None, None, d["cu"], d["kv"], d["out"], 1, 2, 2,
                                    1, D, 0, 16, 0, workspace=ws)
        torch.cuda.synchronize()
        assert (d["out"] == 0).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window", [0, 300])
def test_neighbours_of_any_length(D, window):
    """Single tokens and short chunks whose neighbours have fewer, as many or more key tiles, so
    that every block meets each of these pairs."""
    rng = np.random.default_rng(11)
    kv = np.concatenate([rng.integers(1, 400, 350), rng.integers(1, 1600, 350)])
    rng.shuffle(kv)
    d = make([(int(min(k, rng.integers(1, 4))), int(k)) for k in kv], 4, 1, D, 32, "bf16", seed=50)
    call(d, window=window, sinks=2 if window else 0)
    a = d["out"].clone()
    check(d, window=window, sinks=2 if window else 0)
    for _ in range(10):
        call(d, window=window, sinks=2 if window else 0)
        assert torch.equal(a, d["out"])


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (70, 5), (64, 200)])
def test_chunks_in_fp32(D, window, sinks):
    for Hq, Hkv, page in ((4, 2, 64), (5, 1, 16)):
        d = make([(100, 100), (1, 700), (16, 16), (0, 9), (17, 300), (64, 64), (65, 900)], Hq, Hkv,
                 D, page, "f32", seed=window, pad=2, fill=float("nan"))
        call(d, window=window, sinks=sinks)
        d["kc"], d["vc"] = torch.nan_to_num(d["kc"]), torch.nan_to_num(d["vc"])
        check(d, window=window, sinks=sinks)


def test_one_fp32_chunk_over_a_long_cache():
    d = make([(40, 6000)], 2, 1, 128, 128, "f32", seed=60)  # its keys in parts
    call(d)
    check(d)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_fp32_values_that_only_the_last_token_sees(bad):
    d = make([(70, 200)], 2, 1, 64, 32, "f32", seed=61)
    p = int(d["table_h"][0, 199 // 32])
    d["vc"][p, :, 199 % 32] = bad
    call(d)
    got = d["out"].clone()
    d["vc"][p, :, 199 % 32] = 0
    d["out"].copy_(torch.where(torch.isfinite(got), got, torch.zeros_like(got)))
    assert not torch.isfinite(got[69]).any() and torch.isfinite(got[:69]).all()
    r = ref.paged_attention(host(d["q"])[:69], host(d["kc"]), host(d["vc"]), d["table_h"],
                            np.array([0, 69], np.int32), np.array([199], np.int32), 32)
    lim = (2 * (64 + 8) * 2.0 ** -24 * r[3] + 264 * 2.0 ** -24)[..., None] * r[2]
    assert (np.abs(host(got[:69]) - r[0]) <= lim).all()


def test_more_fp32_chunks_than_blocks_search():
    rng = np.random.default_rng(8)
    q = rng.integers(0, 9, 1100)
    q[::7] += 4
    d = make([(int(x), int(x + k)) for x, k in zip(q, rng.integers(0, 90, 1100))], 8, 1, 32, 16,
             "f32", seed=62)
    assert d["T"] * 8 >= 32 * 1100
    call(d)
    check(d)


@pytest.mark.parametrize("D", [32, 64, 128])
def test_fp32_chunks_over_long_caches(D):
    """Tall tiles with their keys in parts, and values that only the last tokens see."""
    d = make([(40, 6000), (3, 2000)], 4, 2, D, 128, "f32", seed=63)
    call(d)
    check(d)
    for at in (5999, 5998):
        d["vc"][int(d["table_h"][0, at // 128]), :, at % 128] = float("inf")
    call(d)
    got = d["out"][:38].clone()
    assert torch.isfinite(got).all() and not torch.isfinite(d["out"][38:40]).any()
    for at in (5999, 5998):
        d["vc"][int(d["table_h"][0, at // 128]), :, at % 128] = 0
    r = ref.paged_attention(host(d["q"])[:38], host(d["kc"]), host(d["vc"]), d["table_h"],
                            np.array([0, 38], np.int32), np.array([5998], np.int32), 128)
    lim = (2 * (D + 8) * 2.0 ** -24 * r[3] + 6064 * 2.0 ** -24)[..., None] * r[2]
    assert (np.abs(host(got) - r[0]) <= lim).all()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 9, 16])
def test_few_rows_in_fp32(G):
    d = make([(1, 90), (1, 1), (2, 300), (0, 4)], 2 * G, 2, 64, 16, "f32", seed=G)
    call(d)
    check(d)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_two_calls_at_once(dt):
    """Calls with workspaces of their own on two streams give what they give alone."""
    ds = [make([(1, 700), (130, 900), (1, 64), (7, 2000)], 8, 2, 128, 64, dt, seed=70),
          make([(1, int(k)) for k in range(40, 1500, 23)], 8, 2, 64, 32, dt, seed=71)]
    want, ws = [], []
    for d in ds:
        call(d)
        want.append(d["out"].clone())
        n = kda.kda_paged_attention_fwd_workspace_size(
            d["N"], d["T"], 8, 2, d["D"], dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
        ws.append(torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(30):
        for d in ds:
            d["out"].fill_(5)
        torch.cuda.synchronize()
        for d, w, s in zip(ds, ws, streams):
            with torch.cuda.stream(s):
                call(d, ws=w)
        torch.cuda.synchronize()
        assert all(torch.equal(x, d["out"]) for x, d in zip(want, ds))
    assert kda.kda_device_error() == 0


def test_overlapping_sequences_longer_than_the_line():
    """Offsets against the rules, whose tiles in all pass 2^32: no access leaves the buffers (rows
    behind them keep what they held), nothing is reported, and the next call is right."""
    ensure_built()
    N, T, Hkv, D, page = 8192, 4096, 3500, 32, 128
    maxp = T // page
    cache = torch.zeros(1, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T + 1, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 1, Hkv), 7.0, device="cuda")
    table = torch.zeros(N, maxp, dtype=torch.int32, device="cuda")
    cu = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    kv = torch.full((N,), T, dtype=torch.int32, device="cuda")
    n = kda.kda_paged_attention_fwd_workspace_size(N, T, Hkv, Hkv, D)
    ws = torch.zeros(n + 1024, dtype=torch.uint8, device="cuda")
    kda.kda_paged_attention_fwd(q, cache, cache, table, cu, kv, out[:T], N, T, Hkv, Hkv, D, 1, page,
                                maxp, lse=lse[:T], workspace=(ws.data_ptr(), n))
    torch.cuda.synchronize()
    assert (out[T] == 7.0).all() and (lse[T] == 7.0).all() and (ws[n:] == 0).all()
    assert kda.kda_device_error() == 0
    d = make([(1, 70), (40, 140)], 4, 2, D, 32, "bf16", seed=80)
    call(d)
    check(d)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_one_workspace_for_all_batches(dt):
    """A buffer of the size for the largest batch, with bytes behind it that stay."""
    Hq, Hkv, D = 16, 8, 128
    n = kda.kda_paged_attention_fwd_workspace_size(
        16, 4096, Hq, Hkv, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for seqs in ([(1, 900)] * 16, [(1, 3000)], [(64, 64)], [(64, 700)], [(3, 40), (100, 300)],
                 [(7, 7 + 60 * i) for i in range(16)]):
        d = make(seqs, Hq, Hkv, D, 64, dt, seed=len(seqs))
        call(d, ws=(ws.data_ptr(), n))
        check(d)
        assert (ws[n:] == 0x5A).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 5), (1000, 140)])
def test_chunks_of_several_items_over_long_caches(D, window, sinks):
    """Chunks of 256-row items behind more keys than a stretch has, with and without a window."""
    for Hq, Hkv, page in ((2, 1, 64), (5, 1, 16), (2, 2, 128)):
        d = make([(300, 2100), (1, 900), (411, 1300), (140, 140)], Hq, Hkv, D, page, "bf16",
                 seed=D + Hq, pad=1)
        call(d, window=window, sinks=sinks)
        check(d, window=window, sinks=sinks)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("slope", [20.0, 150.0, 300.0, 600.0, -300.0])
@pytest.mark.parametrize("jump", [0, 48])
def test_rising_scores_of_chunks(D, slope, jump):
    """Scores that grow along the keys (per 1500 of them): the running maximum moves at every tile,
    in either half of it, by less or more than what is taken without scaling anew.  With `jump`
    they grow in steps at other places than the tiles' ends."""
    d = make([(200, 1500), (130, 130), (1, 1500)], 2, 1, D, 64, "bf16", seed=13)
    for n in range(3):
        for j in range(int(d["kv_h"][n])):
            at = (j + jump) // 64 * 64 if jump else j
            d["kc"][int(d["table_h"][n, j // 64]), :, j % 64] = slope * at / 1500 / D
    d["q"].copy_(torch.rand_like(d["q"]) + 0.5)
    call(d, softmax_scale=1.0)
    check(d, scale=1.0)


@pytest.mark.parametrize("dt,D", KINDS)
@pytest.mark.parametrize("over", [False, True])
def test_bad_pages_and_lengths_are_clamped(dt, D, over):
    """Entries outside the cache, lengths outside the table and a last offset behind the rows count
    as the nearest ones inside; no row behind the sequences or the buffers is touched."""
    d = make([(2, 100), (1, 40), (1, 64)], 2, 1, D, 16, dt, pad=2, seed=90)
    T, maxp = d["T"], d["table"].shape[1]
    big = torch.full((T + 8, 2, D), 7.0, dtype=DT[dt], device="cuda")
    ends = torch.full((T + 8, 2), 7.0, device="cuda")
    d["out"], d["lse"] = big[4:4 + T], ends[4:4 + T]
    d["table"][0, 1], d["table"][0, 2] = 2 ** 31 - 1, -2 ** 31
    d["kv"][1], d["kv"][2] = 2 ** 31 - 1, -5
    d["table_h"] = np.clip(d["table"].cpu().numpy().astype(np.int64), 0, d["kc"].shape[0] - 1)
    d["kv_h"] = np.array([100, 16 * maxp, 0])
    if over:
        d["cu"][3] = 2 ** 30
        d["cu_h"] = np.array([0, 2, 3, T], np.int32)
        d["live"] = T
    call(d)
    check(d)
    assert (d["out"][3:d["live"]] == 0).all() and torch.isneginf(d["lse"][3:d["live"]]).all()
    for x in (big, ends):
        assert (x[:4] == 7.0).all() and (x[4 + T:] == 7.0).all()
