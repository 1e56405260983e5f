"""kda_paged_prefix_attention_fwd against the fp64 definition, over pages of bf16, fp32 and 8 bits.

Tolerances: those of kda_paged_attention_fwd (test_gpu_paged_attention.py) over all keys a token
sees, and for the joining of its two parts 2^-20 of A = sum p |v| (two factors e^{m_i - m} and the
quotient, each of fp32)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import q8_ref  # noqa: E402
import test_gpu_paged_attention as pa  # noqa: E402
import test_gpu_q8_cache as q8_cache  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

DT = pa.DT
host = pa.host
KINDS = [(dt, D, q8) for dt in ("f32", "bf16") for D in (32, 64, 128) for q8 in (False, True)]


def make(prefixes, seqs, Hq, Hkv, D, page, dt, q8, groups=None, seed=0, pad=0, fill=False, std=1.0):
    """prefixes: keys of each; seqs: (new tokens, own keys); groups: where each group begins (and
    ends).  fill: places behind the keys and pages of nobody hold NaNs."""
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    if groups is None:
        groups = np.linspace(0, len(seqs), len(prefixes) + 1).astype(int)
    cu = np.concatenate([[0], np.cumsum([q for q, _ in seqs])]).astype(np.int32)
    T, kv, pl = int(cu[-1]) + pad, np.array([k for _, k in seqs]), np.array(prefixes, int)
    needs = [[-(-int(k) // page) for k in ks] for ks in (pl, kv)]
    pages = sum(map(sum, needs)) + 3
    perm, at, tables = rng.permutation(pages), 0, []
    used = np.zeros((pages, page), bool)
    for need, lens in zip(needs, (pl, kv)):
        t = np.full((len(need), max(need + [1]) + 1), -7 if fill else 0, np.int32)
        for n, m in enumerate(need):
            t[n, :m] = perm[at:at + m]
            at += m
            for i in range(m):
                used[t[n, i], :min(page, int(lens[n]) - i * page)] = True
        tables.append(t)
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    d = dict(q8=q8, dt=dt, D=D, Hq=Hq, Hkv=Hkv, page=page, pages=pages, T=T, live=int(cu[-1]),
             N=len(seqs), G=len(prefixes), cu_h=cu, kv_h=kv, pl_h=pl, groups_h=np.array(groups),
             pt_h=tables[0], table_h=tables[1], pt=i32(tables[0]), table=i32(tables[1]),
             pl=i32(pl), cg=i32(groups), cu=i32(cu), kv=i32(kv), ks=None, vs=None)
    for n in "kv":
        x = torch.randn(pages, Hkv, page, D, generator=g, device="cuda") * (std if n == "k" else 1)
        odd = ~used[:, None] & np.ones((1, Hkv, 1), bool)
        if q8:
            b, s = q8_ref.quantise(host(x) * np.exp(rng.standard_normal(x.shape[:3]))[..., None])
            d[n + "x"] = q8_ref.value(b, s)
            if fill:
                s[odd] = 255
            d[n + "c"] = torch.from_numpy(b).cuda().view(torch.float8_e4m3fn)
            d[n + "s"] = torch.from_numpy(s).cuda()
        else:
            x = x.to(DT[dt])
            d[n + "x"] = host(x)
            if fill:
                x[torch.from_numpy(odd).cuda()] = float("nan")
            d[n + "c"] = x
    d["q"] = torch.randn(T, Hq + 1, D, generator=g, device="cuda").to(DT[dt])[:, :Hq]
    d["out"] = torch.full((T, Hq, D), 7.0, dtype=DT[dt], device="cuda")
    d["lse"] = torch.full((T, Hq), 7.0, device="cuda")
    return d


def size(d):
    return kda.kda_paged_prefix_attention_fwd_workspace_size(
        d["G"], d["N"], d["T"], d["Hq"], d["Hkv"], d["D"],
        dtype=kda.KDA_F32 if d["dt"] == "f32" else kda.KDA_BF16)


def call(d, ws=None, **kw):
    if ws is None:
        ws = torch.empty(max(size(d), 1), dtype=torch.uint8, device="cuda").fill_(0xFF)
    kda.kda_paged_prefix_attention_fwd(
        d["q"], d["kc"], d["vc"], d["pt"], d["pl"], d["cg"], d["table"], d["cu"], d["kv"],
        d["out"], d["G"], d["N"], d["T"], d["Hq"], d["Hkv"], d["D"], d["pages"], d["page"],
        d["pt"].shape[1], d["table"].shape[1], k_scale=d["ks"], v_scale=d["vs"], lse=d["lse"],
        workspace=ws, **kw)


def check(d, **kw):
    n = d["live"]
    out, lse, A, Z = q8_ref.prefix_attention(
        host(d["q"])[:n], d["kx"], d["vx"], d["pt_h"], d["pl_h"], d["groups_h"], d["table_h"],
        d["cu_h"], d["kv_h"], d["page"], **kw)
    keys = int(max(d["kv_h"], default=0)) + int(max(d["pl_h"], default=0))
    dl = (d["D"] + 8) * 2.0 ** -24 * Z
    lim = (2 * dl + (keys + 64) * 2.0 ** -24 + 2.0 ** -20)[..., None] * A
    if d["dt"] == "bf16":
        lim = lim + 2.0 ** -8 * (A + np.abs(out))
    got = host(d["out"])[:n]
    bad = ~(np.abs(got - out) <= lim)
    assert not bad.any(), (np.abs(got - out)[bad].max(), int(bad.sum()), np.argwhere(bad)[:5])
    gl = host(d["lse"])[:n]
    empty = np.isneginf(lse)
    assert (np.isneginf(gl) == empty).all()
    ok = ~empty
    assert (np.abs(gl[ok] - lse[ok]) <=
            dl[ok] + 2.0 ** -22 * (np.abs(lse[ok]) + 3 + keys / 16)).all()
    assert (host(d["out"])[n:] == 7.0).all() and (host(d["lse"])[n:] == 7.0).all()
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("dt,D,q8", KINDS)
@pytest.mark.parametrize("page", [16, 128])
def test_groups(dt, D, q8, page):
    """Groups of one to four sequences, one of them without a prefix, one without tokens."""
    d = make([200, 0, 33, 129], [(1, 1), (3, 70), (1, 40), (5, 5), (0, 9), (20, 20), (2, 300), (1, 1),
                                 (0, 0)], 4, 2, D, page, dt, q8, groups=[0, 2, 3, 7, 9], pad=3)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D,q8", KINDS)
def test_sequences_outside_the_groups(dt, D, q8):
    d = make([150, 40], [(1, 3), (2, 2), (1, 90), (4, 10), (1, 1), (3, 50)], 4, 1, D, 32, dt, q8,
             groups=[1, 3, 4], seed=2, pad=1)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D,q8", KINDS)
@pytest.mark.parametrize("P", [1, 16, 127, 128, 129, 255, 256, 257, 1000])
def test_prefix_lengths(dt, D, q8, P):
    d = make([P], [(1, 1), (1, 130), (2, 17)], 2, 1, D, 16, dt, q8, seed=P)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D,q8", KINDS)
@pytest.mark.parametrize("fill", [False, True])
def test_what_lies_outside_the_keys_never_counts(dt, D, q8, fill):
    for page in (16, 64):
        d = make([130, 67, 201], [(1, 70), (3, 3), (70, 90), (1, 1)], 4, 2, D, page, dt, q8,
                 fill=fill, seed=5)
        call(d)
        check(d)


@pytest.mark.parametrize("dt,D,q8", KINDS)
def test_more_tokens_than_keys_and_nothing_to_see(dt, D, q8):
    d = make([50, 0], [(10, 4), (3, 0), (4, 2), (2, 0)], 2, 2, D, 16, dt, q8, seed=6)
    call(d)
    check(d)
    assert (host(d["out"])[13:15] == 0).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("q,G,Hkv", [(1, 1, 1), (127, 1, 2), (129, 1, 1), (64, 4, 1), (65, 4, 2),
                                     (31, 8, 1), (100, 5, 1), (300, 2, 1)])
def test_chunks(D, q8, q, G, Hkv):
    """Rows of the prefix's items that fill a tile, or two, or end inside one."""
    d = make([700], [(q, q), (q, q + 90), (1, 1)], G * Hkv, Hkv, D, 64, "bf16", q8, seed=q)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("q8", [False, True])
def test_long_prefix_of_many(dt, D, q8):
    """Prefixes that are cut among many blocks, behind them short sequences."""
    rng = np.random.default_rng(3)
    d = make([6000, 3000], [(1, int(k)) for k in rng.integers(1, 200, 70)], 8, 2, D, 64, dt, q8,
             seed=7)
    call(d)
    check(d)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("bf16", 128), ("f32", 32)])
@pytest.mark.parametrize("q8", [False, True])
def test_more_lists_than_threads(dt, D, q8):
    rng = np.random.default_rng(9)
    for N, G in ((700, 300), (1300, 2), (40, 1)):
        d = make([int(x) for x in rng.integers(0, 60, G)],
                 [(int(q), int(q + k)) for q, k in zip(rng.integers(0, 4, N),
                                                       rng.integers(0, 40, N))],
                 2, 1, D, 16, dt, q8, seed=N)
        call(d)
        check(d)


def test_without_groups_it_is_attention_over_pages():
    for dt, D in (("bf16", 128), ("f32", 64)):
        d = pa.make([(1, 300), (40, 140)], 4, 2, D, 32, dt, seed=3)
        pa.call(d)
        a = d["out"].clone()
        ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
        kda.kda_paged_prefix_attention_fwd(
            d["q"], d["kc"], d["vc"], None, None, None, d["table"], d["cu"], d["kv"], d["out"], 0,
            2, d["T"], 4, 2, D, d["kc"].shape[0], 32, 0, d["table"].shape[1], workspace=ws)
        assert torch.equal(a, d["out"])


@pytest.mark.parametrize("dt,D,q8", [("bf16", 128, False), ("bf16", 64, True), ("f32", 64, False)])
def test_scores_of_all_sizes(dt, D, q8):
    """Large scores: one key takes all, of the prefix or of the sequence's own."""
    d = make([500], [(3, 200), (40, 100), (1, 1)], 4, 4, D, 64, dt, q8, std=30.0, seed=12)
    call(d, softmax_scale=0.7)
    check(d, scale=0.7)


@pytest.mark.parametrize("dt,D,q8", [("bf16", 128, False), ("bf16", 128, True), ("bf16", 64, False),
                                     ("f32", 64, True)])
def test_repeat_stream_and_replay_give_the_same_bits(dt, D, q8):
    d = make([3000, 500], [(1, 300), (90, 200), (1, 20), (5, 100)], 8, 2, D, 32, dt, q8, seed=15)
    call(d)
    check(d)
    a, l = d["out"].clone(), d["lse"].clone()
    s = torch.cuda.Stream()
    d["out"].fill_(1)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call(d)
    s.synchronize()
    assert torch.equal(a, d["out"]) and torch.equal(l, d["lse"])
    ws = torch.empty(size(d), dtype=torch.uint8, device="cuda")
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(d, ws=ws)
    ws.fill_(0xFF)
    for _ in range(2):
        d["out"].fill_(1)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, d["out"]) and torch.equal(l, d["lse"])
    # new lengths and groups under the same graph
    d["kv"].sub_(torch.tensor([100, 0, 5, 0], dtype=torch.int32, device="cuda"))
    d["pl"].copy_(torch.tensor([1100, 499], dtype=torch.int32))
    d["cg"].copy_(torch.tensor([0, 1, 4], dtype=torch.int32))
    d["kv_h"], d["pl_h"], d["groups_h"] = (host(d[n]).astype(int) for n in ("kv", "pl", "cg"))
    gr.replay()
    torch.cuda.synchronize()
    check(d)


@pytest.mark.parametrize("q8", [False, True])
def test_two_calls_at_once(q8):
    ds = [make([900, 100], [(1, 70), (130, 200), (1, 64), (7, 90)], 8, 2, 128, 64, "bf16", q8, seed=70),
          make([2000], [(1, int(k)) for k in range(4, 500, 23)], 8, 2, 64, 32, "bf16", q8, seed=71)]
    want, ws = [], []
    for d in ds:
        call(d)
        want.append(d["out"].clone())
        ws.append(torch.empty(size(d), dtype=torch.uint8, device="cuda"))
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


@pytest.mark.parametrize("dt,D,q8", KINDS)
def test_bad_numbers_stay_inside(dt, D, q8):
    """Pages, lengths and offsets outside are clamped; offsets against the rules give wrong numbers
    in the sequences' rows and touch no other."""
    d = make([100, 60], [(2, 100), (1, 40), (1, 64)], 2, 1, D, 16, dt, q8, pad=2, seed=90)
    d["pt"][0, 1], d["pt"][0, 2] = 2 ** 31 - 1, -2 ** 31
    d["pl"][1] = 2 ** 31 - 1
    d["cg"][2] = 2 ** 30
    d["kv"][2] = -5
    d["pt_h"] = np.clip(d["pt"].cpu().numpy().astype(np.int64), 0, d["pages"] - 1)
    d["pl_h"] = np.array([100, 16 * d["pt"].shape[1]])
    d["kv_h"] = np.array([100, 40, 0])
    d["groups_h"] = np.array([0, d["groups_h"][1], 3])
    call(d)
    check(d)
    n = size(d)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for cg in ([2, 1, 3], [3, 0, 0], [-4, 2, 1], [0, 3, 2]):
        d["cg"].copy_(torch.tensor(cg, dtype=torch.int32))
        d["out"].fill_(7)
        call(d, ws=(ws.data_ptr(), n))
        torch.cuda.synchronize()
        assert (host(d["out"])[d["live"]:] == 7).all() and (ws[n:] == 0x5A).all()
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("dt,q8", [("f32", False), ("f32", True), ("bf16", False), ("bf16", True)])
def test_one_workspace_for_all_batches(dt, q8):
    Hq, Hkv, D = 16, 8, 128
    n = kda.kda_paged_prefix_attention_fwd_workspace_size(
        3, 16, 1024, Hq, Hkv, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for P, seqs in (([300], [(1, 90)] * 16), ([2000], [(1, 300)]), ([64, 64], [(64, 64)] * 2),
                    ([10, 0, 500], [(3, 40), (100, 300), (2, 2)]), ([900], [(200, 200)])):
        d = make(P, seqs, Hq, Hkv, D, 64, dt, q8, seed=len(seqs))
        call(d, ws=(ws.data_ptr(), n))
        check(d)
        assert (ws[n:] == 0x5A).all()


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("G,Hkv", [(4, 1), (8, 2)])
def test_groups_that_fill_tiles_alone(D, q8, G, Hkv):
    """Long sequences, which take their prefix along, beside groups of short ones, which share it:
    groups on both sides of the border, with a short sequence among long ones, without a prefix,
    without tokens, and sequences outside all groups."""
    n = 1000 // G  # tokens of a long sequence
    for page in (16, 64):
        d = make([300, 129, 0, 500, 77, 40],
                 [(3, 3), (n, n), (n + 17, 2 * n), (1, 90), (n, n - 40), (1, 1), (2 * n, 2 * n),
                  (2, 2), (4, 70), (0, 5), (n, n + 1), (1, 7)], G * Hkv, Hkv, D, page, "bf16", q8,
                 groups=[1, 3, 6, 7, 9, 10, 11], seed=n + D, pad=2, fill=True)
        call(d)
        check(d)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("P", [1, 127, 128, 129, 1500])
def test_a_prefix_taken_along(q8, P):
    """Prefix lengths around a tile in front of a long sequence's own keys, cut among many blocks."""
    d = make([P], [(300, 300), (257, 900)], 8, 2, 128, 64, "bf16", q8, seed=P)
    call(d)
    check(d)
    a = d["out"].clone()
    for _ in range(3):
        call(d)
        assert torch.equal(a, d["out"])


def test_bad_groups_of_long_sequences_stay_inside():
    d = make([100, 60, 30], [(200, 300), (190, 200), (210, 210)], 8, 2, 64, 16, "bf16", False, pad=2)
    n = size(d)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    for cg in ([2, 1, 3, 0], [3, 0, 0, 2], [-4, 2, 1, 9], [0, 3, 2, 3], [1, 1, 1, 1]):
        d["cg"].copy_(torch.tensor(cg, dtype=torch.int32))
        d["out"].fill_(7)
        call(d, ws=(ws.data_ptr(), n))
        torch.cuda.synchronize()
        assert (host(d["out"])[d["live"]:] == 7).all() and (ws[n:] == 0x5A).all()
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("D,q8", [(64, False), (128, True)])
def test_a_call_without_tokens_has_ended_before_what_follows(D, q8):
    """No row is in a sequence, so nothing is joined: the workspace is the caller's again behind the
    call in the stream, and the next call's with it."""
    d = make([100], [(2, 100), (1, 40)], 2, 1, D, 16, "bf16", q8, pad=2)
    call(d)
    want, cu = d["out"].clone(), d["cu"].clone()
    ws = torch.empty(size(d), dtype=torch.uint8, device="cuda")
    for _ in range(100):
        d["cu"].zero_()
        d["out"].fill_(7)
        call(d, ws=ws)
        ws.fill_(0x5A)
        d["cu"].copy_(cu)
        torch.cuda.synchronize()
        assert (ws == 0x5A).all() and (d["out"] == 7).all()
        call(d, ws=ws)
        assert torch.equal(d["out"], want)
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("k,q", q8_cache.EXTREMES)
@pytest.mark.parametrize("tokens", [2, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_of_all_magnitudes(D, tokens, k, q):
    """test_gpu_q8_cache.py's, behind prefixes that are shared (2 tokens) or taken along (200)."""
    d = make([500, 90], [(tokens, 300), (tokens, tokens), (tokens, 300)], 4, 1, D, 64, "bf16", True,
             groups=[0, 2, 3], seed=22)
    b, s, sign = q8_cache.keys_of_one_magnitude(d["kc"].shape, k, 6)
    k = float(q8_ref.value(b, s).max())
    d["kc"] = torch.from_numpy(b).cuda().view(torch.float8_e4m3fn)
    d["ks"] = torch.from_numpy(s).cuda()
    d["q"].fill_(q)
    call(d)
    out, lse = host(d["out"]), host(d["lse"])
    for n, (g, p) in enumerate([(0, 500), (0, 500), (1, 90)]):
        kv, t0 = int(d["kv_h"][n]), int(d["cu_h"][n])
        sg, v = (np.concatenate([q8_ref.rows_of(x, d["pt_h"][g], p, 64)[:, 0],
                                 q8_ref.rows_of(x, d["table_h"][n], kv, 64)[:, 0]])
                 for x in (sign, d["vx"]))
        for i in range(tokens):
            m = p + kv - tokens + i + 1
            for h in range(4):
                q8_cache.check_one_magnitude(out[t0 + i, h], lse[t0 + i, h], k, q, sg[:m], v[:m], D)
    assert kda.kda_device_error() == 0


@pytest.mark.parametrize("q8,top,large", [(True, top, 2.0 ** 84) for top in q8_cache.RISES] +
                         [(False, top, 2.0 ** 108) for top in (7.0, 9.0, 30.0, 44.0, 52.0, 72.0)])
@pytest.mark.parametrize("at", [40, 700])
@pytest.mark.parametrize("D", [32, 64, 128])
def test_large_values_under_rising_scores(D, q8, large, at, top):
    """test_gpu_q8_cache.py's, behind prefixes, shared and taken along: a growth of what the call
    absorbs over values that leave room for it and the keys (less than 2^11)."""
    i32 = q8_cache.i32
    for tokens, Hkv in ((2, 80), (200, 24)):
        r = q8_cache.Rise([1200, 300, 500, 800, 600], Hkv, D, top, at, large, q8)
        q, cu, out, lse = r.queries([tokens] * 3, 4)
        a = (2, 3, len(q), 4 * Hkv, Hkv, D)
        ws = torch.empty(kda.kda_paged_prefix_attention_fwd_workspace_size(*a), dtype=torch.uint8,
                         device="cuda")
        w = r.table.shape[1]
        kda.kda_paged_prefix_attention_fwd(
            q, r.kc, r.vc, i32(r.table[:2]), i32(r.lists[:2]), i32([0, 2, 3]), i32(r.table[2:]),
            i32(cu), i32(r.lists[2:]), out, *a, r.pages, 64, w, w, k_scale=r.ks, v_scale=r.vs,
            lse=lse, softmax_scale=q8_cache.LN2, workspace=ws)
        for n, g in enumerate([0, 0, 1]):
            rows = [np.concatenate(x) for x in zip(r.of(g), r.of(2 + n))]
            q8_cache.check_rise(out[cu[n]:cu[n + 1]], lse[cu[n]:cu[n + 1]], *rows, D)
    assert kda.kda_device_error() == 0
