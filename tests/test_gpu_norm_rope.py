"""kda_qk_norm_rope_fwd / _append / _bwd against the fp64 definition.

Tolerances.  A head's sum of squares has D terms in fp32 and halves its relative error in the
root; with the products and the rotation's two terms an output is off by at most
(D / 2 + 16) 2^-24 of the pair's two magnitudes (taken as the row's largest, twice).  A gradient
adds a second row sum: twice that, against the magnitudes of its two terms.  bf16 outputs add
half a step, 2^-8 of the value.  A weight's gradient sums T H terms in fp32 within blocks:
(terms per lane + 64) 2^-24 of the summed magnitudes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import serving_ref as ref  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def host(x):
    return x.detach().double().cpu().numpy()


def make(T, Hq, Hkv, D, R, dt, seed=0, maxpos=1000, weights=True):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    qkv = (rn(T, (Hq + 2 * Hkv) * D) * 2).to(DT[dt])
    d = dict(q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
             v=qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D))
    d["wq"] = 1 + 0.3 * rn(D) if weights else None
    d["wk"] = 1 + 0.3 * rn(D) if weights else None
    d["pos"] = torch.randint(0, maxpos, (T,), generator=g, device="cuda", dtype=torch.int32)
    ang = (torch.arange(maxpos, dtype=torch.float64, device="cuda")[:, None] *
           1e4 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / max(R, 1)))
    d["cos"], d["sin"] = ang.cos().float(), ang.sin().float()
    d["dyq"], d["dyk"] = rn(T, Hq, D).to(DT[dt]), rn(T, Hkv, D).to(DT[dt])
    d.update(T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, dt=dt, maxpos=maxpos)
    return d


def tables(d):
    p = np.clip(host(d["pos"]).astype(int), 0, d["maxpos"] - 1)
    return host(d["cos"])[p], host(d["sin"])[p]


def want_fwd(d, n, il):
    w = 1.0 if d["w" + n] is None else host(d["w" + n])
    return ref.norm_rope(host(d[n]), w, *tables(d), d["R"], EPS, il)


def check_rows(got, want, d, factor=1.0):
    top = 2 * np.abs(want).max(-1, keepdims=True)
    lim = factor * (d["D"] / 2 + 16) * 2.0 ** -24 * top
    if d["dt"] == "bf16":
        lim = lim + 2.0 ** -8 * np.abs(want)
    bad = np.abs(got - want) > lim
    assert not bad.any(), (np.abs(got - want)[bad].max(), int(bad.sum()))


def fwd(d, il, q=None, k=None):
    q = torch.empty(d["T"], d["Hq"], d["D"], dtype=DT[d["dt"]], device="cuda") if q is None else q
    k = torch.empty(d["T"], d["Hkv"], d["D"], dtype=DT[d["dt"]], device="cuda") if k is None else k
    kda.kda_qk_norm_rope_fwd(d["q"], d["k"], d["wq"], d["wk"], d["cos"] if d["R"] else None,
                             d["sin"] if d["R"] else None, d["pos"] if d["R"] else None, q, k,
                             d["T"], d["Hq"], d["Hkv"], d["D"], d["R"],
                             d["maxpos"] if d["R"] else 0, eps=EPS, interleaved=il)
    return q, k


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D,R", [(32, 32), (32, 16), (64, 64), (64, 48), (128, 128), (128, 64),
                                 (128, 80), (128, 16), (128, 0)])
def test_forward(dt, il, D, R):
    d = make(7, 5, 3, D, R, dt)
    q, k = fwd(d, il)
    check_rows(host(q), want_fwd(d, "q", il), d)
    check_rows(host(k), want_fwd(d, "k", il), d)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 32, 8), (513, 17, 1), (33, 9, 9)])
@pytest.mark.parametrize("weights", [True, False])
def test_sizes_and_no_weights(T, Hq, Hkv, weights):
    d = make(T, Hq, Hkv, 64, 32, "bf16", seed=T, weights=weights)
    q, k = fwd(d, False)
    check_rows(host(q), want_fwd(d, "q", False), d)
    check_rows(host(k), want_fwd(d, "k", False), d)


def test_in_place_and_positions_outside_the_table():
    d = make(50, 4, 2, 128, 128, "f32", seed=4, maxpos=64)
    d["q"], d["k"] = d["q"].contiguous(), d["k"].contiguous()
    d["pos"][:3] = torch.tensor([-5, 64, 2 ** 31 - 1], dtype=torch.int32)
    wq, wk = want_fwd(d, "q", False), want_fwd(d, "k", False)
    fwd(d, False, d["q"], d["k"])
    check_rows(host(d["q"]), wq, d)
    check_rows(host(d["k"]), wk, d)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_zero_rows_and_large_values(dt):
    d = make(4, 2, 1, 64, 64, dt)
    d["q"][0] = 0
    d["q"][1] *= 2.0 ** 40
    d["q"][2] *= 2.0 ** -30
    q, _ = fwd(d, False)
    check_rows(host(q), want_fwd(d, "q", False), d)


def append(d, il, kc, vc, slots, q):
    kda.kda_qk_norm_rope_append(d["q"], d["k"], d["v"], d["wq"], d["wk"], d["cos"], d["sin"],
                                d["pos"], slots, q, kc, vc, d["T"], d["Hq"], d["Hkv"], d["D"],
                                d["R"], d["maxpos"], kc.shape[0], kc.shape[2], eps=EPS,
                                interleaved=il)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("il", [False, True])
def test_append(dt, page, il):
    d = make(37, 6, 3, 64, 32, dt, seed=page)
    pages = 5
    kc = torch.randn(pages, 3, page, 64, device="cuda").to(DT[dt])
    vc = torch.randn(pages, 3, page, 64, device="cuda").to(DT[dt])
    slots = torch.randperm(pages * page, device="cuda")[:37].clone()
    slots[3], slots[4], slots[36] = -1, pages * page, -2 ** 40
    wk, kept = want_fwd(d, "k", il), [i for i in range(37) if i not in (3, 4, 36)]
    k0, v0 = host(kc), host(vc)
    q = torch.empty(37, 6, 64, dtype=DT[dt], device="cuda")
    append(d, il, kc, vc, slots, q)
    check_rows(host(q), want_fwd(d, "q", il), d)
    s = slots.tolist()
    gk, gv, v = host(kc), host(vc), host(d["v"])
    for i in kept:
        check_rows(gk[s[i] // page, :, s[i] % page], wk[i], d)
        assert (gv[s[i] // page, :, s[i] % page] == v[i]).all()
        k0[s[i] // page, :, s[i] % page] = gk[s[i] // page, :, s[i] % page]
        v0[s[i] // page, :, s[i] % page] = v[i]
    assert (gk == k0).all() and (gv == v0).all()  # nothing else moved


def bwd(d, il, dq=None, dk=None):
    dq = torch.empty_like(d["dyq"]) if dq is None else dq
    dk = torch.empty_like(d["dyk"]) if dk is None else dk
    dwq, dwk = torch.empty(d["D"], device="cuda"), torch.empty(d["D"], device="cuda")
    ws = torch.empty(kda.kda_qk_norm_rope_bwd_workspace_size(d["T"], d["Hq"], d["Hkv"], d["D"]),
                     dtype=torch.uint8, device="cuda")
    kda.kda_qk_norm_rope_bwd(d["q"], d["k"], d["wq"], d["wk"], d["cos"], d["sin"], d["pos"],
                             d["dyq"], d["dyk"], dq, dk, dwq, dwk, d["T"], d["Hq"], d["Hkv"],
                             d["D"], d["R"], d["maxpos"], eps=EPS, interleaved=il, workspace=ws)
    return dq, dk, dwq, dwk


def check_bwd(d, il, got):
    for n, gx, gw in (("q", got[0], got[2]), ("k", got[1], got[3])):
        w = np.ones(d["D"]) if d["w" + n] is None else host(d["w" + n])
        dx, dw, mag = ref.norm_rope_bwd(host(d[n]), w, *tables(d), d["R"], EPS, il,
                                        host(d["dy" + n]))
        x = host(d[n])
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
        gwt = np.abs(host(d["dy" + n])).max(-1, keepdims=True) * np.abs(w).max() * 2
        size = r * gwt * (1 + (np.abs(x) * r).max(-1, keepdims=True) ** 2)
        lim = 2 * (d["D"] / 2 + 16) * 2.0 ** -24 * size
        if d["dt"] == "bf16":
            lim = lim + 2.0 ** -8 * np.abs(dx)
        assert (np.abs(host(gx) - dx) <= lim).all(), np.abs(host(gx) - dx).max()
        terms = d["T"] * d[n].shape[1] / 64 + 64 + d["D"] / 2
        assert (np.abs(host(gw) - dw) <= terms * 2.0 ** -24 * mag * 2).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("D,R", [(32, 16), (64, 64), (128, 128), (128, 48), (128, 0)])
def test_backward(dt, il, D, R):
    d = make(29, 5, 2, D, R, dt, seed=D + R)
    check_bwd(d, il, bwd(d, il))


@pytest.mark.parametrize("T,Hq,Hkv,weights", [(1, 1, 1, True), (1, 8, 2, False),
                                              (700, 32, 8, True), (2049, 3, 1, True)])
def test_backward_sizes(T, Hq, Hkv, weights):
    d = make(T, Hq, Hkv, 128, 128, "bf16", seed=T, weights=weights)
    got = bwd(d, False)
    check_bwd(d, False, got)
    again = bwd(d, False)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # a fixed order of sums


def test_backward_in_place_of_the_output_gradients():
    d = make(40, 4, 4, 64, 64, "f32", seed=8)
    dq, dk = d["dyq"].clone(), d["dyk"].clone()
    a = bwd(d, False)
    d["dyq"], d["dyk"] = dq, dk
    b = bwd(d, False, dq, dk)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_backward_against_differences():
    """Central differences of the fp64 forward in random directions."""
    d = make(6, 3, 2, 32, 32, "f32", seed=21)
    dq, dk, dwq, dwk = (host(t) for t in bwd(d, True))
    rng = np.random.default_rng(0)
    cos, sin = tables(d)
    h = 1e-5
    for n, dx, dw in (("q", dq, dwq), ("k", dk, dwk)):
        x, w, dy = host(d[n]), host(d["w" + n]), host(d["dy" + n])
        for _ in range(4):
            ux, uw = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
            f = [(ref.norm_rope(x + e * h * ux, w + e * h * uw, cos, sin, d["R"], EPS, True)
                  * dy).sum() for e in (1, -1)]
            num = (f[0] - f[1]) / (2 * h)
            ana = (dx * ux).sum() + (dw * uw).sum()
            size = np.abs(dx * ux).sum() + np.abs(dw * uw).sum()
            # fp32 gradients (200 roundings) and the difference's h^2 term
            assert abs(num - ana) <= (200 * 2.0 ** -24 + 1e-8) * size


def test_no_tokens():
    d = make(0, 2, 1, 64, 64, "f32")
    fwd(d, False)
    _, _, dwq, dwk = bwd(d, False)
    torch.cuda.synchronize()
    assert (dwq == 0).all() and (dwk == 0).all()


def test_capture_and_replay():
    d = make(65, 4, 2, 64, 64, "bf16", seed=3)
    eager = bwd(d, False)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = bwd(d, False)
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, got))


# From 1216 tokens on a warp takes all heads of a kind, several groups of them in turn.
LONG = [("bf16", 128, 128, 17, 1, False), ("bf16", 128, 64, 33, 9, True),
        ("bf16", 32, 32, 65, 33, False),
        ("f32", 128, 128, 9, 5, False), ("f32", 128, 48, 17, 1, True),
        ("f32", 32, 16, 33, 17, True)]


@pytest.mark.parametrize("T", [1215, 1216, 1217, 2049])
@pytest.mark.parametrize("dt,D,R,Hq,Hkv,il", LONG)
def test_forward_of_many_tokens(dt, D, R, Hq, Hkv, il, T):
    d = make(T, Hq, Hkv, D, R, dt, seed=T + D)
    q, k = fwd(d, il)
    check_rows(host(q), want_fwd(d, "q", il), d)
    check_rows(host(k), want_fwd(d, "k", il), d)


@pytest.mark.parametrize("dt,D,R,Hq,Hkv,il", LONG)
def test_forward_of_many_tokens_in_place(dt, D, R, Hq, Hkv, il):
    for T in (1215, 1217):
        d = make(T, Hq, Hkv, D, R, dt, seed=T)
        d["q"], d["k"] = d["q"].contiguous(), d["k"].contiguous()
        wq, wk = want_fwd(d, "q", il), want_fwd(d, "k", il)
        fwd(d, il, d["q"], d["k"])
        check_rows(host(d["q"]), wq, d)
        check_rows(host(d["k"]), wk, d)


@pytest.mark.parametrize("T", [1215, 1216, 2049])
@pytest.mark.parametrize("dt,D,R,Hq,Hkv,il", LONG)
def test_append_of_many_tokens(dt, D, R, Hq, Hkv, il, T):
    """Some tokens without a place; what no token names keeps what it held."""
    page = 16 if il else 128
    d = make(T, Hq, Hkv, D, R, dt, seed=T + R)
    pages = T // page + 3
    kc = torch.randn(pages, Hkv, page, D, device="cuda").to(DT[dt])
    vc = torch.randn(pages, Hkv, page, D, device="cuda").to(DT[dt])
    slots = torch.randperm(pages * page, device="cuda")[:T].clone()
    slots[5::97] = -1
    slots[7::101] = pages * page + 3
    s = slots.cpu().numpy()
    kept = (s >= 0) & (s < pages * page)
    wk = want_fwd(d, "k", il)[kept]
    k0, v0 = (host(x).transpose(0, 2, 1, 3).reshape(-1, Hkv, D) for x in (kc, vc))
    q = torch.empty(T, Hq, D, dtype=DT[dt], device="cuda")
    append(d, il, kc, vc, slots, q)
    check_rows(host(q), want_fwd(d, "q", il), d)
    gk, gv = (host(x).transpose(0, 2, 1, 3).reshape(-1, Hkv, D) for x in (kc, vc))
    check_rows(gk[s[kept]], wk, d)
    v0[s[kept]] = host(d["v"])[kept]
    k0[s[kept]] = gk[s[kept]]
    assert (gv == v0).all() and (gk == k0).all()
