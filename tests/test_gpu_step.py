"""kda_attention_step against the fp64 definition and the oracle of the whole-sequence call.

Tolerances.  Sums over dk run in fp32: dk + 16 roundings of 2^-24 per token, relative to the
largest state, value or output, doubled for the two chained reductions, and every token's error
enters the next one's state.  bf16 outputs add half a step, 2^-8 of the value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import serving_ref as ref  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(x):
    return None if x is None else x.detach().double().cpu().numpy()


def make(lens, Hk, Hv, dk, dv, dt, seed=0, extra=3, pad=0, strided=True):
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = int(cu[-1]) + pad
    N = len(lens)

    def rn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    qkv = rn(rows, 2 * Hk * dk + Hv * dv).to(DT[dt])
    q = qkv[:, :Hk * dk].view(rows, Hk, dk)
    k = qkv[:, Hk * dk:2 * Hk * dk].view(rows, Hk, dk)
    v = qkv[:, 2 * Hk * dk:].view(rows, Hv, dv)
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    slots = N + extra
    d = dict(q=q, k=k, v=v, beta=torch.sigmoid(rn(rows, Hv)),
             decay=-torch.nn.functional.softplus(rn(rows, Hv) - 2),
             pool=rn(slots, Hv, dk, dv) * 0.1,
             slots=torch.randperm(slots, generator=g, device="cuda")[:N].int(),
             cu=torch.from_numpy(cu).cuda(), out=torch.full((rows, Hv, dv), 7.0, device="cuda",
                                                            dtype=DT[dt]))
    d.update(N=N, rows=rows, Hk=Hk, Hv=Hv, dk=dk, dv=dv, ns=slots, cu_h=cu, dt=dt,
             tok=max([1, *lens]))
    return d


def call(d, **kw):
    kda.kda_attention_step(d["q"], d["k"], d["v"], d["beta"], d["decay"], d["pool"], d["slots"],
                           d["out"], d["N"], kw.pop("T", d["rows"]), d["Hk"], d["Hv"], d["dk"],
                           d["dv"], d["ns"], cu_seqlens=kw.pop("cu", d["cu"]), **kw)


def want(d, out_slots=None, **kw):
    return ref.step(host(d["q"]), host(d["k"]), host(d["v"]), host(d["beta"]), host(d["decay"]),
                    host(d["pool"]), d["slots"].tolist(), d["cu_h"], out=host(d["out"]),
                    out_slots=None if out_slots is None else out_slots.tolist(), **kw)


def check(d, w):
    top = max(1.0, float(np.abs(w[1]).max()), float(host(d["v"]).__abs__().max(initial=0)))
    tol = 2 * (d["dk"] + 16) * d["tok"] * 2.0 ** -24 * top
    o = host(d["out"])
    lim = tol + (2.0 ** -8 * np.abs(w[0]) if d["dt"] == "bf16" else 0)
    assert (np.abs(o - w[0]) <= lim).all(), np.abs(o - w[0]).max()
    assert (np.abs(host(d["pool"]) - w[1]) <= tol).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 128), (64, 64), (64, 128), (128, 32),
                                   (128, 64), (128, 128)])
def test_shapes(dt, dk, dv):
    d = make([1, 3, 0, 2, 1], 2, 6, dk, dv, dt, pad=2)
    w = want(d)
    call(d)
    check(d, w)
    assert (host(d["out"])[d["cu_h"][-1]:] == 7.0).all()


@pytest.mark.parametrize("l2norm", [True, False])
@pytest.mark.parametrize("literal", [True, False])
@pytest.mark.parametrize("decay", [True, False])
def test_variants(l2norm, literal, decay):
    d = make([2, 1, 5], 3, 3, 64, 32, "f32", seed=1)
    if not decay:
        d["decay"] = None
    if not l2norm:  # keep the update a contraction, as a caller's own norm would
        d["k"] = d["k"] * 0.1
    w = want(d, l2norm=l2norm, literal=literal, scale=0.37)
    call(d, use_qk_l2norm=l2norm, order="literal" if literal else "decay_first",
         softmax_scale=0.37)
    check(d, w)


def test_fixed_token_count_and_dense_rows():
    d = make([3] * 7, 1, 2, 128, 64, "bf16", strided=False)
    w = want(d)
    call(d, T=3, cu=None)
    check(d, w)


def test_out_slots_and_missing_requests():
    """Read one slot, write another or nowhere; requests without a slot leave their rows."""
    d = make([1, 2, 4, 0, 1, 3], 2, 4, 64, 64, "f32", extra=8, seed=3)
    free = [s for s in range(d["ns"]) if s not in d["slots"].tolist()]
    o = torch.tensor([free[0], -1, d["ns"], free[1], int(d["slots"][4]), free[2]],
                     dtype=torch.int32, device="cuda")
    d["slots"][2] = -1
    d["slots"][5] = d["ns"] + 4
    w = want(d, out_slots=o)
    call(d, out_slots=o)
    check(d, w)
    assert (host(d["out"])[3:7] == 7.0).all()


@pytest.mark.parametrize("N,Hk,Hv", [(1, 1, 1), (1, 16, 32), (130, 4, 8)])
def test_batches_and_repeat(N, Hk, Hv):
    d = make([1] * N, Hk, Hv, 128, 128, "bf16", seed=5)
    for i in range(3):
        w = want(d)
        call(d)
        check(d, w)


def test_steps_follow_the_whole_sequence_call():
    """Prefill by kda_attention_fwd, then tokens one by one: the oracle's whole sequence."""
    from oracle import kda_attention
    ensure_built()
    B, T, P, H, D = 2, 21, 16, 3, 64
    g = torch.Generator(device="cuda").manual_seed(11)
    q, k, v = (torch.randn(B, T, H, D, generator=g, device="cuda") for _ in range(3))
    beta = torch.rand(B, T, H, generator=g, device="cuda")
    decay = -0.2 * torch.rand(B, T, H, generator=g, device="cuda")
    ro, rs = kda_attention(host(q), host(k), host(v), host(beta), host(decay))
    pool = torch.zeros(B, H, D, D, device="cuda")
    out = torch.empty(B, P, H, D, device="cuda")
    c = lambda x: x.contiguous()  # noqa: E731
    kda.kda_attention_fwd(c(q[:, :P]), c(k[:, :P]), c(v[:, :P]), c(beta[:, :P]),
                          c(decay[:, :P]), None, out, pool, B, P, H, D, D)
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    o1 = torch.empty(B, H, D, device="cuda")
    for t in range(P, T):
        kda.kda_attention_step(q[:, t], k[:, t], v[:, t], c(beta[:, t]), c(decay[:, t]), pool,
                               slots, o1, B, 1, H, H, D, D, B)
        assert np.abs(host(o1) - ro[:, t]).max() <= 1e-4  # the fp32 bound of the prefill call
    assert np.abs(host(pool) - rs).max() <= 1e-4


def test_capture_replay_and_other_stream():
    d = make([1, 2, 1], 2, 2, 64, 64, "bf16", seed=9)
    start = d["pool"].clone()
    call(d)
    o, p = d["out"].clone(), d["pool"].clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(d)  # warm on the side stream
    s.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(d)
    d["pool"].copy_(start)
    d["out"].fill_(0)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(d["out"], o) and torch.equal(d["pool"], p)


def test_pool_beyond_32_bit_offsets():
    """A pool of more than 2^32 elements: the far slots are the ones used."""
    ensure_built()
    Hv, D = 64, 128
    ns = (1 << 32) // (Hv * D * D) + 6
    d = make([1, 2], 32, Hv, D, D, "f32", seed=2)
    small = d["pool"]
    pool = torch.empty(ns, Hv, D, D, device="cuda")
    far = torch.tensor([ns - 1, ns - 3], dtype=torch.int32, device="cuda")
    pool[far.long()] = small[d["slots"].long()]
    w = want(d)
    near = d["slots"].long()
    d.update(pool=pool, slots=far, ns=ns)
    call(d)
    got = pool[far.long()]
    d["pool"] = small
    d["pool"][near] = got
    check(d, w)


def test_empty_calls():
    d = make([1], 1, 1, 32, 32, "f32")
    kda.kda_attention_step(d["q"], d["k"], d["v"], d["beta"], d["decay"], d["pool"], d["slots"],
                           d["out"], 0, 0, 1, 1, 32, 32, d["ns"])
    before = d["pool"].clone()
    kda.kda_attention_step(d["q"][:0], d["k"][:0], d["v"][:0], d["beta"][:0], None, d["pool"],
                           d["slots"], d["out"][:0], 1, 0, 1, 1, 32, 32, d["ns"])
    torch.cuda.synchronize()
    assert torch.equal(before, d["pool"])
