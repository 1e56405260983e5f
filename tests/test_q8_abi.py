"""Host-only checks of the calls on 8-bit pages and shared prefixes: bad arguments are refused with
the documented codes before anything touches a device."""
import pytest

import gated_delta_rule_55_gb300 as kda
import test_serving_abi as sa
from test_serving_abi import FAKE, L  # noqa: F401


def _append(L, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=None, cos=FAKE, sin=FAKE, pos=FAKE, slots=FAKE,
             qo=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, eps=1e-6, T=3, Hq=4, Hkv=2, D=64, R=64,
             mp=100, pages=4, page=16, qs=256, kst=128, vst=128, flags=0, dtype=1)
    a.update(over)
    return L.kda_qk_norm_rope_append_q8(*[a[n] for n in (
        "q", "k", "v", "wq", "wk", "cos", "sin", "pos", "slots", "qo", "kc", "vc", "ks", "vs",
        "eps", "T", "Hq", "Hkv", "D", "R", "mp", "pages", "page", "qs", "kst", "vst", "flags",
        "dtype")], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(v=None), -1), (dict(slots=None), -1), (dict(qo=None), -1),
    (dict(kc=None), -1), (dict(ks=None), -1), (dict(vs=None), -1), (dict(T=-1), -2),
    (dict(pages=-1), -2), (dict(mp=0), -2), (dict(D=96), -3), (dict(page=8), -14),
    (dict(R=20), -15), (dict(eps=0.0), -10), (dict(flags=4), -13), (dict(dtype=2), -7),
    (dict(ks=FAKE + 8), -6), (dict(vs=FAKE + 1), -6), (dict(vc=FAKE + 4), -6),
    (dict(qs=250), -16), (dict(vst=120), -16), (dict(pages=1 << 30, page=128), -11),
])
def test_append_refuses(L, over, code):  # noqa: F811
    assert _append(L, **over) == code


def _read(L, **over):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, slots=FAKE, ko=FAKE, vo=FAKE, T=3, Hkv=2, D=64,
             pages=4, page=16, dtype=1)
    a.update(over)
    return L.kda_paged_cache_read_q8(*[a[n] for n in (
        "kc", "vc", "ks", "vs", "slots", "ko", "vo", "T", "Hkv", "D", "pages", "page", "dtype")],
        None)


@pytest.mark.parametrize("over,code", [
    (dict(kc=None), -1), (dict(vs=None), -1), (dict(slots=None), -1), (dict(vo=None), -1),
    (dict(T=-1), -2), (dict(Hkv=0), -2), (dict(pages=-1), -2), (dict(D=48), -3),
    (dict(page=20), -14), (dict(dtype=5), -7), (dict(ks=FAKE + 4), -6), (dict(ko=FAKE + 8), -6),
    (dict(pages=1 << 30, page=128), -11), (dict(T=1 << 30, Hkv=64), -11),
])
def test_read_refuses(L, over, code):  # noqa: F811
    assert _read(L, **over) == code


def _attn(L, prefix=False, **over):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, pt=FAKE, pl=FAKE, cg=FAKE, table=FAKE,
             cu=FAKE, kv=FAKE, out=FAKE, lse=None, scale=0.0, groups=1, N=2, T=5, Hq=8, Hkv=2,
             D=128, pages=10, page=64, maxpp=3, maxp=4, window=0, sinks=0, qs=1024, dtype=1,
             ws=FAKE, wb=1 << 40)
    a.update(over)
    if prefix:
        return L.kda_paged_prefix_attention_fwd(*[a[n] for n in (
            "q", "kc", "vc", "ks", "vs", "pt", "pl", "cg", "table", "cu", "kv", "out", "lse",
            "scale", "groups", "N", "T", "Hq", "Hkv", "D", "pages", "page", "maxpp", "maxp", "qs",
            "dtype", "ws", "wb")], None)
    return L.kda_paged_attention_q8_fwd(*[a[n] for n in (
        "q", "kc", "vc", "ks", "vs", "table", "cu", "kv", "out", "lse", "scale", "N", "T", "Hq",
        "Hkv", "D", "pages", "page", "maxp", "window", "sinks", "qs", "dtype", "ws", "wb")], None)


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(ks=None), -1), (dict(vs=None), -1),
    (dict(table=None), -1), (dict(cu=None), -1), (dict(kv=None), -1), (dict(out=None), -1),
    (dict(N=-1), -2), (dict(T=-1), -2), (dict(Hq=7), -2), (dict(pages=-1), -2),
    (dict(maxp=-1), -2), (dict(D=256), -3), (dict(page=24), -14), (dict(scale=float("nan")), -10),
    (dict(dtype=9), -7), (dict(kv=FAKE + 4), -6), (dict(ks=FAKE + 8), -6), (dict(qs=1000), -16),
    (dict(pages=1 << 26), -11), (dict(maxp=1 << 26), -11), (dict(N=65536), -11),
    (dict(N=60000, maxp=1 << 20), -11), (dict(ws=None), -12), (dict(ws=FAKE + 16), -12),
    (dict(wb=8), -12),
])
def test_attention_refuses(L, prefix, over, code):  # noqa: F811
    assert _attn(L, prefix, **over) == code


@pytest.mark.parametrize("over,code", [
    (dict(pt=None), -1), (dict(pl=None), -1), (dict(cg=None), -1), (dict(groups=-1), -2),
    (dict(maxpp=-1), -2), (dict(pl=FAKE + 4), -6), (dict(cg=FAKE + 2), -6),
    (dict(groups=65536), -11), (dict(maxpp=1 << 26), -11), (dict(ks=None), -1),
    (dict(groups=60000, maxpp=1 << 20), -11),
    # a workspace that is enough without prefixes
    (dict(wb=kda.kda_paged_attention_fwd_workspace_size(2, 5, 8, 2, 128)), -12),
])
def test_prefix_refuses(L, over, code):  # noqa: F811
    assert _attn(L, True, **over) == code


def test_windows_refuse(L):  # noqa: F811
    assert _attn(L, window=-1) == -2
    assert _attn(L, sinks=-1) == -2


def test_valid_calls_without_a_device_report_no_device(L):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this case is only meaningful without one")
    for dtype in (0, 1):
        assert _append(L, dtype=dtype) == _read(L, dtype=dtype) == -9
        assert _attn(L, dtype=dtype) == _attn(L, True, dtype=dtype) == -9
        assert _attn(L, True, dtype=dtype, ks=None, vs=None) == -9
        assert _attn(L, True, dtype=dtype, groups=0, pt=None, pl=None, cg=None) == -9


@pytest.mark.parametrize("dtype", [kda.KDA_F32, kda.KDA_BF16])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (32, 8, 128), (4, 4, 64), (10, 2, 32)])
def test_prefix_workspace_of_the_largest_batch_serves_smaller_ones(L, dtype, Hq, Hkv, D):  # noqa: F811
    import torch

    def size(g, N, T):
        return kda.kda_paged_prefix_attention_fwd_workspace_size(g, N, T, Hq, Hkv, D, dtype)

    gs, Ns, Ts = [0, 1, 3, 50], [1, 2, 16, 64, 300], [1, 2, 15, 17, 64, 256, 1024, 70000]
    for i, N in enumerate(Ns):
        for j, T in enumerate(Ts):
            for k, g in enumerate(gs):
                for less in ((gs[max(k - 1, 0)], N, T), (g, Ns[max(i - 1, 0)], T),
                             (g, N, Ts[max(j - 1, 0)])):
                    assert size(*less) <= size(g, N, T)
    if torch.cuda.is_available():
        return  # (the addresses below are never to reach a device)
    for g in gs:
        for N in Ns:
            for T in Ts:
                for maxp in (1, 64, 4096):
                    for wb in (size(g, N, T), size(gs[-1], Ns[-1], Ts[-1])):
                        assert _attn(L, True, groups=g, N=N, T=T, Hq=Hq, Hkv=Hkv, D=D, maxp=maxp,
                                     maxpp=maxp, qs=Hq * D, dtype=dtype, wb=wb) == -9


@pytest.mark.parametrize("dtype", [kda.KDA_F32, kda.KDA_BF16])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (4, 4, 64)])
def test_q8_workspace_of_the_largest_batch_serves_smaller_ones(L, dtype, Hq, Hkv, D):  # noqa: F811
    import torch

    def size(N, T):
        return kda.kda_paged_attention_q8_fwd_workspace_size(N, T, Hq, Hkv, D, dtype)

    Ns, Ts = [1, 2, 16, 300], [1, 15, 17, 64, 1024, 70000]
    for i, N in enumerate(Ns):
        for j, T in enumerate(Ts):
            assert size(Ns[max(i - 1, 0)], T) <= size(N, T)
            assert size(N, Ts[max(j - 1, 0)]) <= size(N, T)
            if not torch.cuda.is_available():  # (the addresses are never to reach a device)
                for wb in (size(N, T), size(Ns[-1], Ts[-1])):
                    assert _attn(L, N=N, T=T, Hq=Hq, Hkv=Hkv, D=D, qs=Hq * D, dtype=dtype,
                                 wb=wb) == -9
    if dtype == kda.KDA_BF16 and D == 128:
        assert _attn(L, wb=kda.kda_paged_attention_fwd_workspace_size(2, 5, 8, 2, 128)) == -12


def test_binding_refuses_other_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="query"):
        kda.kda_paged_attention_q8_fwd(x, x, x, x, x, x, x, x, x, 1, 2, 4, 4, 64, 1, 16, 1)
    with pytest.raises(ValueError, match="dtype"):
        kda.kda_paged_cache_read_q8(x, x, x, x, x, x.half(), x, 2, 4, 64, 1, 16)
    assert sa.FAKE == FAKE


def test_lists_whose_positions_would_pass_31_bits(L):  # noqa: F811
    """A list of 2^31 - 1 keys has a tile that ends at 2^31, and a token behind a prefix of that
    many the position 2^31 - 2 + its number: both would wrap."""
    page = 16
    most = (2 ** 31 - 128) // page
    for dtype in (0, 1):
        assert _attn(L, page=page, maxp=most + 1, N=1, Hkv=1, dtype=dtype) == -11
        for over in (dict(maxp=most + 1), dict(maxpp=most + 1), dict(maxpp=most, T=200)):
            a = dict(page=page, N=1, Hkv=1, Hq=1, D=32, qs=32, dtype=dtype, ws=None)
            a.update(over)
            assert _attn(L, True, **a) == -11
            assert _attn(L, True, ks=None, vs=None, **a) == -11
    # at the limits the next check refuses (no workspace)
    a = dict(page=page, N=1, Hkv=1, Hq=1, D=32, qs=32, ws=None)
    assert _attn(L, maxp=most, **a) == -12
    assert _attn(L, True, maxp=most, maxpp=4, **a) == -12
    assert _attn(L, True, maxp=4, maxpp=most, T=127, **a) == -12
    # without prefixes, over pages of query's type: as before
    assert _attn(L, True, ks=None, vs=None, groups=0, maxp=most + 1, **a) == -12
