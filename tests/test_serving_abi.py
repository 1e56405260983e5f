"""Host-only checks of the serving operators' C ABI: bad arguments are refused with the
documented codes before anything touches a device, and empty calls need no device memory."""
import pytest

import gated_delta_rule_55_gb300 as kda
from gated_delta_rule_55_gb300 import build_lib

FAKE = 0x10000  # a 256-byte-aligned non-NULL address; never dereferenced by these tests


@pytest.fixture(scope="module")
def L():
    build_lib.build()
    return kda.lib()


def _step(L, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, beta=FAKE, decay=None, state=FAKE, slots=FAKE, oslots=None,
             cu=None, out=FAKE, scale=0.0, N=2, T=1, Hk=2, Hv=4, dk=64, dv=128, ns=4, qs=128,
             ks=128, vs=512, flags=0, dtype=1)
    a.update(over)
    return L.kda_attention_step(*[a[n] for n in (
        "q", "k", "v", "beta", "decay", "state", "slots", "oslots", "cu", "out", "scale", "N",
        "T", "Hk", "Hv", "dk", "dv", "ns", "qs", "ks", "vs", "flags", "dtype")], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(state=None), -1), (dict(slots=None), -1), (dict(beta=None), -1),
    (dict(out=None), -1), (dict(N=-1), -2), (dict(T=-1), -2), (dict(Hk=0), -2),
    (dict(Hv=3), -2), (dict(ns=-1), -2), (dict(dk=96), -3), (dict(dv=256), -3),
    (dict(scale=float("nan")), -10), (dict(dtype=2), -7), (dict(flags=2), -13),
    (dict(flags=8), -13), (dict(slots=FAKE + 4), -6), (dict(state=FAKE + 8), -6),
    (dict(qs=120), -16), (dict(qs=132), -16), (dict(ks=64), -16), (dict(vs=511), -16),
    (dict(T=1 << 30), -11), (dict(ns=1 << 30), -11),
])
def test_step_refuses(L, over, code):
    assert _step(L, **over) == code


def _rope(L, kind="fwd", **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=None, cos=FAKE, sin=FAKE, pos=FAKE, slots=FAKE,
             qo=FAKE, ko=FAKE, kc=FAKE, vc=FAKE, dqo=FAKE, dko=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE,
             dwk=None, eps=1e-6, T=3, Hq=4, Hkv=2, D=64, R=64, mp=100, pages=4, page=16, qs=256,
             ks=128, vs=128, flags=0, dtype=1, ws=FAKE, wb=1 << 30)
    a.update(over)
    head = ["q", "k"] + (["v"] if kind == "append" else []) + ["wq", "wk", "cos", "sin", "pos"]
    sizes = ["eps", "T", "Hq", "Hkv", "D", "R", "mp"]
    if kind == "fwd":
        names = head + ["qo", "ko"] + sizes + ["qs", "ks", "flags", "dtype"]
        return L.kda_qk_norm_rope_fwd(*[a[n] for n in names], None)
    if kind == "append":
        names = (head + ["slots", "qo", "kc", "vc"] + sizes +
                 ["pages", "page", "qs", "ks", "vs", "flags", "dtype"])
        return L.kda_qk_norm_rope_append(*[a[n] for n in names], None)
    names = head + ["dqo", "dko", "dq", "dk", "dwq", "dwk"] + sizes + ["qs", "ks", "flags",
                                                                      "dtype", "ws", "wb"]
    return L.kda_qk_norm_rope_bwd(*[a[n] for n in names], None)


@pytest.mark.parametrize("kind", ["fwd", "append", "bwd"])
@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(cos=None), -1), (dict(pos=None), -1),
    (dict(T=-1), -2), (dict(Hq=0), -2), (dict(Hkv=0), -2), (dict(mp=0), -2), (dict(D=80), -3),
    (dict(R=24), -15), (dict(R=80), -15), (dict(R=-16), -15), (dict(eps=0.0), -10),
    (dict(eps=float("inf")), -10), (dict(flags=2), -13), (dict(dtype=3), -7),
    (dict(wq=FAKE + 4), -6), (dict(qs=248), -16), (dict(qs=257), -16), (dict(ks=132), -16),
    (dict(T=(1 << 31) - 1, qs=256), -11),
])
def test_norm_rope_refuses(L, kind, over, code):
    assert _rope(L, kind, **over) == code


@pytest.mark.parametrize("kind,over,code", [
    ("fwd", dict(qo=None), -1), ("fwd", dict(ko=None), -1), ("fwd", dict(ko=FAKE + 8), -6),
    ("append", dict(v=None), -1), ("append", dict(slots=None), -1), ("append", dict(kc=None), -1),
    ("append", dict(page=48), -14), ("append", dict(page=0), -14), ("append", dict(pages=-1), -2),
    ("append", dict(vs=120), -16), ("append", dict(vc=FAKE + 2), -6),
    ("append", dict(pages=1 << 30, page=128), -11),
    ("bwd", dict(dq=None), -1), ("bwd", dict(dko=None), -1), ("bwd", dict(ws=None), -12),
    ("bwd", dict(wb=16), -12), ("bwd", dict(ws=FAKE + 16), -12),
])
def test_norm_rope_variants_refuse(L, kind, over, code):
    assert _rope(L, kind, **over) == code


def _attn(L, **over):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, cu=FAKE, kv=FAKE, out=FAKE, lse=None,
             scale=0.0, N=2, T=5, Hq=8, Hkv=2, D=128, pages=10, page=64, maxp=4, window=0,
             sinks=0, qs=1024, dtype=1, ws=FAKE, wb=1 << 40)
    a.update(over)
    return L.kda_paged_attention_fwd(*[a[n] for n in (
        "q", "kc", "vc", "table", "cu", "kv", "out", "lse", "scale", "N", "T", "Hq", "Hkv", "D",
        "pages", "page", "maxp", "window", "sinks", "qs", "dtype", "ws", "wb")], None)


@pytest.mark.parametrize("over,code", [
    (dict(q=None), -1), (dict(kc=None), -1), (dict(table=None), -1), (dict(cu=None), -1),
    (dict(kv=None), -1), (dict(out=None), -1), (dict(N=-1), -2), (dict(T=-1), -2),
    (dict(Hq=0), -2), (dict(Hq=7), -2), (dict(pages=-1), -2), (dict(maxp=-1), -2),
    (dict(window=-1), -2), (dict(sinks=-1), -2), (dict(D=256), -3), (dict(page=24), -14),
    (dict(page=256), -14), (dict(scale=float("inf")), -10), (dict(dtype=9), -7),
    (dict(kv=FAKE + 4), -6), (dict(lse=FAKE + 4), -6), (dict(qs=1000), -16),
    (dict(qs=1028), -16), (dict(pages=1 << 26), -11), (dict(maxp=1 << 26), -11),
    (dict(N=65536), -11), (dict(N=60000, maxp=1 << 20), -11), (dict(ws=None), -12), (dict(ws=FAKE + 16), -12), (dict(wb=8), -12),
])
def test_paged_attention_refuses(L, over, code):
    assert _attn(L, **over) == code


def test_valid_calls_without_a_device_report_no_device(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this case is only meaningful without one")
    assert _step(L) == -9
    assert _attn(L) == -9
    for kind in ("fwd", "append", "bwd"):
        assert _rope(L, kind) == -9


def test_binding_refuses_tensors_of_another_kind():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="query"):
        kda.kda_paged_attention_fwd(x, x, x, x, x, x, x, 1, 2, 4, 4, 64, 1, 16, 1)
    with pytest.raises(ValueError, match="dtype"):
        kda.kda_attention_step(x.half(), x, x, x, x, x, x, x, 2, 1, 4, 4, 64, 64, 4)


@pytest.mark.parametrize("dtype", [kda.KDA_F32, kda.KDA_BF16])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 128), (32, 8, 128), (4, 4, 64), (10, 2, 32),
                                      (1, 1, 64)])
def test_paged_attention_workspace_of_the_largest_batch_serves_smaller_ones(L, dtype, Hq, Hkv, D):
    """The size never decreases in the number of sequences or of tokens, and no smaller call is
    refused with it, at any capacity of the block table."""
    import torch

    def size(N, T):
        return kda.kda_paged_attention_fwd_workspace_size(N, T, Hq, Hkv, D, dtype)

    Ns, Ts = [1, 2, 5, 16, 64, 300, 2000], [1, 2, 15, 16, 17, 64, 100, 256, 1024, 4096, 70000]
    for i, N in enumerate(Ns):
        for j, T in enumerate(Ts):
            for n in Ns[max(i - 1, 0):i + 1]:
                for t in Ts[max(j - 1, 0):j + 1]:
                    assert size(n, t) <= size(N, T), (n, t, N, T)
    if torch.cuda.is_available():
        return  # (the addresses below are never to reach a device)
    for N in Ns:
        for T in Ts:
            for maxp in (1, 4, 64, 4096):
                code = _attn(L, N=N, T=T, Hq=Hq, Hkv=Hkv, D=D, maxp=maxp, qs=Hq * D, dtype=dtype,
                             ws=FAKE, wb=size(Ns[-1], Ts[-1]))
                assert code == -9, (code, N, T, maxp)
                # and what the call's own size gives is enough for it
                assert _attn(L, N=N, T=T, Hq=Hq, Hkv=Hkv, D=D, maxp=maxp, qs=Hq * D, dtype=dtype,
                             ws=FAKE, wb=size(N, T)) == -9


def test_first_calls_from_two_threads(monkeypatch):
    """A call that begins while another one's first look-up is at any of its lines finds all of it
    (or looks up for itself)."""
    import sys
    import threading
    torch = pytest.importorskip("torch")
    from gated_delta_rule_55_gb300 import kda as binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 77, raising=False)
    for n in ("f32", "bf16", "i32", "i64", "device", "raw_stream", "where", "dense", "address"):
        monkeypatch.setattr(binding._Call, n, None)
    lines, got = [], []

    def other():
        try:
            got.append(binding._begin(FAKE, kda.KDA_F32, None))
        except Exception as e:  # noqa: BLE001
            got.append(e)

    names = [n for n in vars(binding._Call) if not n.startswith("_")]

    def trace(frame, event, arg):
        if frame.f_code is binding._setup.__code__ and event == "line":
            lines.append(frame.f_lineno)
            before = {n: getattr(binding._Call, n) for n in names}
            t = threading.Thread(target=other)
            t.start()
            t.join()
            for n in names:
                setattr(binding._Call, n, before[n])
        return trace

    old = sys.gettrace()
    sys.settrace(trace)
    try:
        binding._setup()
    finally:
        sys.settrace(old)
    assert len(lines) >= 4 and len(got) == len(lines)
    assert all(g == (kda.KDA_F32, torch.float32, 0, 77) for g in got), got


def test_binding_refuses_a_workspace_on_another_device(monkeypatch):
    torch = pytest.importorskip("torch")
    from gated_delta_rule_55_gb300 import kda as binding
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(binding._Call, "f32", None)  # look up anew, and again afterwards
    monkeypatch.setattr(binding._Call, "raw_stream", None)
    monkeypatch.setattr(binding._Call, "device", None)

    class Scratch:  # a tensor of the second device
        is_cuda = True
        is_contiguous = staticmethod(lambda: True)
        get_device = staticmethod(lambda: 1)
        data_ptr = staticmethod(lambda: FAKE)
        numel = staticmethod(lambda: 1 << 30)
        element_size = staticmethod(lambda: 1)

    with pytest.raises(ValueError, match="workspace"):
        kda.kda_paged_attention_fwd(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1, 0, 4, 4, 64, 1,
                                    16, 1, dtype=kda.KDA_BF16, workspace=Scratch())
    with pytest.raises(ValueError, match="workspace"):
        kda.kda_qk_norm_rope_bwd(FAKE, FAKE, None, None, None, None, None, FAKE, FAKE, FAKE, FAKE,
                                 None, None, 0, 4, 4, 64, 0, 0, dtype=kda.KDA_BF16,
                                 workspace=Scratch())
