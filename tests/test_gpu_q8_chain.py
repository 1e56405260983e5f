"""The calls on 8-bit pages as a server uses them: a system prompt appended once, questions and then
single tokens of several users behind it, attention over the shared and the own pages, and tokens
read back; against the fp64 definitions of attention over what the pages hold."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import q8_ref  # noqa: E402
import serving_ref as ref  # noqa: E402
import test_gpu_prefix_attention as px  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402

host = px.host


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_users_behind_a_system_prompt(dt):
    ensure_built()
    el = px.DT[dt]
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N, Hq, Hkv, D, page, maxp, pages, P = 3, 4, 2, 64, 16, 6, 40, 150
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    ptable, table = perm[:10].view(1, 10), perm[10:10 + N * maxp].clone().view(N, maxp)
    tb, ptb = table.cpu().numpy(), ptable.cpu().numpy()
    kb, vb = (torch.zeros(pages, Hkv, page, D, dtype=torch.uint8, device="cuda").view(
        torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.full((pages, Hkv, page), 255, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    ang = torch.arange(512, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (
        -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    wq, wk = 1 + 0.2 * rn(D), 1 + 0.2 * rn(D)
    vals = {}  # slot -> the values appended there

    def append(pos, slots):
        T = len(pos)
        q, k, v = rn(T, Hq, D).to(el), rn(T, Hkv, D).to(el), rn(T, Hkv, D).to(el)
        qo = torch.empty_like(q)
        sl = torch.from_numpy(np.asarray(slots, np.int64)).cuda()
        kda.kda_qk_norm_rope_append_q8(
            q, k, v, wq, wk, cos, sin, torch.from_numpy(np.asarray(pos, np.int32)).cuda(), sl, qo,
            kb, vb, ks, vs, T, Hq, Hkv, D, D, 512, pages, page)
        ko, vo = (torch.empty(T, Hkv, D, dtype=el, device="cuda") for _ in range(2))
        kda.kda_paged_cache_read_q8(kb, vb, ks, vs, sl, ko, vo, T, Hkv, D, pages, page)
        want = ref.norm_rope(host(k), host(wk), host(cos)[pos], host(sin)[pos], D, 1e-6, False)
        top = np.abs(want).max(-1, keepdims=True)
        assert (np.abs(host(ko) - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -15 * top).all()
        b, s = q8_ref.quantise(host(v))
        assert (host(vo) == q8_ref.value(b, s)).all()
        vals.update(zip(map(int, slots), host(vo)))
        return qo

    at = lambda t, j: t[j // page].astype(np.int64) * page + j % page  # noqa: E731
    j = np.arange(P)
    qo = append(j, at(ptb[0], j))
    # the prompt itself is plain attention over its pages
    out = torch.empty(P, Hq, D, dtype=el, device="cuda")
    lse = torch.empty(P, Hq, device="cuda")
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kda.kda_paged_attention_q8_fwd(qo, kb, vb, ks, vs, ptable, i32(0, P), i32(P), out, 1, P, Hq,
                                   Hkv, D, pages, page, 10, lse=lse, workspace=ws)
    kx, vx = q8_ref.value(px_raw(kb), px_raw(ks)), q8_ref.value(px_raw(vb), px_raw(vs))
    r = ref.paged_attention(host(qo), kx, vx, ptb, [0, P], [P], page)
    half = 2.0 ** -8 if dt == "bf16" else 0.0
    assert (np.abs(host(out) - r[0]) <= 2e-4 * r[2] + half * (r[2] + np.abs(r[0]))).all()
    done = [0] * N
    for step in range(4):
        new = [37, 5, 50] if step == 0 else [1] * N
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        seq = np.repeat(np.arange(N), new)
        own = np.concatenate([np.arange(done[n], done[n] + new[n]) for n in range(N)])
        slots = tb[seq, own // page].astype(np.int64) * page + own % page
        qo = append(P + own, slots)
        done = [a + b for a, b in zip(done, new)]
        d = dict(q=qo, kc=kb, vc=vb, ks=ks, vs=vs, pt=ptable, pl=i32(P), cg=i32(0, N), table=table,
                 cu=torch.from_numpy(cu).cuda(), kv=i32(*done), G=1, N=N, T=T, live=T, Hq=Hq,
                 Hkv=Hkv, D=D, pages=pages, page=page, dt=dt, q8=True, cu_h=cu,
                 kv_h=np.array(done), pl_h=np.array([P]), groups_h=np.array([0, N]), table_h=tb,
                 pt_h=ptb, out=torch.empty(T, Hq, D, dtype=el, device="cuda"),
                 lse=torch.empty(T, Hq, device="cuda"))
        d["kx"], d["vx"] = (q8_ref.value(px_raw(b), px_raw(s)) for b, s in ((kb, ks), (vb, vs)))
        px.call(d)
        px.check(d)
    # all that was appended is still there
    sl = torch.tensor(sorted(vals), device="cuda")
    ko, vo = (torch.empty(len(vals), Hkv, D, dtype=el, device="cuda") for _ in range(2))
    kda.kda_paged_cache_read_q8(kb, vb, ks, vs, sl, ko, vo, len(vals), Hkv, D, pages, page)
    assert (host(vo) == np.stack([vals[s] for s in sorted(vals)])).all()


def px_raw(t):
    return t.view(torch.uint8).cpu().numpy()
