"""The serving operators as they are used together: a stack of one delta-rule layer and one
softmax layer, a prompt chunk followed by single tokens, against the fp64 definitions on the
same (rounded) intermediate values."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gated_delta_rule_55_gb300 as kda  # noqa: E402
import serving_ref as ref  # noqa: E402
import test_gpu_paged_attention as pa  # noqa: E402
from gpu_helpers import ensure_built  # noqa: E402


def host(x):
    return x.detach().double().cpu().numpy()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_hybrid_stack(dt):
    ensure_built()
    el = pa.DT[dt]
    g = torch.Generator(device="cuda").manual_seed(5)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    N, Hq, Hkv, D, page, maxp, pages = 3, 4, 2, 64, 16, 6, 20
    Hv = 4
    prompts = [37, 5, 50]
    table = torch.randperm(pages, generator=g, device="cuda")[:N * maxp].view(N, maxp).int()
    kc, vc = torch.zeros(pages, Hkv, page, D, device="cuda", dtype=el), torch.zeros(
        pages, Hkv, page, D, device="cuda", dtype=el)
    pool = torch.zeros(N, Hv, D, D, device="cuda")
    sl = torch.arange(N, dtype=torch.int32, device="cuda")
    ang = torch.arange(128, device="cuda", dtype=torch.float64)[:, None] * 1e4 ** (
        -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
    cos, sin = ang.cos().float(), ang.sin().float()
    wq, wk = 1 + 0.2 * rn(D), 1 + 0.2 * rn(D)
    done = [0] * N
    K = [np.zeros((0, Hkv, D))] * N  # the definition's own cache
    V = [np.zeros((0, Hkv, D))] * N
    rpool = host(pool)
    for step in range(4):
        new = prompts if step == 0 else [1] * N
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(cu[-1])
        cud = torch.from_numpy(cu).cuda()
        pos = np.concatenate([np.arange(done[n], done[n] + new[n]) for n in range(N)])
        seq = np.concatenate([np.full(new[n], n) for n in range(N)])
        tb = table.cpu().numpy()
        slots = torch.from_numpy(tb[seq, pos // page].astype(np.int64) * page + pos % page).cuda()
        qkv = rn(T, (Hq + 2 * Hkv) * D).to(el)
        q = qkv[:, :Hq * D].view(T, Hq, D)
        k = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        v = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        qo = torch.empty(T, Hq, D, dtype=el, device="cuda")
        att = torch.empty(T, Hq, D, dtype=el, device="cuda")
        lse = torch.empty(T, Hq, device="cuda")
        kda.kda_qk_norm_rope_append(q, k, v, wq, wk, cos, sin,
                                    torch.from_numpy(pos.astype(np.int32)).cuda(), slots, qo, kc,
                                    vc, T, Hq, Hkv, D, D, 128, pages, page)
        kv = [done[n] + new[n] for n in range(N)]
        kvd = torch.tensor(kv, dtype=torch.int32, device="cuda")
        n_ws = kda.kda_paged_attention_fwd_workspace_size(
            N, T, Hq, Hkv, D, dtype=kda.KDA_F32 if dt == "f32" else kda.KDA_BF16)
        ws = torch.empty(max(n_ws, 1), dtype=torch.uint8, device="cuda")
        kda.kda_paged_attention_fwd(qo, kc, vc, table, cud, kvd, att, N, T, Hq, Hkv, D, pages,
                                    page, maxp, lse=lse, window=40, sinks=2, workspace=ws)
        # the softmax layer's output is the delta-rule layer's value
        beta, decay = torch.sigmoid(rn(T, Hv)), -torch.rand(T, Hv, generator=g, device="cuda")
        out = torch.empty(T, Hv, D, dtype=el, device="cuda")
        kda.kda_attention_step(q[:, :2], k, att, beta, decay, pool, sl, out, N, T, 2, Hv, D, D,
                               N, cu_seqlens=cud)
        torch.cuda.synchronize()
        # norm and rotation
        c, s = host(cos)[pos], host(sin)[pos]
        rq = ref.norm_rope(host(q), host(wq), c, s, D, 1e-6, False)
        rk = ref.norm_rope(host(k), host(wk), c, s, D, 1e-6, False)
        half = 2.0 ** -8 if dt == "bf16" else 0.0
        assert (np.abs(host(qo) - rq) <= half * np.abs(rq) + 1e-5).all()
        # attention over what the pages hold, which is what was appended
        d = dict(q=qo, out=att, lse=lse, D=D, dt=dt, kv_h=np.array(kv), live=T)
        r = ref.paged_attention(host(qo), host(kc), host(vc), tb, cu, kv, page, window=40,
                                sinks=2)
        pa.compare(d, r)
        for n in range(N):
            K[n] = np.concatenate([K[n], rk[cu[n]:cu[n + 1]]])
            V[n] = np.concatenate([V[n], host(v)[cu[n]:cu[n + 1]]])
            assert (np.abs(ref.key_rows(host(kc), tb[n], kv[n], page) - K[n]) <=
                    half * np.abs(K[n]) + 1e-5).all()
            assert (ref.key_rows(host(vc), tb[n], kv[n], page) == V[n]).all()
        # the delta rule on the attention's (rounded) output
        ro, rpool = ref.step(host(q)[:, :2], host(k), host(att), host(beta), host(decay), rpool,
                             list(range(N)), cu)
        tol = 2 * (D + 16) * max(prompts) * 2.0 ** -24 * max(1.0, np.abs(rpool).max())
        assert (np.abs(host(out) - ro) <= tol + half * np.abs(ro)).all()
        assert (np.abs(host(pool) - rpool) <= tol * (step + 1)).all()
        done = kv
