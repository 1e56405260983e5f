"""Operators of a hybrid delta-rule / softmax-attention stack, as workloads to be timed.

Three operators: the single-step serving form of the gated delta rule over a pool of states
(kda_attention_step), the per-head RMS norm of queries and keys with the position rotation in
the same pass (kda_qk_norm_rope_fwd / _bwd / _append), and attention of a chunk of new tokens
over a paged cache (kda_paged_attention_fwd).  Each has a plain form in elementary torch
operations (own = False) and the library's call (own = True)."""
import math
import random

import torch

own = False

EPS_L2 = 1e-6   # x / sqrt(sum x^2 + eps): the delta rule's q and k
EPS_RMS = 1e-6  # x / sqrt(mean x^2 + eps): the per-head norms
ROPE_BASE = 1e6


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one user's next token through one delta-rule layer: latency
        dict(name="step_one", op="step", N=1, tlo=1, thi=1, Hk=16, Hv=32, dk=128, dv=128,
             f32=False, fork=False, pad=0, literal=False, lens=1),
        # the decode batch of the library's benchmark, bf16 tokens, one token per request
        dict(name="step_batch64", op="step", N=64, tlo=1, thi=1, Hk=32, Hv=32, dk=128, dv=128,
             f32=False, fork=False, pad=0, literal=False, lens=2),
        # a few drafted tokens per request verified from a shared state into other slots, in a
        # padded batch, fp32
        dict(name="step_verify", op="step", N=37, tlo=1, thi=6, Hk=4, Hv=16, dk=64, dv=128,
             f32=True, fork=True, pad=3, literal=False, lens=3),
        # a decode batch's q, k, v out of the fused projection: normed, rotated, into the pages
        dict(name="rope_append_batch64", op="append", T=64, Hq=32, Hkv=8, D=128, R=128,
             page=64, interleaved=False, f32=False, pad=0, maxpos=8192),
        # the new tokens of a prefill chunk, half of each head rotated in neighbouring pairs, with
        # padded rows behind the chunk
        dict(name="rope_append_chunk", op="append", T=4095, Hq=16, Hkv=2, D=128, R=64,
             page=16, interleaved=True, f32=False, pad=31, maxpos=32768),
        # a training step's tokens (4 sequences of 4096), forward
        dict(name="rope_train_fwd", op="rope_fwd", T=16384, Hq=32, Hkv=8, D=128, R=128,
             interleaved=False, f32=False, maxpos=4096),
        # and backward, with the gradients of both weights
        dict(name="rope_train_bwd", op="rope_bwd", T=16384, Hq=32, Hkv=8, D=128, R=128,
             interleaved=False, f32=False, maxpos=4096),
        # one user's next token over its cache: latency
        dict(name="attn_decode_one", op="attn", N=1, qlo=1, qhi=1, plo=999, phi=999, Hq=32, Hkv=8,
             D=128, page=16, window=0, sinks=0, f32=False, lens=4),
        # a decode batch over ragged caches
        dict(name="attn_decode_batch64", op="attn", N=64, qlo=1, qhi=1, plo=511, phi=8191, Hq=32,
             Hkv=8, D=128, page=64, window=0, sinks=0, f32=False, lens=5),
        # long-prompt prefill: chunks of 4096 new tokens behind 12288 cached ones
        dict(name="attn_chunk_long", op="attn", N=2, qlo=4096, qhi=4096, plo=12288, phi=12288,
             Hq=32, Hkv=8, D=128, page=64, window=0, sinks=0, f32=False, lens=6),
        # decode tokens and chunks in one call, sliding window with first tokens kept visible
        dict(name="attn_window_mixed", op="attn", N=9, qlo=1, qhi=700, plo=0, phi=5000, Hq=16,
             Hkv=2, D=64, page=32, window=1024, sinks=4, f32=False, lens=7),
        # a small fp32 model's mixed batch
        dict(name="attn_f32_small", op="attn", N=5, qlo=1, qhi=17, plo=0, phi=700, Hq=4, Hkv=4,
             D=64, page=16, window=0, sinks=0, f32=True, lens=8),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed one."""
    op = rng.choice(["step", "step", "append", "rope_fwd", "rope_bwd", "attn", "attn", "attn"])
    lens = rng.randrange(1 << 30)
    if op == "step":
        Hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        Hv = Hk * rng.choice([1, 1, 2, 4])
        thi = _logint(rng, 1, 8)
        return dict(op=op, N=_logint(rng, 1, max(1, 2048 // Hv)), tlo=rng.choice([0, 1]),
                    thi=thi, Hk=Hk, Hv=Hv, dk=rng.choice([32, 64, 128, 128]),
                    dv=rng.choice([32, 64, 128, 128]), f32=rng.random() < 0.3,
                    fork=rng.random() < 0.4, pad=rng.choice([0, 0, 1, 5]),
                    literal=rng.random() < 0.2, lens=lens)
    if op in ("append", "rope_fwd", "rope_bwd"):
        Hkv = rng.choice([1, 2, 3, 4, 8])
        D = rng.choice([32, 64, 128, 128])
        c = dict(op=op, T=_logint(rng, 1, 16384), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D,
                 R=rng.choice([D, D, D // 2, 16, 0]), interleaved=rng.random() < 0.4,
                 f32=rng.random() < 0.3, maxpos=_logint(rng, 64, 65536))
        if op == "append":
            c.update(page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, 1, 17]))
        return c
    D = rng.choice([32, 64, 64, 128, 128, 128])
    f32 = rng.random() < 0.2
    Hkv = rng.choice([1, 2, 3, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16] if Hkv <= 2 else [1, 2, 3, 4])
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    if kind == "decode":
        N = _logint(rng, 1, 128)
        q = (1, rng.choice([1, 1, 2, 5]))
        phi = _logint(rng, 1, 100000 if N <= 4 else 8192)
    elif kind == "chunk":
        N = _logint(rng, 1, 4)
        q = (_logint(rng, 16, 2048),) * 2
        phi = _logint(rng, 1, 16384)
    else:
        N = _logint(rng, 2, 24)
        q = (rng.choice([0, 1]), _logint(rng, 2, 900))
        phi = _logint(rng, 1, 6000)
    if f32 or D == 32:  # fp32 and narrow heads: small models
        phi = min(phi, 4096)
        q = tuple(min(x, 256) for x in q)
        N = min(N, 16)
    w = rng.choice([0, 0, _logint(rng, 1, 4096)])
    return dict(op="attn", N=N, qlo=q[0], qhi=q[1], plo=rng.choice([0, phi // 2, phi]), phi=phi,
                Hq=Hq, Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]), window=w,
                sinks=rng.choice([0, 1, 4, 100]) if w else 0, f32=f32, lens=lens)


# ------------------------------------------------------------- sizes that follow from a case

def _step_lens(c):
    r = random.Random(c["lens"])
    lens = [r.randint(c["tlo"], c["thi"]) for _ in range(c["N"])]
    return [max(lens[0], 1)] + lens[1:]


def _attn_lens(c):
    """(new tokens, cached tokens before them) of each sequence."""
    r = random.Random(c["lens"])
    lens = [(r.randint(c["qlo"], c["qhi"]), r.randint(c["plo"], c["phi"])) for _ in range(c["N"])]
    return [(max(lens[0][0], 1), lens[0][1])] + lens[1:]


def _visible_pairs(q, p, window, sinks):
    """Visible (query, key) pairs of q new tokens behind p cached ones, and the distinct keys."""
    if window <= 0:
        return q * p + q * (q + 1) // 2, (p + q if q else 0)
    pairs = 0
    for i in range(q):
        pos = p + i
        lo = max(0, pos - window + 1)
        pairs += pos - lo + 1 + min(sinks, lo)
    lo0 = max(0, p - window + 1)
    return pairs, (p + q - lo0 + min(sinks, lo0) if q else 0)


def work(case):
    c = case
    e = 4 if c["f32"] else 2
    if c["op"] == "step":
        lens = _step_lens(c)
        rows = sum(lens)
        state = 2 * c["N"] * c["Hv"] * c["dk"] * c["dv"] * 4
        tok = rows * (e * (2 * c["Hk"] * c["dk"] + 2 * c["Hv"] * c["dv"]) + 8 * c["Hv"])
        return {"bytes": state + tok, "flops": rows * c["Hv"] * 7 * c["dk"] * c["dv"]}
    if c["op"] == "attn":
        b = f = 0
        for q, p in _attn_lens(c):
            pairs, keys = _visible_pairs(q, p, c["window"], c["sinks"])
            f += 4 * c["D"] * c["Hq"] * pairs
            b += e * c["D"] * (2 * c["Hq"] * q + 2 * c["Hkv"] * keys)
        return {"bytes": b, "flops": f}
    heads = c["Hq"] + c["Hkv"]
    tok = 4 * c["T"] + 4 * c["R"] * min(c["T"], c["maxpos"])
    if c["op"] == "append":
        b = c["T"] * c["D"] * e * 2 * (heads + c["Hkv"]) + tok + 8 * c["T"]
        f = c["T"] * heads * c["D"] * 8
    elif c["op"] == "rope_fwd":
        b = c["T"] * c["D"] * e * 2 * heads + tok
        f = c["T"] * heads * c["D"] * 8
    else:
        b = c["T"] * c["D"] * e * 3 * heads + tok
        f = c["T"] * heads * c["D"] * 16
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    c = case
    g = _gen(seed * 1000003 + 17)
    dt = torch.float32 if c["f32"] else torch.bfloat16
    s = {"case": c}
    if c["op"] == "step":
        lens = _step_lens(c)
        cu = _offsets(lens)
        rows = cu[-1] + c["pad"]
        Hk, Hv, dk, dv, N = c["Hk"], c["Hv"], c["dk"], c["dv"], c["N"]
        # q, k, v as views of one projection's rows
        qkv = _randn(g, rows, 2 * Hk * dk + Hv * dv, dtype=dt)
        s["q"] = qkv[:, :Hk * dk].view(rows, Hk, dk)
        s["k"] = qkv[:, Hk * dk:2 * Hk * dk].view(rows, Hk, dk)
        s["v"] = qkv[:, 2 * Hk * dk:].view(rows, Hv, dv)
        s["beta"] = torch.sigmoid(_randn(g, rows, Hv))
        s["decay"] = -torch.nn.functional.softplus(_randn(g, rows, Hv) - 2.0)
        slots = N + 2 + (N if c["fork"] else 0)
        s["pool"] = _randn(g, slots, Hv, dk, dv, std=0.05)
        perm = torch.randperm(slots, generator=g, device="cuda").to(torch.int32)
        s["slots"] = perm[:N].clone()
        s["out_slots"] = perm[N:2 * N].clone() if c["fork"] else None
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["lens"], s["cu_host"], s["num_slots"], s["rows"] = lens, cu, slots, rows
        s["out"] = torch.zeros(rows, Hv, dv, dtype=dt, device="cuda")
    elif c["op"] == "attn":
        lens = _attn_lens(c)
        page, D, Hq, Hkv = c["page"], c["D"], c["Hq"], c["Hkv"]
        q_cu = _offsets([q for q, _ in lens])
        kv = [q + p for q, p in lens]
        need = [(n + page - 1) // page for n in kv]
        pages = sum(need) + 3
        maxp = max(max(need), 1)
        s["q"] = _randn(g, q_cu[-1], Hq, D, dtype=dt)
        s["kc"] = torch.empty(pages, Hkv, page, D, dtype=dt, device="cuda").normal_(generator=g)
        s["vc"] = torch.empty(pages, Hkv, page, D, dtype=dt, device="cuda").normal_(generator=g)
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
        table = torch.zeros(len(lens), maxp, dtype=torch.int32)
        at = 0
        for n, m in enumerate(need):
            table[n, :m] = perm[at:at + m]
            at += m
        s["table"] = table.cuda()
        s["cu"] = torch.tensor(q_cu, dtype=torch.int32, device="cuda")
        s["kv"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["lens"], s["cu_host"], s["pages"], s["maxp"] = lens, q_cu, pages, maxp
        s["out"] = torch.zeros(q_cu[-1], Hq, D, dtype=dt, device="cuda")
    else:
        T, Hq, Hkv, D, R = c["T"], c["Hq"], c["Hkv"], c["D"], c["R"]
        if c["op"] == "append":
            qkv = _randn(g, T, (Hq + 2 * Hkv) * D, dtype=dt, std=1.5)
            s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
            s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
            s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
            page = c["page"]
            pages = (T + page - 1) // page + 5
            s["kc"] = _randn(g, pages, Hkv, page, D, dtype=dt)
            s["vc"] = _randn(g, pages, Hkv, page, D, dtype=dt)
            # tokens of many requests land anywhere; padded rows have no place
            slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].clone()
            if c["pad"]:
                slots[max(0, T - c["pad"]):] = -1
            s["slots"], s["pages"] = slots, pages
        else:
            s["q"] = _randn(g, T, Hq, D, dtype=dt, std=1.5)
            s["k"] = _randn(g, T, Hkv, D, dtype=dt, std=1.5)
            if c["op"] == "rope_bwd":
                s["dyq"] = _randn(g, T, Hq, D, dtype=dt)
                s["dyk"] = _randn(g, T, Hkv, D, dtype=dt)
        s["wq"] = 1.0 + _randn(g, D, std=0.2)
        s["wk"] = 1.0 + _randn(g, D, std=0.2)
        s["pos"] = torch.randint(0, c["maxpos"], (T,), generator=g, device="cuda",
                                 dtype=torch.int32)
        # the rotation's table, its angles in 64 bits
        inv = ROPE_BASE ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) /
                            max(R, 1))
        ang = torch.arange(c["maxpos"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    if own:
        s["ws"] = _workspace(s)
    return s


def _workspace(s):
    """The scratch buffer that a program keeps for a call of these sizes."""
    import gated_delta_rule_55_gb300 as kda
    c, n = s["case"], 0
    if c["op"] == "attn":
        n = kda.kda_paged_attention_fwd_workspace_size(
            c["N"], s["cu_host"][-1], c["Hq"], c["Hkv"], c["D"],
            dtype=kda.KDA_F32 if c["f32"] else kda.KDA_BF16)
    elif c["op"] == "rope_bwd":
        n = kda.kda_qk_norm_rope_bwd_workspace_size(c["T"], c["Hq"], c["Hkv"], c["D"])
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


# ---------------------------------------------------------------------------- plain forms

def _plain_step(s):
    c = s["case"]
    rep = c["Hv"] // c["Hk"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS_L2) * c["dk"] ** -0.5
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS_L2)
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    S = s["pool"][s["slots"].long()]
    out = torch.zeros(q.shape[0], c["Hv"], c["dv"], device="cuda")
    for t in range(max(s["lens"], default=0)):
        live = [n for n, m in enumerate(s["lens"]) if m > t]
        rows = torch.tensor([s["cu_host"][n] + t for n in live], device="cuda")
        idx = torch.tensor(live, device="cuda")
        M = S[idx]
        kt, qt = k[rows][..., None], q[rows][..., None]
        dec = torch.exp(s["decay"][rows])[..., None, None]
        if c["literal"]:
            seen = (M * kt).sum(-2)
            M = M * dec
        else:
            M = M * dec
            seen = (M * kt).sum(-2)
        u = s["beta"][rows][..., None] * (v[rows] - seen)
        M = M + kt * u[..., None, :]
        out[rows] = (M * qt).sum(-2)
        S[idx] = M
    dst = s["slots"] if s["out_slots"] is None else s["out_slots"]
    s["pool"][dst.long()] = S
    return {"out": out.to(s["q"].dtype), "state": s["pool"]}


def _rotate(x, cos, sin, R, interleaved, sign):
    """Rotates the first R elements of x [T, H, D] by the angles of cos, sin [T, R / 2]."""
    if R == 0:
        return x
    cos, sin = cos[:, None], sin[:, None] * sign
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * cos - b * sin
        y[..., 1:R:2] = a * sin + b * cos
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * cos - b * sin
        y[..., R // 2:R] = a * sin + b * cos
    return y


def _plain_norm_rope(x, w, cos, sin, c):
    x = x.float()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS_RMS) * w
    return _rotate(y, cos, sin, c["R"], c["interleaved"], 1.0)


def _plain_rope(s):
    c = s["case"]
    dt = s["q"].dtype
    pos = s["pos"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    if c["op"] == "rope_bwd":
        out = {}
        for n in "qk":
            x, w = s[n].float(), s["w" + n]
            gr = _rotate(s["dy" + n].float(), cos, sin, c["R"], c["interleaved"], -1.0)
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS_RMS)
            gw = gr * w
            out["d" + n] = (r * (gw - x * r * r * (gw * x).mean(-1, keepdim=True))).to(dt)
            # a long sum: in 64 bits
            out["dw" + n] = (gr * x * r).sum((0, 1), dtype=torch.float64).float()
        return out
    q = _plain_norm_rope(s["q"], s["wq"], cos, sin, c).to(dt)
    k = _plain_norm_rope(s["k"], s["wk"], cos, sin, c).to(dt)
    if c["op"] == "rope_fwd":
        return {"q": q, "k": k}
    live = (s["slots"] >= 0).nonzero()[:, 0]
    sl = s["slots"][live]
    pg, of = sl // c["page"], sl % c["page"]
    s["kc"][pg, :, of] = k[live]
    s["vc"][pg, :, of] = s["v"][live]
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _gather(cache, table_row, n, page):
    """The first n tokens of a sequence: [n, Hkv, D]."""
    m = (n + page - 1) // page
    x = cache[table_row[:m].long()]
    return x.permute(0, 2, 1, 3).reshape(m * page, x.shape[1], x.shape[3])[:n]


def _plain_attn(s):
    c = s["case"]
    G, D = c["Hq"] // c["Hkv"], c["D"]
    out = torch.zeros(s["q"].shape[0], c["Hq"], D, device="cuda")
    for n, (ql, p) in enumerate(s["lens"]):
        if ql == 0:
            continue
        kv = p + ql
        a = s["cu_host"][n]
        K = _gather(s["kc"], s["table"][n], kv, c["page"]).float()
        V = _gather(s["vc"], s["table"][n], kv, c["page"]).float()
        j = torch.arange(kv, device="cuda")
        blk = max(1, (1 << 28) // (kv * c["Hq"]))
        for i0 in range(0, ql, blk):
            i1 = min(ql, i0 + blk)
            q = s["q"][a + i0:a + i1].float().view(i1 - i0, c["Hkv"], G, D)
            pos = (p + torch.arange(i0, i1, device="cuda"))[:, None]
            hide = j[None] > pos
            if c["window"]:
                hide |= (j[None] <= pos - c["window"]) & (j[None] >= c["sinks"])
            sc = torch.matmul(q.permute(1, 2, 0, 3), K.permute(1, 2, 0)[:, None]) * D ** -0.5
            sc.masked_fill_(hide, float("-inf"))
            sc -= sc.amax(-1, keepdim=True)
            sc.exp_()
            o = torch.matmul(sc, V.permute(1, 0, 2)[:, None]) / sc.sum(-1, keepdim=True)
            out[a + i0:a + i1] = o.permute(2, 0, 1, 3).reshape(i1 - i0, c["Hq"], D)
    return {"out": out.to(s["q"].dtype)}


# -------------------------------------------------------------------------- library calls

def _own(s):
    import gated_delta_rule_55_gb300 as kda
    c = s["case"]
    if "ws" not in s:
        s["ws"] = _workspace(s)
    if c["op"] == "step":
        kda.kda_attention_step(
            s["q"], s["k"], s["v"], s["beta"], s["decay"], s["pool"], s["slots"], s["out"],
            c["N"], s["rows"], c["Hk"], c["Hv"], c["dk"], c["dv"], s["num_slots"],
            out_slots=s["out_slots"], cu_seqlens=s["cu"],
            order="literal" if c["literal"] else "decay_first")
        return {"out": s["out"], "state": s["pool"]}
    if c["op"] == "attn":
        kda.kda_paged_attention_fwd(
            s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["kv"], s["out"], c["N"],
            s["cu_host"][-1], c["Hq"], c["Hkv"], c["D"], s["pages"], c["page"], s["maxp"],
            window=c["window"], sinks=c["sinks"], workspace=s["ws"])
        return {"out": s["out"]}
    if c["op"] == "rope_bwd":
        dq, dk = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        dwq, dwk = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        kda.kda_qk_norm_rope_bwd(
            s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["dyq"], s["dyk"],
            dq, dk, dwq, dwk, c["T"], c["Hq"], c["Hkv"], c["D"], c["R"], c["maxpos"],
            eps=EPS_RMS, interleaved=c["interleaved"], workspace=s["ws"])
        return {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}
    q = torch.empty(c["T"], c["Hq"], c["D"], dtype=s["q"].dtype, device="cuda")
    if c["op"] == "rope_fwd":
        k = torch.empty_like(s["k"])
        kda.kda_qk_norm_rope_fwd(
            s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], q, k, c["T"],
            c["Hq"], c["Hkv"], c["D"], c["R"], c["maxpos"], eps=EPS_RMS,
            interleaved=c["interleaved"])
        return {"q": q, "k": k}
    kda.kda_qk_norm_rope_append(
        s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["slots"], q,
        s["kc"], s["vc"], c["T"], c["Hq"], c["Hkv"], c["D"], c["R"], c["maxpos"], s["pages"],
        c["page"], eps=EPS_RMS, interleaved=c["interleaved"])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "step":
        return _plain_step(state)
    if op == "attn":
        return _plain_attn(state)
    return _plain_rope(state)


# ------------------------------------------------------------- the definitions in 64 bits

def _exact_step(s):
    c = s["case"]
    rep = c["Hv"] // c["Hk"]
    pool = s["pool"].double()
    out = torch.zeros(s["rows"], c["Hv"], c["dv"], dtype=torch.float64, device="cuda")
    src = s["slots"].tolist()
    dst = src if s["out_slots"] is None else s["out_slots"].tolist()
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    dec, beta = s["decay"].double().exp(), s["beta"].double()
    new = []
    for n in range(c["N"]):
        S = pool[src[n]].clone()
        for row in range(s["cu_host"][n], s["cu_host"][n + 1]):
            qn = q[row] * (c["dk"] ** -0.5 * (q[row].square().sum(1, True) + EPS_L2).rsqrt())
            kn = k[row] * (k[row].square().sum(1, True) + EPS_L2).rsqrt()
            qn, kn = (x[:, None].expand(-1, rep, -1).reshape(c["Hv"], c["dk"]) for x in (qn, kn))
            old = torch.einsum("hkv,hk->hv", S, kn)
            S = S * dec[row][:, None, None]
            if not c["literal"]:
                old = old * dec[row][:, None]
            S = S + torch.einsum("hk,hv->hkv", kn, beta[row][:, None] * (v[row] - old))
            out[row] = torch.einsum("hkv,hk->hv", S, qn)
        new.append((dst[n], S))
    for d, S in new:
        pool[d] = S
    return {"out": out, "state": pool}


def _pair_index(c):
    """For each element of a head: its partner, the sign of the partner's sine, its angle."""
    D, R = c["D"], c["R"]
    mate, sign, ang = list(range(D)), [0.0] * D, [-1] * D
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        mate[a], mate[b], sign[a], sign[b], ang[a], ang[b] = b, a, -1.0, 1.0, i, i
    return mate, sign, ang


def _exact_rope(s):
    c = s["case"]
    mate, sign, ang = _pair_index(c)
    mate = torch.tensor(mate, device="cuda")
    sign = torch.tensor(sign, dtype=torch.float64, device="cuda")
    rot = torch.tensor([a >= 0 for a in ang], device="cuda")
    ai = torch.tensor([max(a, 0) for a in ang], device="cuda")
    p = s["pos"].long()
    if c["R"]:
        one = torch.ones((), dtype=torch.float64, device="cuda")
        C = torch.where(rot, s["cos"].double()[p][:, ai], one)[:, None]
        Sn = (torch.where(rot, s["sin"].double()[p][:, ai], 0 * one) * sign)[:, None]
    else:
        C, Sn = 1.0, torch.zeros(1, 1, 1, dtype=torch.float64, device="cuda")

    def spin(x, way):
        return x * C + x[..., mate] * Sn * way

    res = {}
    for n in "qk":
        x, w = s[n].double(), s["w" + n].double()
        inv = (x.square().mean(-1, keepdim=True) + EPS_RMS).pow(-0.5)
        xh = x * inv
        if c["op"] == "rope_bwd":
            gr = spin(s["dy" + n].double(), -1.0)
            t = gr * w
            res["d" + n] = inv * (t - xh * (t * xh).mean(-1, keepdim=True))
            res["dw" + n] = torch.einsum("thd,thd->d", gr, xh)
        else:
            res[n] = spin(xh * w, 1.0)
    if c["op"] != "append":
        return res
    kc, vc = s["kc"].double(), s["vc"].double()
    v = s["v"].double()
    ok = s["slots"] >= 0
    flat = s["slots"][ok]
    kc = kc.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
    vc = vc.transpose(1, 2).reshape(-1, c["Hkv"], c["D"])
    kc[flat], vc[flat] = res["k"][ok], v[ok]
    shape = (s["pages"], c["page"], c["Hkv"], c["D"])
    return {"q": res["q"], "k_cache": kc.view(shape).transpose(1, 2).contiguous(),
            "v_cache": vc.view(shape).transpose(1, 2).contiguous()}


def _exact_attn(s):
    c = s["case"]
    G = c["Hq"] // c["Hkv"]
    out = torch.zeros(s["q"].shape[0], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    for n, (ql, p) in enumerate(s["lens"]):
        if ql == 0:
            continue
        a, kv = s["cu_host"][n], p + ql
        at = torch.arange(kv, device="cuda")
        row = s["table"][n][at // c["page"]].long()
        where = p + torch.arange(ql, device="cuda")
        gap = where[:, None] - at[None, :]
        see = gap >= 0
        if c["window"] > 0:
            see &= (gap < c["window"]) | (at[None, :] < c["sinks"])
        for h in range(c["Hkv"]):
            k = s["kc"][row, h, at % c["page"]].double()
            v = s["vc"][row, h, at % c["page"]].double()
            for hq in range(h * G, (h + 1) * G):
                x = s["q"][a:a + ql, hq].double() @ k.T / math.sqrt(c["D"])
                x = torch.where(see, x, torch.full_like(x, -math.inf))
                out[a:a + ql, hq] = torch.softmax(x, -1) @ v
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "attn":
        return _exact_attn(s)
    return _exact_rope(s)
