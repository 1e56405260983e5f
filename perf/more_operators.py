"""Serving from 8-bit pages and from shared prefixes, as workloads to be timed.

Operators: the append of normed and rotated keys and of values into a paged cache that holds
them in 8 bits (kda_qk_norm_rope_append_q8), reading kept tokens back (kda_paged_cache_read_q8),
attention over such pages (kda_paged_attention_q8_fwd), and attention of a batch whose sequences
share long prefixes, each of which is worked on once for all of them
(kda_paged_prefix_attention_fwd).  Each has a plain form in elementary torch operations
(own = False) and the library's calls (own = True).

A kept row (one token's key or value of one kv head) is D numbers of e4m3 and one byte e: it
stands for number * 2^(e - 127), with the smallest power of two whose 448-fold reaches the row's
largest magnitude."""
import math
import random

import torch

own = False

EPS_RMS = 1e-6
ROPE_BASE = 1e6
E4M3_MAX = 448.0
SCALE_LO, SCALE_HI = -110, 119  # exponents of a row's scale


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode batch's q, k, v out of the fused projection, into 8-bit pages, and the same
        # tokens read back
        dict(name="q8_append_batch64", op="append", T=64, Hq=32, Hkv=8, D=128, R=128, page=64,
             interleaved=False, f32=False, pad=0, maxpos=8192),
        # the new tokens of a prefill chunk, half of each head rotated in neighbouring pairs, with
        # padded rows behind the chunk
        dict(name="q8_append_chunk", op="append", T=4095, Hq=16, Hkv=2, D=128, R=64, page=16,
             interleaved=True, f32=False, pad=31, maxpos=32768),
        # a cached context of four sequences of 4096 tokens handed to a dense kernel
        dict(name="q8_read_context", op="read", T=16384, Hkv=8, D=128, page=64, f32=False, pad=0),
        # a short context of a small fp32 model, some of its tokens gone
        dict(name="q8_read_small", op="read", T=333, Hkv=4, D=64, page=32, f32=True, pad=5),
        # one user's next token over its cache: latency
        dict(name="q8_attn_one", op="attn", N=1, qlo=1, qhi=1, plo=999, phi=999, Hq=32, Hkv=8,
             D=128, page=16, window=0, sinks=0, f32=False, lens=4),
        # a decode batch over ragged caches
        dict(name="q8_attn_batch64", op="attn", N=64, qlo=1, qhi=1, plo=511, phi=8191, Hq=32,
             Hkv=8, D=128, page=64, window=0, sinks=0, f32=False, lens=5),
        # prefill chunks behind a cache
        dict(name="q8_attn_chunk", op="attn", N=2, qlo=2048, qhi=2048, plo=8192, phi=8192, Hq=32,
             Hkv=8, D=128, page=64, window=0, sinks=0, f32=False, lens=6),
        # decode tokens and chunks in one call, sliding window with first tokens kept visible
        dict(name="q8_attn_window_mixed", op="attn", N=9, qlo=1, qhi=700, plo=0, phi=5000, Hq=16,
             Hkv=2, D=64, page=32, window=1024, sinks=4, f32=False, lens=7),
        # four users behind one system prompt: latency
        dict(name="prefix_few", op="prefix", N=4, groups=1, Llo=1000, Lhi=1000, qlo=1, qhi=1, plo=0,
             phi=60, Hq=16, Hkv=4, D=128, page=16, q8=False, f32=False, lens=8),
        # a decode batch in which all sequences answer about one long document
        dict(name="prefix_decode64", op="prefix", N=64, groups=1, Llo=16384, Lhi=16384, qlo=1,
             qhi=1, plo=15, phi=1023, Hq=32, Hkv=8, D=128, page=64, q8=False, f32=False, lens=9),
        # drafted tokens of 37 sequences behind five prompts of their own lengths, 8-bit pages
        dict(name="prefix_groups_q8", op="prefix", N=37, groups=5, Llo=300, Lhi=6000, qlo=1, qhi=6,
             plo=0, phi=700, Hq=16, Hkv=2, D=64, page=32, q8=True, f32=False, lens=10),
        # eight questions about one document, prefilled behind it
        dict(name="prefix_chunk", op="prefix", N=8, groups=1, Llo=8191, Lhi=8191, qlo=100, qhi=512,
             plo=0, phi=0, Hq=32, Hkv=8, D=128, page=64, q8=False, f32=False, lens=11),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the same ranges; costs no more than the largest listed one."""
    op = rng.choice(["append", "read", "attn", "attn", "attn", "prefix", "prefix", "prefix"])
    lens = rng.randrange(1 << 30)
    Hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        D = rng.choice([32, 64, 128, 128])
        return dict(op=op, T=_logint(rng, 1, 8192), Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv,
                    D=D, R=rng.choice([D, D, D // 2, 16, 0]), page=page,
                    interleaved=rng.random() < 0.4, f32=rng.random() < 0.3,
                    pad=rng.choice([0, 0, 1, 17]), maxpos=_logint(rng, 64, 65536))
    if op == "read":
        return dict(op=op, T=_logint(rng, 1, 16384), Hkv=Hkv, D=rng.choice([32, 64, 128, 128]),
                    page=page, f32=rng.random() < 0.3, pad=rng.choice([0, 0, 1, 17]))
    D = rng.choice([32, 64, 64, 128, 128, 128])
    f32 = rng.random() < 0.2
    Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16] if Hkv <= 2 else [1, 2, 3, 4])
    kind = rng.choice(["decode", "decode", "chunk", "mixed"])
    if kind == "decode":
        N = _logint(rng, 1, 128)
        q = (1, rng.choice([1, 1, 2, 5]))
    elif kind == "chunk":
        N = _logint(rng, 1, 4)
        q = (_logint(rng, 16, 1500),) * 2
    else:
        N = _logint(rng, 2, 24)
        q = (rng.choice([0, 1]), _logint(rng, 2, 700))
    if f32 or D == 32:  # fp32 and narrow heads: small models
        q = tuple(min(x, 200) for x in q)
        N = min(N, 16)
    # keys: at most what the padded scores and cache rows of the plain form leave room for
    most = min(8192, int(1.5e9 / (N * Hq * max(q[1], 8))), int(1e9 / (N * Hkv * D)))
    if f32 or D == 32:
        most = min(most, 4096)
    c = dict(op=op, N=N, qlo=q[0], qhi=q[1], Hq=Hq, Hkv=Hkv, D=D, page=page, f32=f32, lens=lens)
    if op == "attn":
        phi = _logint(rng, 1, most)
        w = rng.choice([0, 0, _logint(rng, 1, 4096)])
        c.update(plo=rng.choice([0, phi // 2, phi]), phi=phi, window=w,
                 sinks=rng.choice([0, 1, 4, 100]) if w else 0)
    else:
        phi = _logint(rng, 1, max(1, most // 4))
        hi = _logint(rng, 1, max(1, most * 3 // 4))
        c.update(groups=rng.randint(1, min(N, 6)), Llo=rng.choice([0, hi // 2, hi]), Lhi=hi,
                 plo=rng.choice([0, phi // 2, phi]), phi=phi, q8=rng.random() < 0.5)
    return c


# ------------------------------------------------------------- sizes that follow from a case

def _attn_lens(c):
    """(new tokens, cached tokens before them) of each sequence."""
    r = random.Random(c["lens"])
    lens = [(r.randint(c["qlo"], c["qhi"]), r.randint(c["plo"], c["phi"])) for _ in range(c["N"])]
    return [(max(lens[0][0], 1), lens[0][1])] + lens[1:]


def _groups(c):
    """Where each group of sequences starts (and the end), and the prefixes' lengths."""
    r = random.Random(c["lens"] + 1)
    cuts = sorted(r.sample(range(1, c["N"]), c["groups"] - 1)) if c["groups"] > 1 else []
    return [0] + cuts + [c["N"]], [r.randint(c["Llo"], c["Lhi"]) for _ in range(c["groups"])]


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
    if c["op"] == "append":
        heads = c["Hq"] + 2 * c["Hkv"]
        rows = 2 * c["Hkv"] * c["T"]  # kept: written, read back, written out as bf16
        b = (c["T"] * c["D"] * e * (heads + c["Hq"]) + rows * (2 * (c["D"] + 1) + 2 * c["D"]) +
             4 * c["T"] + 4 * c["R"] * min(c["T"], c["maxpos"]) + 16 * c["T"])
        return {"bytes": b, "flops": c["T"] * heads * c["D"] * 8}
    if c["op"] == "read":
        rows = 2 * c["Hkv"] * c["T"]
        return {"bytes": rows * (c["D"] + 1 + e * c["D"]) + 8 * c["T"], "flops": rows * c["D"]}
    b = f = 0
    lens = _attn_lens(c)
    kept = c["D"] + 1 if c["op"] == "attn" or c["q8"] else e * c["D"]  # bytes of a cached row
    for q, p in lens:
        pairs, keys = _visible_pairs(q, p, c.get("window", 0), c.get("sinks", 0))
        f += 4 * c["D"] * c["Hq"] * pairs
        b += 2 * e * c["D"] * c["Hq"] * q + 2 * kept * c["Hkv"] * keys
    if c["op"] == "prefix":
        starts, Lp = _groups(c)
        for g, n in enumerate(Lp):
            tokens = sum(q for q, _ in lens[starts[g]:starts[g + 1]])
            f += 4 * c["D"] * c["Hq"] * tokens * n
            b += 2 * kept * c["Hkv"] * n if tokens else 0
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pages(s, g, pages):
    """The caches of a case: k and v [pages, Hkv, page, D], as the tokens before left them."""
    c = s["case"]
    shape = (pages, c["Hkv"], c["page"], c["D"])
    for n in "kv":
        # rows of different magnitudes: values vary from token to token and head to head
        x = torch.empty(shape, device="cuda").normal_(generator=g)
        if c.get("q8", True):
            mag = torch.empty(shape[:3], device="cuda").normal_(0.0, 0.7, generator=g).exp_()
            x *= mag[..., None]
            s[n + "c"], s[n + "s"] = _quantise(x)
        else:
            s[n + "c"] = x.to(torch.float32 if c["f32"] else torch.bfloat16)
            s[n + "s"] = None


def _tables(g, needs, pages):
    """A block table for each list of needed page counts, all pages different."""
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    at, tables = 0, []
    for need in needs:
        t = torch.zeros(len(need), max(need + [1]), dtype=torch.int32)
        for n, m in enumerate(need):
            t[n, :m] = perm[at:at + m]
            at += m
        tables.append(t.cuda())
    return tables


def prepare(case, seed):
    c = case
    g = _gen(seed * 1000003 + 29)
    dt = torch.float32 if c["f32"] else torch.bfloat16
    s = {"case": c}
    D, Hkv, page = c["D"], c["Hkv"], c["page"]
    if c["op"] in ("append", "read"):
        T = c["T"]
        pages = (T + page - 1) // page + 5
        _pages(s, g, pages)
        # tokens of many requests land anywhere; padded rows have no place
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].clone()
        if c["pad"]:
            slots[max(0, T - c["pad"]):] = -1
        s["slots"], s["pages"] = slots, pages
        if c["op"] == "append":
            Hq, R = c["Hq"], c["R"]
            qkv = _randn(g, T, (Hq + 2 * Hkv) * D, dtype=dt, std=1.5)
            s["q"] = qkv[:, :Hq * D].view(T, Hq, D)
            s["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
            s["v"] = qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D)
            s["wq"] = 1.0 + _randn(g, D, std=0.2)
            s["wk"] = 1.0 + _randn(g, D, std=0.2)
            s["pos"] = torch.randint(0, c["maxpos"], (T,), generator=g, device="cuda",
                                     dtype=torch.int32)
            # the rotation's table, its angles in 64 bits
            inv = ROPE_BASE ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) /
                                max(R, 1))
            ang = torch.arange(c["maxpos"], device="cuda", dtype=torch.float64)[:, None] * inv
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        return s
    lens = _attn_lens(c)
    q_cu = _offsets([q for q, _ in lens])
    kv = [q + p for q, p in lens]
    needs = [[(n + page - 1) // page for n in kv]]
    if c["op"] == "prefix":
        starts, Lp = _groups(c)
        needs.append([(n + page - 1) // page for n in Lp])
        s["cug"], s["plen"], s["Lp"] = _i32(starts), _i32(Lp), Lp
        s["starts"] = starts
    s["pages"] = sum(map(sum, needs)) + 3
    _pages(s, g, s["pages"])
    s["q"] = _randn(g, q_cu[-1], c["Hq"], D, dtype=dt)
    tables = _tables(g, needs, s["pages"])
    s["table"], s["maxp"] = tables[0], tables[0].shape[1]
    if c["op"] == "prefix":
        s["ptable"], s["maxpp"] = tables[1], tables[1].shape[1]
    s["cu"], s["kv"] = _i32(q_cu), _i32(kv)
    s["lens"], s["cu_host"] = lens, q_cu
    s["qmax"], s["kmax"] = max(q for q, _ in lens), max(kv)
    return s


# ---------------------------------------------------------------------------- plain forms

def _quantise(x):
    """(e4m3 numbers, exponents + 127) of the rows of x [..., D] in 32 bits."""
    m, e = torch.frexp(x.abs().amax(-1))  # largest = m 2^e with m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9)  # 448 = 0.875 2^9
    e = torch.where(m == 0, SCALE_LO, e).clamp(SCALE_LO, SCALE_HI)
    n = torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return n.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _value(numbers, scale):
    """What kept rows stand for, in 32 bits (scale None: rows that are kept as they are)."""
    x = numbers.float()
    return x if scale is None else torch.ldexp(x, (scale.int() - 127)[..., None])


def _rotate(x, cos, sin, R, interleaved):
    """Rotates the first R elements of x [T, H, D] by the angles of cos, sin [T, R / 2]."""
    if R == 0:
        return x
    cos, sin = cos[:, None], sin[:, None]
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
    return _rotate(y, cos, sin, c["R"], c["interleaved"])


def _plain_read(s, dt):
    ok = (s["slots"] >= 0)
    sl = s["slots"].clamp_min(0)
    pg, of = sl // s["case"]["page"], sl % s["case"]["page"]
    zero = torch.zeros((), device="cuda")
    return {n: torch.where(ok[:, None, None],
                           _value(s[n + "c"][pg, :, of], s[n + "s"][pg, :, of]), zero).to(dt)
            for n in "kv"}


def _plain_append(s):
    c = s["case"]
    pos = s["pos"].long()
    cos, sin = s["cos"][pos], s["sin"][pos]
    q = _plain_norm_rope(s["q"], s["wq"], cos, sin, c).to(s["q"].dtype)
    live = (s["slots"] >= 0).nonzero()[:, 0]
    sl = s["slots"][live]
    pg, of = sl // c["page"], sl % c["page"]
    for n, x in (("k", _plain_norm_rope(s["k"], s["wk"], cos, sin, c)), ("v", s["v"].float())):
        numbers, scale = _quantise(x[live])
        s[n + "c"].view(torch.uint8)[pg, :, of] = numbers.view(torch.uint8)
        s[n + "s"][pg, :, of] = scale
    return {"q": q, **_plain_read(s, torch.bfloat16)}


def _keys(s, table, n, most):
    """Keys and values of up to `most` tokens of each row of a block table, as [rows, Hkv, most,
    D] in 32 bits, and which of them there are, n [rows]."""
    page = s["case"]["page"]
    j = torch.arange(most, device="cuda")
    pg = table.long().gather(1, (j // page)[None].expand(table.shape[0], -1))
    of, there = (j % page)[None].expand_as(pg), j[None] < n[:, None]
    got = []
    for x in "kv":
        sc = s[x + "s"]
        y = _value(s[x + "c"][pg, :, of], None if sc is None else sc[pg, :, of])
        got.append(y.masked_fill_(~there[..., None, None], 0.0).transpose(1, 2))
    return got[0], got[1], there


def _plain_attn(s):
    """Attention of the padded batch: queries [N, Hkv, G, qmax, D] against keys [N, Hkv, L, D],
    a sequence's own ones and, in front of them, those of its group's prefix."""
    c = s["case"]
    G, D, N, Hkv, qm = c["Hq"] // c["Hkv"], c["D"], c["N"], c["Hkv"], s["qmax"]
    first, count = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(qm, device="cuda")
    there = i[None] < count[:, None]  # [N, qmax]
    rows = (first[:, None] + i).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(N, qm, Hkv, G, D).permute(0, 2, 3, 1, 4)
    K, V, key = _keys(s, s["table"], s["kv"], s["kmax"])
    j = torch.arange(s["kmax"], device="cuda")
    pos = (s["kv"] - count)[:, None] + i[None]  # [N, qmax]
    see = key[:, None] & (j <= pos[..., None])
    if c.get("window"):
        see &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    if c["op"] == "prefix":
        n = torch.arange(N, device="cuda")
        group = (n[:, None] >= s["cug"][None, 1:]).sum(1)
        Kp, Vp, kp = _keys(s, s["ptable"], s["plen"], max(max(s["Lp"]), 1))
        K, V = torch.cat([Kp[group], K], 2), torch.cat([Vp[group], V], 2)
        see = torch.cat([kp[group][:, None].expand(-1, qm, -1), see], 2)
    sc = torch.matmul(q.reshape(N, Hkv, G * qm, D), K.transpose(2, 3)).view(N, Hkv, G, qm, -1)
    sc *= D ** -0.5
    sc.masked_fill_(~see[:, None, None], float("-inf"))
    sc -= sc.amax(-1, keepdim=True)
    sc.exp_()
    total = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc.view(N, Hkv, G * qm, -1), V).view(N, Hkv, G, qm, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(N, qm, c["Hq"], D)
    return {"out": o[there].to(s["q"].dtype)}


# -------------------------------------------------------------------------- library calls

def _workspace(s, kda):
    """The scratch buffer that a program keeps for a call of these sizes."""
    c, n = s["case"], 0
    dt = kda.KDA_F32 if c["f32"] else kda.KDA_BF16
    if c["op"] == "attn":
        n = kda.kda_paged_attention_q8_fwd_workspace_size(
            c["N"], s["cu_host"][-1], c["Hq"], c["Hkv"], c["D"], dtype=dt)
    elif c["op"] == "prefix":
        n = kda.kda_paged_prefix_attention_fwd_workspace_size(
            c["groups"], c["N"], s["cu_host"][-1], c["Hq"], c["Hkv"], c["D"], dtype=dt)
    return torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")


def _own_read(s, kda, dt):
    c = s["case"]
    k = torch.empty(c["T"], c["Hkv"], c["D"], dtype=dt, device="cuda")
    v = torch.empty_like(k)
    kda.kda_paged_cache_read_q8(s["kc"], s["vc"], s["ks"], s["vs"], s["slots"], k, v, c["T"],
                                c["Hkv"], c["D"], s["pages"], c["page"])
    return {"k": k, "v": v}


def _own(s):
    import gated_delta_rule_55_gb300 as kda
    c = s["case"]
    if c["op"] == "read":
        return _own_read(s, kda, torch.float32 if c["f32"] else torch.bfloat16)
    if c["op"] == "append":
        q = torch.empty(c["T"], c["Hq"], c["D"], dtype=s["q"].dtype, device="cuda")
        kda.kda_qk_norm_rope_append_q8(
            s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], s["slots"], q,
            s["kc"], s["vc"], s["ks"], s["vs"], c["T"], c["Hq"], c["Hkv"], c["D"], c["R"],
            c["maxpos"], s["pages"], c["page"], eps=EPS_RMS, interleaved=c["interleaved"])
        return {"q": q, **_own_read(s, kda, torch.bfloat16)}
    if "ws" not in s:
        s["ws"] = _workspace(s, kda)
    T = s["cu_host"][-1]
    out = torch.empty(T, c["Hq"], c["D"], dtype=s["q"].dtype, device="cuda")
    if c["op"] == "attn":
        kda.kda_paged_attention_q8_fwd(
            s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv"], out, c["N"],
            T, c["Hq"], c["Hkv"], c["D"], s["pages"], c["page"], s["maxp"], window=c["window"],
            sinks=c["sinks"], workspace=s["ws"])
    else:
        kda.kda_paged_prefix_attention_fwd(
            s["q"], s["kc"], s["vc"], s["ptable"], s["plen"], s["cug"], s["table"], s["cu"],
            s["kv"], out, c["groups"], c["N"], T, c["Hq"], c["Hkv"], c["D"], s["pages"],
            c["page"], s["maxpp"], s["maxp"], k_scale=s["ks"], v_scale=s["vs"],
            workspace=s["ws"])
    return {"out": out}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "append":
        return _plain_append(state)
    if op == "read":
        return _plain_read(state, torch.float32 if state["case"]["f32"] else torch.bfloat16)
    return _plain_attn(state)


# ------------------------------------------------------------- the definitions in 64 bits

def _grid(x):
    """x [rows, D] in 64 bits, as the 8-bit rows stand for it: e4m3 has steps of an eighth of a
    power of two down to 2^-6, and of 2^-9 below; halves go to the even neighbour."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / E4M3_MAX)).clamp(SCALE_LO, SCALE_HI)
    e = torch.where((e > SCALE_LO) & (top <= E4M3_MAX * torch.exp2(e - 1)), e - 1, e)
    e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e).clamp(SCALE_LO, SCALE_HI)
    y = x * torch.exp2(-e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(y / step) * step * torch.exp2(e)


def _exact_rows(s, ids):
    """Keys and values of cache rows page * page_size + offset, [n, Hkv, D] in 64 bits."""
    page = s["case"]["page"]
    got = []
    for n in "kv":
        x = s[n + "c"][ids // page, :, ids % page].double()
        if s[n + "s"] is not None:
            x = x * torch.exp2(s[n + "s"][ids // page, :, ids % page].double() - 127)[..., None]
        got.append(x)
    return got


def _exact_append(s):
    c = s["case"]
    D, R, T = c["D"], c["R"], c["T"]
    mate, sign, ang = list(range(D)), [0.0] * D, [0] * D
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + R // 2)
        mate[a], mate[b], sign[a], sign[b], ang[a], ang[b] = b, a, -1.0, 1.0, i, i
    sign = torch.tensor(sign, dtype=torch.float64, device="cuda")
    if R:
        p = s["pos"].long()
        C = torch.where(sign != 0, s["cos"].double()[p][:, ang], 1.0)[:, None]
        Sn = (s["sin"].double()[p][:, ang] * sign)[:, None]
    else:
        C, Sn = 1.0, 0.0

    def turned(x, w):
        x = x.double()
        x = x * (x.square().mean(-1, keepdim=True) + EPS_RMS).pow(-0.5) * w.double()
        return x * C + x[..., mate] * Sn

    ok = (s["slots"] >= 0)[:, None, None]
    rows = {"k": turned(s["k"], s["wk"]), "v": s["v"].double()}
    out = {"q": turned(s["q"], s["wq"])}
    for n, x in rows.items():
        out[n] = torch.where(ok, _grid(x.reshape(-1, D)).view(T, c["Hkv"], D), 0.0)
    return out


def _exact_attn(s):
    c = s["case"]
    G, page = c["Hq"] // c["Hkv"], c["page"]
    out = torch.zeros(s["q"].shape[0], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    for n, (ql, p) in enumerate(s["lens"]):
        if ql == 0:
            continue
        a, kv = s["cu_host"][n], p + ql
        at = torch.arange(kv, device="cuda")
        K, V = _exact_rows(s, s["table"][n].long()[at // page] * page + at % page)
        gap = p + torch.arange(ql, device="cuda")[:, None] - at[None, :]
        see = gap >= 0
        if c.get("window", 0) > 0:
            see &= (gap < c["window"]) | (at[None, :] < c["sinks"])
        if c["op"] == "prefix":
            m = max(i for i in range(c["groups"]) if s["starts"][i] <= n)
            at = torch.arange(s["Lp"][m], device="cuda")
            Kp, Vp = _exact_rows(s, s["ptable"][m].long()[at // page] * page + at % page)
            K, V = torch.cat([Kp, K]), torch.cat([Vp, V])
            see = torch.cat([torch.ones(ql, len(at), dtype=torch.bool, device="cuda"), see], 1)
        for hq in range(c["Hq"]):
            x = s["q"][a:a + ql, hq].double() @ K[:, hq // G].T / math.sqrt(c["D"])
            x = torch.where(see, x, torch.full_like(x, -math.inf))
            out[a:a + ql, hq] = torch.softmax(x, -1) @ V[:, hq // G]
    return {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "read":
        ok = (s["slots"] >= 0)[:, None, None]
        return {n: torch.where(ok, x, 0.0)
                for n, x in zip("kv", _exact_rows(s, s["slots"].clamp_min(0)))}
    return _exact_attn(s)
