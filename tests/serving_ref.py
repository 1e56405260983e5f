"""fp64 numpy definitions of the serving operators (plain loops over requests, tokens and
heads), shared by their tests."""
import numpy as np


def step(q, k, v, beta, decay, pool, slots, cu, scale=None, out_slots=None, l2norm=True,
         literal=False, out=None):
    """q, k [rows, Hk, dk], v [rows, Hv, dv]; returns (out, pool) of the packed requests."""
    rows, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    scale = dk ** -0.5 if scale is None else scale
    out = np.zeros((rows, Hv, dv)) if out is None else out.astype(np.float64)
    new = pool.astype(np.float64).copy()
    for n in range(len(cu) - 1):
        if not 0 <= slots[n] < len(pool):
            continue
        S = pool[slots[n]].astype(np.float64).copy()
        for t in range(cu[n], cu[n + 1]):
            for h in range(Hv):
                qh, kh = q[t, h * Hk // Hv], k[t, h * Hk // Hv]
                if l2norm:
                    qh = qh / np.sqrt((qh * qh).sum() + 1e-6)
                    kh = kh / np.sqrt((kh * kh).sum() + 1e-6)
                d = np.exp(decay[t, h]) if decay is not None else 1.0
                seen = S[h].T @ kh * (1.0 if literal else d)
                S[h] = d * S[h] + np.outer(kh, beta[t, h] * (v[t, h] - seen))
                out[t, h] = S[h].T @ (scale * qh)
        dst = slots[n] if out_slots is None else out_slots[n]
        if 0 <= dst < len(pool):
            new[dst] = S
    return out, new


def rotate(x, cos, sin, R, interleaved, sign=1.0):
    """x [T, H, D], cos / sin [T, R / 2]."""
    y = x.copy()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = cos[:, None, i], sign * sin[:, None, i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def norm_rope(x, w, cos, sin, R, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, cos, sin, R, interleaved)


def norm_rope_bwd(x, w, cos, sin, R, eps, interleaved, dy):
    """(dx, dw, |terms of dw| summed)."""
    g = rotate(dy, cos, sin, R, interleaved, -1.0)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dx = r * (g * w - x * r * r * (g * w * x).mean(-1, keepdims=True))
    return dx, (g * x * r).sum((0, 1)), np.abs(g * x * r).sum((0, 1))


def key_rows(cache, table_row, n, page):
    """The first n keys of a sequence: [n, Hkv, D]."""
    Hkv, D = cache.shape[1], cache.shape[3]
    out = np.zeros((n, Hkv, D))
    for j in range(n):
        out[j] = cache[table_row[j // page], :, j % page]
    return out


def paged_attention(q, kc, vc, table, cu, kv_lens, page, scale=None, window=0, sinks=0):
    """q [T, Hq, D], caches [pages, Hkv, page, D].  Returns out, lse, A = sum p |v| and
    Z = the largest sum |q_d k_d| scale of a row (the scale of its scores' rounding)."""
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    A, Z = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for n in range(len(cu) - 1):
        L, kv = cu[n + 1] - cu[n], kv_lens[n]
        if L == 0:
            continue
        K, V = key_rows(kc, table[n], kv, page), key_rows(vc, table[n], kv, page)
        for i in range(L):
            pos = kv - L + i
            if pos < 0:
                continue
            see = np.zeros(kv, bool)
            lo = 0 if window == 0 else max(0, pos - window + 1)
            see[lo:pos + 1] = True
            if window:
                see[:min(sinks, pos + 1)] = True
            idx = np.nonzero(see)[0]
            for h in range(Hq):
                kh, vh = K[idx, h // (Hq // Hkv)], V[idx, h // (Hq // Hkv)]
                s = kh @ q[cu[n] + i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[cu[n] + i, h] = p @ vh / l
                A[cu[n] + i, h] = p @ np.abs(vh) / l
                lse[cu[n] + i, h] = m + np.log(l)
                Z[cu[n] + i, h] = (np.abs(kh) @ np.abs(q[cu[n] + i, h])).max() * scale
    return out, lse, A, Z
