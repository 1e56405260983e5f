"""fp64 numpy definitions of 8-bit cache rows and of attention behind shared prefixes, for the
tests."""
import numpy as np

LO, HI = -110, 119
# what each byte of e4m3 stands for (127 and 255: NaN)
E4M3 = np.array([(-1.0 if b & 128 else 1.0) *
                 ((b & 7) * 2.0 ** -9 if b & 120 == 0 else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10))
                 for b in range(256)])
E4M3[[127, 255]] = np.nan


def exponents(y):
    """The scale's exponent of each row of y [..., D]."""
    top = np.abs(y).max(-1)
    e = np.full(top.shape, LO)
    for x in range(LO, HI):
        e[top > 448 * 2.0 ** x] = x + 1
    return e


def quantise(y):
    """(bytes of e4m3, scale bytes) of rows y [..., D] in 64 bits; halves go to the even number."""
    odd = ~np.isfinite(y).all(-1)
    y = np.where(odd[..., None], 0.0, y)
    e = exponents(y)
    x = np.clip(y * 2.0 ** -e[..., None].astype(float), -448, 448)
    m = np.abs(x)
    step = 2.0 ** (np.floor(np.log2(np.maximum(m, 2.0 ** -6))) - 3)
    m = np.round(m / step) * step  # (numpy rounds halves to even)
    b = np.searchsorted(E4M3[:127], m)
    assert (E4M3[b] == m).all()
    b = np.where(np.signbit(x), b | 128, b).astype(np.uint8)
    return b, np.where(odd, 255, e + 127).astype(np.uint8)


def value(numbers, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(float) - 127))
    return E4M3[numbers] * s[..., None]


def rows_of(cache, table_row, n, page):
    j = np.arange(n)
    return cache[np.asarray(table_row)[j // page], :, j % page]


def prefix_attention(q, kc, vc, ptable, plens, groups, table, cu, kv_lens, page, scale=None):
    """q [T, Hq, D]; sequences groups[g] .. groups[g + 1] - 1 see prefix g.  Returns out, lse, A and Z
    as serving_ref.paged_attention does."""
    T, Hq, D = q.shape
    Hkv = kc.shape[1]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    A, Z = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for n in range(len(cu) - 1):
        L, kv = cu[n + 1] - cu[n], kv_lens[n]
        if L == 0:
            continue
        K, V, P = rows_of(kc, table[n], kv, page), rows_of(vc, table[n], kv, page), 0
        for g in range(len(groups) - 1):
            if groups[g] <= n < groups[g + 1]:
                P = plens[g]
                K = np.concatenate([rows_of(kc, ptable[g], P, page), K])
                V = np.concatenate([rows_of(vc, ptable[g], P, page), V])
        for i in range(L):
            top = P + max(kv - L + i + 1, 0)
            if top == 0:
                continue
            t = cu[n] + i
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                k, v = K[:top, h], V[:top, h]
                s = q[t, hs] @ k.T * scale
                m = s.max(1)
                p = np.exp(s - m[:, None])
                l = p.sum(1)
                out[t, hs] = p @ v / l[:, None]
                A[t, hs] = p @ np.abs(v) / l[:, None]
                lse[t, hs] = m + np.log(l)
                Z[t, hs] = (np.abs(q[t, hs]) @ np.abs(k).T).max(1) * scale
    return out, lse, A, Z
