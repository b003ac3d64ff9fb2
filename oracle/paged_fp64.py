"""Plain fp64 forms of what surrounds attention in a serving or training loop:
the per-head norm and rotation of q and k with its gradient, a cache in pages,
and attention of new tokens over it.  NumPy, one row or one head at a time;
nothing here is tiled or shared with the CUDA side."""
import numpy as np


def rotate(y, pos, cos, sin, interleaved, transposed=False):
    """y [T, H, d]: pair i of token t turned by the angle (cos, sin)[pos[t], i]."""
    if cos is None:
        return y.copy()
    half = cos.shape[1]
    c, s = cos[pos].astype(np.float64)[:, None, :], sin[pos].astype(np.float64)[:, None, :]
    if transposed:
        s = -s
    a_at, b_at = (np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)) if interleaved else \
        (np.arange(half), np.arange(half, 2 * half))
    a, b = y[..., a_at], y[..., b_at]
    z = y.copy()
    z[..., a_at] = a * c - b * s
    z[..., b_at] = b * c + a * s
    return z


def norm_rope(x, w, eps, pos, cos, sin, interleaved):
    x = x.astype(np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
    return rotate(x, pos, cos, sin, interleaved)


def norm_rope_backward(x, dz, w, eps, pos, cos, sin, interleaved):
    """(dx, dw); dw None without norm."""
    x = x.astype(np.float64)
    dy = rotate(dz.astype(np.float64), pos, cos, sin, interleaved, transposed=True)
    if w is None:
        return dy, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh, g = x * r, dy * w.astype(np.float64)
    return r * (g - xh * (g * xh).mean(-1, keepdims=True)), (dy * xh).sum((0, 1))


def slots(table_row, L, page_size):
    """Slot of each of a sequence's L tokens in the flattened pool."""
    j = np.arange(L)
    return table_row[j // page_size].astype(np.int64) * page_size + j % page_size


def append(pool, rows, table, lens, cu, page_size):
    """`pool` [pages, page_size, H, d] with the new tokens' rows [T, H, d] in place."""
    out = pool.copy().reshape(-1, *pool.shape[2:])
    for b, L in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n:
            out[slots(table[b], L, page_size)[L - n:]] = rows[cu[b]:cu[b + 1]]
    return out.reshape(pool.shape)


def attention(q, k_pool, v_pool, table, lens, cu, page_size, scale, causal=True, window=None,
              slopes=None):
    """(O [T, Hq, d], LSE [Hq, T]) of each sequence's newest tokens over its
    pages; a row that sees no key has O = 0 and LSE = -inf, and rows of no
    sequence are NaN."""
    T, Hq, d = q.shape
    Hkv = k_pool.shape[2]
    kf, vf = k_pool.reshape(-1, Hkv, d), v_pool.reshape(-1, Hkv, d)
    O, lse = np.full((T, Hq, d), np.nan), np.full((Hq, T), np.nan)
    for b, L in enumerate(lens):
        n = int(cu[b + 1] - cu[b])
        if n == 0:
            continue
        at = slots(table[b], L, page_size)
        i, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
        seen = np.ones((n, L), bool)
        if causal:
            seen &= j <= i
        if window is not None and window >= 0:
            seen &= j >= i - window
        used = seen.any(0)
        rows = slice(cu[b], cu[b + 1])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            k, v = np.zeros((L, d)), np.zeros((L, d))
            k[used], v[used] = kf[at[used], g], vf[at[used], g]
            s = scale * (q[rows, h].astype(np.float64) @ k.T)
            if slopes is not None:
                s = s - float(slopes[h]) * (i - j)
            s = np.where(seen, s, -np.inf)
            m = s.max(1, keepdims=True, initial=-np.inf)
            p = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0)), 0.0)
            z = p.sum(1, keepdims=True)
            with np.errstate(divide="ignore"):
                lse[h, rows] = np.where(z > 0, m + np.log(z), -np.inf)[:, 0]
            O[rows, h] = p @ v / np.where(z > 0, z, 1)
    return O, lse
