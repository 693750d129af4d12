"""Plain 64-bit forms of the paged-cache operators (numpy), and small cases for them."""
import numpy as np


def rotate(x, pos, n_rot, base, layout, axis=None, scale=1.0, factors=None, magnitude=1.0):
    """x (n_tok, heads, D) float64; pos (n_axes, n_tok); layout 0 adjacent pairs, 1 halves."""
    y = x.astype(np.float64).copy()
    for i in range(n_rot // 2):
        f = scale * base ** (-2.0 * i / n_rot) / (1.0 if factors is None else float(np.float32(factors[i])))
        t = pos[0 if axis is None else axis[i]].astype(np.float64) * f
        c, s = magnitude * np.cos(t)[:, None], magnitude * np.sin(t)[:, None]
        a, b = (i, i + n_rot // 2) if layout == 1 else (2 * i, 2 * i + 1)
        xa, xb = x[:, :, a].astype(np.float64), x[:, :, b].astype(np.float64)
        y[:, :, a] = xa * c - xb * s
        y[:, :, b] = xa * s + xb * c
    return y


def attention(q, k, v, pos, first, prefix, window, scale, cap, slopes):
    """One sequence: q (n, H, D), k and v (len, K, D), pos and first (n): (out, bound) in float64.
    bound: the largest |v| seen times (1 + the largest sum |q_i k_i| scale), per row."""
    n, H, D = q.shape
    ln, K = k.shape[:2]
    out = np.zeros((n, H, D))
    size = np.zeros((n, H, 1))
    j = np.arange(ln)
    for t in range(n):
        seen = (j >= first[t]) & ((j < prefix) | ((j <= pos[t]) & ((window == 0) | (pos[t] - j < window))))
        idx = np.nonzero(seen)[0]
        if idx.size == 0:
            continue
        for h in range(H):
            kk, vv = k[idx, h // (H // K)].astype(np.float64), v[idx, h // (H // K)].astype(np.float64)
            qq = q[t, h].astype(np.float64)
            s = kk @ qq * scale
            if cap > 0:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - float(slopes[h]) * np.abs(pos[t] - idx)
            p = np.exp(s - s.max())
            out[t, h] = p @ vv / p.sum()
            size[t, h] = np.abs(vv).max() * (1 + (np.abs(kk) @ np.abs(qq)).max() * scale
                                             + (0 if slopes is None else float(slopes[h]) * np.abs(pos[t] - idx).max()))
    return out, size
