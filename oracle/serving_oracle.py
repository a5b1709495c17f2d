"""fp64 definitions of rotary positions, the paged cache and attention of one
new token (NumPy; scalar loops over tokens and pages, nothing shared with the
package)."""
import math

import numpy as np

E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100


def rope(x, positions, inv_freq, axes=None, pairs="half", inverse=False):
    """x [T, H, D]; positions [T] or [n_axes, T] (integers); inv_freq [rot/2].
    Pair i of token t turns by positions[axes[i]][t] * inv_freq[i]."""
    x = np.asarray(x, np.float64)
    pos = np.asarray(positions, np.float64)
    pos = pos[None] if pos.ndim == 1 else pos
    half = len(inv_freq)
    y = x.copy()
    for i in range(half):
        a = pos[0 if axes is None else int(axes[i])] * float(inv_freq[i])
        c, s = np.cos(a)[:, None], np.sin(a)[:, None] * (-1.0 if inverse else 1.0)
        u, v = (i, i + half) if pairs == "half" else (2 * i, 2 * i + 1)
        y[..., u] = x[..., u] * c - x[..., v] * s
        y[..., v] = x[..., u] * s + x[..., v] * c
    return y


def e4m3(x):
    """Nearest e4m3 value (ties to even, largest 448) of each element."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)          # 3 fraction bits; subnormals from 2^-6 down
    return np.sign(x) * np.minimum(np.round(a / step) * step, E4M3_MAX)   # np.round: ties to even


def quantise(rows):
    """(codes, scale) of rows [..., D]: scale = max(max|x|, 2^-100) / 448,
    codes = e4m3(x / scale); unrounded scale."""
    scale = np.maximum(np.max(np.abs(rows), axis=-1), MIN_AMAX) / E4M3_MAX
    return e4m3(rows / scale[..., None]), scale


def place(page_table, page_size, b, p):
    """(page, slot) of position p of sequence b."""
    return int(page_table[b][p // page_size]), p % page_size


def cache_rows(cache, page_table, b, n, first=0):
    """Rows [n, H, D] of positions first ... first + n - 1 of sequence b."""
    out = np.empty((n, cache.shape[1]) + cache.shape[3:], cache.dtype)
    for i in range(n):
        pg, sl = place(page_table, cache.shape[2], b, first + i)
        out[i] = cache[pg, :, sl]
    return out


def decode(q, k, v, scale=None):
    """q [H_q, D], k, v [n, H_kv, D] -> (o [H_q, D], lse [H_q]); no keys: 0, -inf."""
    Hq, D = q.shape
    o, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if len(k) == 0:
        return o, lse
    G = Hq // k.shape[1]
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    for h in range(Hq):
        s = sc * (k[:, h // G] @ q[h])
        m = s.max()
        e = np.exp(s - m)
        lse[h] = m + math.log(e.sum())
        o[h] = (e / e.sum()) @ v[:, h // G]
    return o, lse
