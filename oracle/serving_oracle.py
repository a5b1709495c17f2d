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


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E2M1_BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)      # half way between neighbours: to the even code


def e2m1(z):
    """Codes 0-15 (bit 3 the sign) of the nearest e2m1 values, ties to the even
    code, at most 6."""
    a = np.abs(np.asarray(z, np.float64))
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(E2M1_BORDERS):
        code += (a >= m) if i % 2 else (a > m)               # up to code i + 1: even where i is odd
    return code + 8 * np.signbit(z)


def quantise4(rows):
    """(codes [..., D], block scales [..., D/16], row scale [...]) of rows
    [..., D] in 4 bits: scale the least power of two with max(max|x|, 2^-100) <=
    2688 scale, block scales e4m3(max|x / scale| / 6), codes e2m1(x / scale /
    block scale), 0 where that is 0."""
    rows = np.asarray(rows, np.float64)
    part, e = np.frexp(np.maximum(np.max(np.abs(rows), -1), MIN_AMAX) / 2688.0)
    scale = np.ldexp(1.0, e - (part == 0.5))
    y = (rows / scale[..., None]).reshape(rows.shape[:-1] + (-1, 16))
    block = e4m3(np.max(np.abs(y), -1) / 6.0)
    z = np.where(block[..., None] > 0, y / np.where(block > 0, block, 1.0)[..., None], 0.0)
    return e2m1(z).reshape(rows.shape), block, scale


def values4(codes, block, scale):
    """Rows from codes, block scales and row scales."""
    c = np.asarray(codes)
    v = np.array(E2M1)[c & 7] * np.where(c & 8, -1.0, 1.0)
    return v * np.repeat(block, 16, -1) * np.asarray(scale)[..., None]


def attention_weights(q, k, scale=None):
    """What each key gathers from one new token: [n, H_kv], sums over the query
    heads of each kv head; no keys, or none of weight: 0."""
    Hq, D = q.shape
    n, H = k.shape[:2]
    w = np.zeros((n, H))
    sc = 1.0 / math.sqrt(D) if scale is None else scale
    for h in range(Hq if n else 0):
        s = sc * (k[:, h // (Hq // H)] @ q[h])
        e = np.exp(s - s.max())
        w[:, h // (Hq // H)] += e / e.sum()
    return w


def stays(weights, keep, recent):
    """The positions of one sequence's head that an eviction keeps, rising:
    weights [n]; keep < 0: all."""
    n = len(weights)
    m = n if keep < 0 else min(n, keep)
    if m == n:
        return list(range(n))
    r = min(m, recent)
    # by falling weight (NaN first), then by rising position
    order = sorted(range(n - r), key=lambda i: (not math.isnan(weights[i]), -weights[i] if not math.isnan(weights[i]) else 0.0, i))
    return sorted(order[:m - r]) + list(range(n - r, n))
