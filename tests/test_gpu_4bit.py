"""The 4-bit cache: rows written and read (ulysses_cache_write / _read with
ULYSSES_E2M1) and attention over it, against the fp64 definitions.

Codes and scales are compared whole: every step of their definition (a power of
two, quotients rounded to nearest) is exact in fp32 for bf16 rows, whose borders
no quotient misses.  An fp32 quotient may land on a border that it lies 2^-24
beside, so fp32 elements within 2^-22 of one are left out.

Bound of attention, with e = 2^-24 (the matrix pipe cuts sums instead of
rounding them: 2 e), keys' weights p_j and row scales r_j:
  ds = 2 (D + 4) e scale sum |q_d k_jd| + scale 2^-39 max|q| sum_d |k_jd|   (q in f16, scaled to its top)
  |do| <= (2 ds + 2 (n + 16) e + 2^-20) sum_j p_j |v_j|     (weights: two f16 parts 2^-22, log2 of r_j and exp2)
          + n 2^-32 2688 max_j(p_j r_j)                     (f16's smallest step under the largest weight, 2^7)
          + half a step of the output's type
FP32 queries: products of 11-bit parts, 2^-21 of each and u = 2^-21 of the
weights; SIMT: neither.  LSE: ds + (n + 16) e + 2 e |lse|."""
import math

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
E = 2.0 ** -24


def f64(t):
    return t.detach().float().double().cpu().numpy()


def unpack(cache, page, D):
    """(codes [P, H, page, D], block scales [P, H, page, D/16]) of a 4-bit cache."""
    raw = cache.cpu().numpy().reshape(*cache.shape[:2], -1)
    c = raw[..., :page * D // 2].reshape(*cache.shape[:2], page, D // 2)
    codes = np.stack((c & 15, c >> 4), -1).reshape(*cache.shape[:2], page, D)
    b = raw[..., page * D // 2:].reshape(*cache.shape[:2], page, D // 16)
    return codes.astype(np.int64), f64(torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn))


def pack(codes, block):
    """The other way round."""
    P, H, page, D = codes.shape
    c = (codes[..., ::2] | codes[..., 1::2] << 4).astype(np.uint8).reshape(P, H, -1)
    b = torch.from_numpy(block).to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(P, H, -1)
    return torch.from_numpy(np.concatenate((c, b), -1).reshape(P, H, page, 9 * D // 16))


def same_codes(a, b):
    """Element by element; a code of magnitude 0 may have either sign."""
    return (a == b) | (((a | b) & 7) == 0)


def rows_in(shape, dtype, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[-1:], generator=g)) * gain).to(DT[dtype])


def place(tab, page, b, p):
    return int(tab[b][p // page]), p % page


WRITES = [  # new tokens, tokens before, H, D, page, dtype, layout
    ([1], [0], 1, 128, 16, "bf16", "seq"),
    ([37], [5], 2, 64, 16, "bf16", "head"),
    ([37], [5], 2, 128, 48, "fp32", "head"),
    ([0, 20, 1, 0, 65], [7, 15, 31, 0, 100], 3, 128, 64, "bf16", "seq"),
    ([0, 20, 1, 0, 65], [7, 15, 31, 0, 100], 8, 64, 32, "fp32", "seq"),
    ([700, 333], [1, 0], 8, 128, 256, "bf16", "head"),
    ([4097], [63], 4, 64, 64, "bf16", "seq"),
]


@pytest.mark.parametrize("new,before,H,D,page,dtype,layout", WRITES)
def test_write_and_read(new, before, H, D, page, dtype, layout):
    T, B = sum(new), len(new)
    lens = [a + b for a, b in zip(new, before)]
    per = [-(-n // page) for n in lens]
    total = sum(per) + 2
    order = np.random.default_rng(3).permutation(total)
    tab = np.full((B, max(per) + 1), 1 << 30, np.int32)
    at = 0
    for b in range(B):
        tab[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    # K and V as slices of one fused tensor
    x = rows_in((T, 2 * H + 1, D), dtype, 7)
    if layout == "head":
        x = x.transpose(0, 1).contiguous()
    xd = x.cuda()
    k, v = (xd[:, 1:1 + H], xd[:, 1 + H:]) if layout == "seq" else (xd[1:1 + H], xd[1 + H:])
    kc, vc, ks, vs = U.kv_cache(total, page, H, D, torch.uint8)
    assert kc.shape == (total, H, page, 9 * D // 16) and ks.shape == (total, H, page)
    for t in (kc, vc):
        t.fill_(0xA5)
    w = U.cache_weights(kc).fill_(3.0)
    cu = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    U.cache_write(k, v, kc, vc, i32(tab), i32(lens), cu_new=i32(cu), k_scale=ks, v_scale=vs, layout=layout, weights=w)
    U.check()
    written = np.zeros((total, page), bool)
    for name, src, cache, scale in (("k", k, kc, ks), ("v", v, vc, vs)):
        rows = f64(src if layout == "seq" else src.transpose(0, 1))
        codes, block, sc = so.quantise4(rows)
        got_c, got_b = unpack(cache, page, D)
        got_s = f64(scale)
        for b in range(B):
            for i in range(new[b]):
                pg, sl = place(tab, page, b, before[b] + i)
                written[pg, sl] = True
                t = cu[b] + i
                assert np.array_equal(got_s[pg, :, sl], sc[t]), (name, b, i)
                assert np.array_equal(got_b[pg, :, sl], block[t]), (name, b, i)
                ok = same_codes(got_c[pg, :, sl], codes[t])
                if dtype == "fp32":
                    z = np.abs(rows[t] / sc[t][:, None] / np.repeat(np.where(block[t] > 0, block[t], 1), 16, -1))
                    ok |= np.min(np.abs(z[..., None] / np.array(so.E2M1_BORDERS) - 1), -1) < 2.0 ** -22
                assert ok.all(), (name, b, i)
        # nothing else was touched
        assert np.all(got_c[~written.repeat(H, 0).reshape(total, H, page)] == np.tile([5, 10], D // 2))
    left = torch.from_numpy(written).cuda()
    assert torch.equal(w, torch.where(left, 0.0, 3.0)[:, None].expand_as(w))
    # back again: a value has few bits, so both types hold it exactly
    first = i32(before)
    for out in ("bf16", "fp32"):
        rk, rv = U.cache_read(kc, vc, i32(tab), i32(cu), T, first=first, k_scale=ks, v_scale=vs, dtype=DT[out], layout=layout)
        for cache, scale, r in ((kc, ks, rk), (vc, vs, rv)):
            want = so.values4(*unpack(cache, page, D), f64(scale))
            got = f64(r if layout == "seq" else r.transpose(0, 1))
            for b in range(B):
                for i in range(new[b]):
                    pg, sl = place(tab, page, b, before[b] + i)
                    assert np.array_equal(got[cu[b] + i], want[pg, :, sl])
    U.check()


def one_row(x, D=64):
    """codes, block scales, scale and the row read back of one row."""
    kc, vc, ks, vs = U.kv_cache(1, 16, 1, D, torch.uint8)
    t = torch.tensor(x, dtype=torch.float32).view(1, 1, D).cuda()
    tab, one = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    U.cache_write(t, t, kc, vc, tab, one, k_scale=ks, v_scale=vs)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    r, _ = U.cache_read(kc, vc, tab, cu, 1, k_scale=ks, v_scale=vs, dtype=torch.float32)
    U.check()
    c, b = unpack(kc, 16, D)
    return c[0, 0, 0], b[0, 0, 0], float(ks[0, 0, 0]), f64(r)[0, 0]


def test_rows_at_the_edges():
    # every border, both signs, under a block scale of 448 and a row scale of 1
    z = np.zeros(64)
    z[:7], z[7:14], z[15] = so.E2M1_BORDERS, [-m for m in so.E2M1_BORDERS], 6.0
    c, b, s, r = one_row(z * 448.0)
    assert s == 1.0 and b[0] == 448.0 and list(b[1:]) == [0, 0, 0]
    want = [0, 2, 2, 4, 4, 6, 6]
    assert list(c[:7]) == want and same_codes(c[7:14], np.array([8 + x for x in want])).all()
    assert c[15] == 7 and not c[16:].any()
    assert r[15] == 2688.0 and r[12] == -1792.0
    # zeros; the smallest numbers; blocks far below the row's largest
    c, b, s, r = one_row(np.zeros(64))
    assert not c.any() and not b.any() and s == 2.0 ** -111 and not r.any()
    for x in (1e-45, 1e-38, 2.0 ** -100, 2.0 ** -99):
        row = np.zeros(64)
        row[5], row[20] = x, -x
        codes, block, scale = so.quantise4(np.float64(np.float32(row))[None])
        c, b, s, r = one_row(row)
        assert np.array_equal(c & 7, codes[0] & 7) and np.array_equal(b, block[0]) and s == scale[0], x
    row = np.zeros(64)
    row[0], row[16], row[32], row[48] = 2688.0, 6 * 2.0 ** -9, 3 * 2.0 ** -9, 6 * 2.0 ** -9 * 1.5
    c, b, s, _ = one_row(row)
    assert s == 1.0 and list(b) == [448.0, 2.0 ** -9, 0.0, 2.0 ** -8] and c[16] == 7 and c[32] == 0
    # the largest, and what is no number
    for big in (3.4028234663852886e38, -3.4028234663852886e38, 2.0 ** 127):
        row = np.linspace(-1, 1, 64) * abs(big) * 0.99
        row[3] = big
        codes, block, scale = so.quantise4(np.float64(np.float32(row))[None])
        c, b, s, r = one_row(row)
        assert same_codes(c, codes[0]).all() and np.array_equal(b, block[0]) and s == scale[0]
        assert big != 2.0 ** 127 or np.isfinite(r).all()
    for bad in (math.inf, -math.inf, math.nan):
        row = np.ones(64)
        row[17] = bad
        _, _, s, r = one_row(row)
        assert math.isnan(s) and np.isnan(r).all()


def build4(lens, Hq, H, D, page, dtype, layout, seed=0, gain=1.0, slack=2):
    """Random 4-bit cache in pages of a mixed order; slots that no sequence owns
    hold NaN scales, unused table entries a wild id."""
    rng = np.random.default_rng(seed)
    per = [-(-n // page) for n in lens]
    total = sum(per) + slack
    order = rng.permutation(total)
    tab = np.full((len(lens), max(per) + 1), 1 << 30, np.int32)
    own = np.zeros((total, page), bool)
    at = 0
    for b, n in enumerate(lens):
        for i in range(per[b]):
            p = int(order[at])
            at += 1
            tab[b, i] = p
            own[p, :min(page, n - i * page)] = True
    bufs = []
    for _ in range(2):
        x = rng.standard_normal((total, H, page, D)) * np.exp(rng.standard_normal((total, H, page, 1))) * gain
        codes, block, scale = so.quantise4(x)
        vals = so.values4(codes, block, scale)
        off = ~np.broadcast_to(own[:, None], scale.shape)
        raw = pack(codes, block)
        scale = torch.from_numpy(scale).float()
        scale[torch.from_numpy(off)] = float("nan")
        c = raw.cuda()
        bufs.append((c, scale.cuda(), vals))
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((len(lens), Hq, D), generator=g) * 2).to(DT[dtype])
    rows = [(f64(q[b]), *(so.cache_rows(bufs[i][2], tab, b, n) for i in range(2))) for b, n in enumerate(lens)]
    scales = [so.cache_rows(f64(bufs[1][1])[..., None], tab, b, n)[..., 0] for b, n in enumerate(lens)]
    qd = (q if layout == "seq" else q.transpose(0, 1)).contiguous().cuda()
    return dict(q=qd, k_cache=bufs[0][0], v_cache=bufs[1][0], page_table=torch.from_numpy(tab).cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_scale=bufs[0][1], v_scale=bufs[1][1],
                layout=layout), rows, scales


def widen(args, positions=1 << 20):
    """A table of room for many more positions: the keys are split over the launch."""
    tab = args["page_table"]
    wide = torch.full((tab.shape[0], max(tab.shape[1], positions // args["k_cache"].shape[2])), -5, dtype=torch.int32,
                      device="cuda")
    wide[:, :tab.shape[1]] = tab
    return {**args, "page_table": wide}


def check4(o, lse, rows, scales, dtype, layout, simt=False, scale=None):
    o = f64(o)
    o = o if layout == "seq" else o.transpose(1, 0, 2)
    lse = f64(lse)
    for b, (q, k, v) in enumerate(rows):
        Hq, D = q.shape
        n, sc = len(k), 1.0 / math.sqrt(D) if scale is None else scale
        ro, rl = so.decode(q, k, v, scale)
        if n == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        G = Hq // k.shape[1]
        for h in range(Hq):
            K, V = k[:, h // G], v[:, h // G]
            ds = sc * 2 * (D + 4) * E * (np.abs(K) @ np.abs(q[h])).max()
            u = 2.0 ** -20 if dtype == "bf16" and not simt else 2.0 ** -21 if not simt else 0.0
            if dtype == "bf16" and not simt:
                ds += sc * 2.0 ** -39 * np.abs(q[h]).max() * np.abs(K).sum(-1).max()
            elif not simt:
                ds += sc * 2.0 ** -21 * (np.abs(K) @ np.abs(q[h])).max()
            p = np.exp(sc * (K @ q[h]) - rl[h])
            lim = (2 * ds + 2 * (n + 16) * E + u) * (p @ np.abs(V))
            if dtype == "bf16" and not simt:
                lim = lim + n * 2.0 ** -32 * 2688 * (p * scales[b][:, h // G]).max()
            lim = lim + np.abs(ro[h]) * (2.0 ** -8 if dtype == "bf16" else E) * 1.01 + 1e-37
            err = np.abs(o[b, h] - ro[h])
            assert np.all(err <= lim), (b, h, n, float((err / lim).max()))
            assert abs(lse[b, h] - rl[h]) <= ds + (n + 16) * E + 2 * E * abs(rl[h]), (b, h, lse[b, h], rl[h])


DECODES = [  # lens, Hq, H, D, page, dtype, layout
    ([1], 1, 1, 128, 16, "bf16", "seq"),
    ([0], 4, 1, 64, 16, "bf16", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 128, 16, "bf16", "head"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 64, 32, "bf16", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 2, 2, 128, 16, "fp32", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 64, 32, "fp32", "head"),
    ([777, 3], 32, 8, 128, 48, "bf16", "head"),
    ([300, 20], 5, 1, 64, 16, "bf16", "seq"),
    ([513, 127], 16, 1, 128, 128, "bf16", "head"),
    ([513, 127], 12, 2, 128, 64, "bf16", "seq"),
    ([513, 127], 16, 2, 64, 128, "bf16", "head"),
    ([200, 90], 20, 1, 64, 16, "bf16", "seq"),
    ([1200, 64, 0, 65], 6, 2, 64, 64, "fp32", "seq"),
    ([1200, 64, 0, 65], 16, 1, 128, 256, "fp32", "seq"),
    ([2500], 8, 2, 128, 64, "bf16", "head"),
    ([1025, 1, 0, 1040], 32, 8, 64, 16, "bf16", "seq"),           # eight warps a CTA, of four CTAs
    ([2047, 1031], 32, 2, 128, 64, "bf16", "head"),
    ([8100], 12, 2, 64, 16, "bf16", "seq"),
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", range(len(DECODES)))
def test_decode(case, wide):
    lens, Hq, H, D, page, dtype, layout = DECODES[case]
    args, rows, scales = build4(lens, Hq, H, D, page, dtype, layout, seed=case)
    if wide:
        args = widen(args)
    o, lse = U.attn_decode(**args)
    U.check()
    check4(o, lse, rows, scales, dtype, layout)
    again = U.attn_decode(**args)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("case", [3, 4, 5, 6, 7, 11])
def test_decode_simt(case):
    lens, Hq, H, D, page, dtype, layout = DECODES[case]
    args, rows, scales = build4(lens, Hq, H, D, page, dtype, layout, seed=50 + case)
    U.set_kernel(U.KERNEL_SIMT)
    try:
        for a in (args, widen(args)):
            o, lse = U.attn_decode(scale=0.11, **a)
            U.check()
            check4(o, lse, rows, scales, dtype, layout, simt=True, scale=0.11)
    finally:
        U.set_kernel(U.KERNEL_AUTO)


@pytest.mark.parametrize("gain", [2.0 ** -60, 2.0 ** 20])
def test_decode_of_far_scales(gain):
    """Row scales of any size, V's far below and above 1, and rows of zeros."""
    args, rows, scales = build4([600, 40], 8, 2, 128, 64, "bf16", "seq", seed=77)
    args["v_scale"] = args["v_scale"] * gain
    rows = [(q, k, v * gain) for q, k, v in rows]
    o, lse = U.attn_decode(**args)
    U.check()
    check4(o, lse, rows, [s * gain for s in scales], "bf16", "seq")


def test_a_row_of_nan_poisons_its_sequence_alone():
    args, rows, _ = build4([100, 50], 4, 1, 128, 16, "bf16", "seq", seed=5)
    pg, sl = place(args["page_table"].cpu().numpy(), 16, 0, 33)
    args["k_scale"][pg, 0, sl] = float("nan")
    o, lse = U.attn_decode(**args)
    assert bool(o[0].isnan().all()) and bool(lse[0].isnan().all())
    assert bool(o[1].isfinite().all()) and bool(lse[1].isfinite().all())
