"""Single-token attention where its weights, its values and its joins are
extreme, against the fp64 definition.

Bound of an e4m3 cache with bf16 queries, tighter than test_gpu_decode's.  A
weight (softmax weight times V's scale, at most 2^15 in f16 and at least 2^7
for the largest of a piece) goes in as an f16 value and the f16 rest: 2^-22 of
it, and half of f16's smallest step, 2^-25, which is 2^-32 of the largest:
  sum_j 2^-32 max_i(p_i scale_i) |code_jd|.
Queries have their largest element at 2^14 to 2^15 in f16, where bf16's eight
bits are exact down to 2^-31 of it and the smallest step's half is 2^-39 of it:
a score is off by scale 2^-39 max|q| sum |k_d|.
The rest is test_gpu_decode's: ds = (D + 4) e scale sum |q k|, e = 2^-24,
|do| <= (2 max ds + (n + 16) e + 2^-22) sum p |v| + the above + half a step of
the output."""
import math

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so
from tests.test_gpu_decode import CASES, DT, E, build, check, f64, widen

pytestmark = pytest.mark.gpu


def rows_of(args):
    """q, k, v of each sequence in fp64, and V's scales and codes, from the call's own tensors."""
    tab = args["page_table"].cpu().numpy()
    q = f64(args["q"])
    q = q if args["layout"] == "seq" else q.transpose(1, 0, 2)
    out = []
    for b, n in enumerate(args["seq_lens"].tolist()):
        got = []
        for c, s in ((args["k_cache"], args["k_scale"]), (args["v_cache"], args["v_scale"])):
            r = so.cache_rows(f64(c), tab, b, n)
            w = so.cache_rows(f64(s)[..., None], tab, b, n)
            got.append((r * w, w[..., 0], r))
        out.append((q[b], got[0][0], got[1][0], got[1][1], got[1][2]))
    return out


def check_e4m3(o, lse, args):
    o = f64(o)
    o = o if args["layout"] == "seq" else o.transpose(1, 0, 2)
    lse = f64(lse)
    for b, (q, k, v, sv, cv) in enumerate(rows_of(args)):
        Hq, D = q.shape
        n, sc = len(k), 1.0 / math.sqrt(D)
        ro, rl = so.decode(q, k, v)
        if n == 0:
            assert np.all(o[b] == 0) and np.all(np.isneginf(lse[b]))
            continue
        G = Hq // k.shape[1]
        for h in range(Hq):
            K, V = k[:, h // G], v[:, h // G]
            ds = sc * ((D + 4) * E * (np.abs(K) @ np.abs(q[h])).max()
                       + 2.0 ** -39 * np.abs(q[h]).max() * np.abs(K).sum(-1).max())
            p = np.exp(sc * (K @ q[h]) - rl[h])
            lim = (2 * ds + (n + 16) * E + 2.0 ** -22) * (p @ np.abs(V))
            lim = lim + 2.0 ** -32 * (p * sv[:, h // G]).max() * np.abs(cv[:, h // G]).sum(0)
            lim = lim + np.abs(ro[h]) * 2.0 ** -8 * 1.01 + 1e-37
            err = np.abs(o[b, h] - ro[h])
            assert np.all(err <= lim), (b, h, n, float((err / lim).max()))
            assert abs(lse[b, h] - rl[h]) <= ds + (n + 16) * E + 2 * E * abs(rl[h]), (b, h, lse[b, h], rl[h])


# ------------------------------------------------------------------ e4m3 weights

@pytest.mark.parametrize("lens,Hq,Hkv,D,page,dtype,cache,layout",
                         [c for c in CASES if c[5:7] == ("bf16", "e4m3")])
def test_e4m3_weights_keep_more_than_f16(lens, Hq, Hkv, D, page, dtype, cache, layout):
    args, _ = build(lens, Hq, Hkv, D, page, dtype, cache, layout, seed=20)
    for x in (args, widen(args)):
        o, lse = U.attn_decode(**x)
        U.check()
        check_e4m3(o, lse, x)


@pytest.mark.parametrize("above", [10.0, 15.0, 18.0])
@pytest.mark.parametrize("D,Hq", [(128, 8), (128, 16), (64, 24)])
@pytest.mark.parametrize("how", ["cluster", "split"])
def test_one_key_far_above_the_others(above, D, Hq, how):
    """One key's score `above` nats over the others', its V row zero: the output
    is the others' alone, weights of e^-above beside it."""
    n = 700
    args, _ = build([n], Hq, 2, D, 16, "bf16", "e4m3", "seq", seed=21)
    tab = args["page_table"].cpu().numpy()
    args["q"][..., 0] = 4.0
    args["q"][..., 1:] *= 0.05
    pg, sl = so.place(tab, 16, 0, 37)
    kc, vc = args["k_cache"].float(), args["v_cache"].float()
    kc[..., 0] = 0.0
    kc[pg, :, sl] = 0.0
    kc[pg, :, sl, 0] = 1.0
    vc[pg, :, sl] = 0.0
    args["k_cache"], args["v_cache"] = kc.to(DT["e4m3"]), vc.to(DT["e4m3"])
    args["k_scale"][pg, :, sl] = above * math.sqrt(D) / 4.0
    args["v_scale"][pg, :, sl] = 3.0 / 448.0                 # as of a row of usual size
    if how == "split":
        args = widen(args)
    o, lse = U.attn_decode(**args)
    U.check()
    check_e4m3(o, lse, args)


@pytest.mark.parametrize("how", ["cluster", "split"])
def test_queries_with_one_huge_element(how):
    """An element 2^28 times the others, where K is zero: the scores are the
    others' products."""
    args, _ = build([400, 0, 33], 8, 2, 128, 16, "bf16", "e4m3", "seq", seed=22)
    args["q"] *= 2.0 ** -9
    args["q"][..., 5] = 2.0 ** 20
    kc = args["k_cache"].float()
    kc[..., 5] = 0.0
    args["k_cache"] = kc.to(DT["e4m3"])
    args["k_scale"] *= 2.0 ** 8
    if how == "split":
        args = widen(args)
    o, lse = U.attn_decode(**args)
    U.check()
    check_e4m3(o, lse, args)


# ------------------------------------------------------------------ infinite V

@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (8, 2, 64), (24, 2, 128), (2, 2, 128)])
@pytest.mark.parametrize("how", ["cluster", "split"])
@pytest.mark.parametrize("simt", [False, True])
def test_infinite_values_of_a_bf16_cache(Hq, Hkv, D, how, simt):
    """Infinite V elements make their element of the output infinite, both signs
    in one element NaN, and leave the others as they are."""
    n = 300
    args, _ = build([n, 40], Hq, Hkv, D, 16, "bf16", "bf16", "seq", seed=23)
    tab = args["page_table"].cpu().numpy()
    inf = float("inf")
    clean = args["v_cache"].clone()
    for d, keys in ((3, [(7, inf)]), (20, [(150, -inf)]), (41, [(9, inf), (280, -inf)]), (50, [(i, inf) for i in range(n)])):
        for key, x in keys:
            pg, sl = so.place(tab, 16, 0, key)
            args["v_cache"][pg, 0, sl, d] = x
            clean[pg, 0, sl, d] = 0.0
    if how == "split":
        args = widen(args)
    U.set_kernel(U.KERNEL_SIMT if simt else U.KERNEL_AUTO)
    try:
        o, _ = U.attn_decode(**args)
        want, _ = U.attn_decode(**{**args, "v_cache": clean})
        U.check()
    finally:
        U.set_kernel(U.KERNEL_AUTO)
    g = Hq // Hkv
    mine = o[0, :g].float()
    assert bool((mine[:, 3] == inf).all()) and bool((mine[:, 20] == -inf).all()), (mine[:, 3], mine[:, 20])
    assert bool(torch.isnan(mine[:, 41]).all()) and bool((mine[:, 50] == inf).all())
    left = torch.ones(D, dtype=torch.bool, device="cuda")
    left[[3, 20, 41, 50]] = False
    assert torch.equal(o[0, :g][:, left], want[0, :g][:, left])
    assert torch.equal(o[0, g:], want[0, g:]) and torch.equal(o[1], want[1])


# ------------------------------------------------------------------ no key that counts

@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("Hq", [2, 8])
@pytest.mark.parametrize("how", ["cluster", "split"])
@pytest.mark.parametrize("simt", [False, True])
def test_a_sequence_whose_pages_are_all_bad_is_empty(dtype, cache, Hq, how, simt):
    """Its keys are left out, every one: O = 0 and LSE = -inf, as of length 0."""
    n = 900
    args, rows = build([40, n, 70], Hq, 2, 128, 16, dtype, cache, "seq", seed=24)
    if how == "split":
        args = widen(args)
    args["page_table"][1] = -1
    U.set_kernel(U.KERNEL_SIMT if simt else U.KERNEL_AUTO)
    try:
        o, lse = U.attn_decode(**args)
    finally:
        U.set_kernel(U.KERNEL_AUTO)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    assert bool((o[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    check(o[::2], lse[::2], rows[::2], dtype, cache, "seq", simt=simt)


@pytest.mark.parametrize("dtype,Hq,simt", [("bf16", 8, False), ("bf16", 8, True), ("fp32", 2, False), ("fp32", 8, True)])
@pytest.mark.parametrize("n", [1, 900])
@pytest.mark.parametrize("how", ["cluster", "split"])
def test_scores_of_minus_infinity_alone_are_empty(dtype, Hq, simt, n, how):
    args, rows = build([40, n], Hq, 2, 128, 16, dtype, dtype, "seq", seed=25)
    args["q"][1, :, 0] = 1.0
    tab = args["page_table"].cpu().numpy()
    for i in range(n):
        pg, sl = so.place(tab, 16, 1, i)
        args["k_cache"][pg, :, sl] = 0.0
        args["k_cache"][pg, :, sl, 0] = float("-inf")
    if how == "split":
        args = widen(args)
    U.set_kernel(U.KERNEL_SIMT if simt else U.KERNEL_AUTO)
    try:
        o, lse = U.attn_decode(**args)
        U.check()
    finally:
        U.set_kernel(U.KERNEL_AUTO)
    assert bool((o[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    check(o[:1], lse[:1], rows[:1], dtype, dtype, "seq", simt=simt)


# ------------------------------------------------------------------ joins

@pytest.mark.parametrize("dtype,cache,D", [("bf16", "bf16", 128), ("fp32", "fp32", 128), ("bf16", "e4m3", 64),
                                           ("fp32", "fp32", 64)])
@pytest.mark.parametrize("B,longest", [(6, 2100), (16, 900), (24, 700), (64, 330), (80, 300)])
def test_every_way_to_join(dtype, cache, D, B, longest):
    """192, 512, 768, 2048 and 2560 output rows of 32 heads each, from items
    whose keys several warps walk, and an empty place."""
    lens = [longest] + [1 + (i * 389) % longest for i in range(1, B)]
    lens[B // 2] = 0
    args, rows = build(lens, 32, 8, D, 16, dtype, cache, "head", seed=26)
    args = widen(args)
    o, lse = U.attn_decode(**args)
    U.check()
    check(o, lse, rows, dtype, cache, "head")
    o2, lse2 = U.attn_decode(**args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ------------------------------------------------------------------ roundings of bf16 outputs

@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [2, 5])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (16, 8, 64), (64, 8, 128), (32, 2, 64)])
@pytest.mark.parametrize("how", ["cluster", "split"])
def test_outputs_are_rounded_from_fp32_sums(cache, n, Hq, Hkv, D, how):
    """Few keys and small scores, so that fp32 arithmetic is within
    lim = (2 max ds + (n + 16) e + 2^-22) sum p |v| of the output (the last term an
    e4m3 cache's), about 2^-19 of it: every element is one that bf16 rounds a value
    within lim of the definition's to, and not the next."""
    B = 48
    args, rows = build([n] * B, Hq, Hkv, D, 16, "bf16", cache, "seq", seed=27)
    args["q"] = (args["q"].float() * 0.02).bfloat16()
    if how == "split":
        args = widen(args)
    o, _ = U.attn_decode(**args)
    U.check()
    got, sc = f64(o), 1.0 / math.sqrt(D)
    low, high = np.empty_like(got), np.empty_like(got)
    for b, (_, k, v) in enumerate(rows):
        q = f64(args["q"][b])
        ro, rl = so.decode(q, k, v)
        for h in range(Hq):
            K, V = k[:, h * Hkv // Hq], v[:, h * Hkv // Hq]
            ds = sc * (D + 4) * E * (np.abs(K) @ np.abs(q[h])).max()
            lim = (2 * ds + (n + 16) * E + (2.0 ** -22 if cache == "e4m3" else 0.0)) * (np.exp(sc * (K @ q[h]) - rl[h]) @ np.abs(V))
            low[b, h], high[b, h] = ro[h] - lim, ro[h] + lim
    low, high = (f64(torch.from_numpy(x).to(torch.bfloat16)) for x in (low, high))
    assert np.all((low <= got) & (got <= high)), int(np.sum((got < low) | (got > high)))
