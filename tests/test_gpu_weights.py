"""Attention weights that cached tokens gather (ulysses_attn_decode_weights)
against the fp64 definition, and the outputs beside them.

A weight p = exp2(s - m) / l: with ds the score's bound (test_gpu_decode's and
test_gpu_4bit's) and l summed over n keys of that error, p is off by
p (2 max ds + (n + 32) 2 e); the G heads' sum and the addition to what the slot
holds round by (G + 1) e of the result."""
import math

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

from tests.test_gpu_4bit import build4, check4
from tests.test_gpu_decode import build, check, f64, widen

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def make(lens, Hq, H, D, page, dtype, cache, layout, seed=0):
    if cache == "e2m1":
        return build4(lens, Hq, H, D, page, dtype, layout, seed=seed)[:2]
    return build(lens, Hq, H, D, page, dtype, cache, layout, seed=seed)


def start(args, seed=0):
    return torch.rand(args["k_cache"].shape[:3], generator=torch.Generator().manual_seed(seed)).cuda()


def check_weights(got, before, args, rows, times=1, scale=None):
    """got against before + times the weights of the definition; other slots as before."""
    tab, page = args["page_table"].cpu().numpy(), args["k_cache"].shape[2]
    got, want = f64(got), f64(before)
    lim = np.zeros(want.shape)
    for b, (q, k, _) in enumerate(rows):
        n, (Hq, D) = len(k), q.shape
        if n == 0:
            continue
        w, H = so.attention_weights(q, k, scale), k.shape[1]
        sc = 1.0 / math.sqrt(D) if scale is None else scale
        G = Hq // H
        at = np.array([(int(tab[b][p // page]), p % page) for p in range(n)])
        for h in range(H):
            aq = np.abs(q[h * G:(h + 1) * G])
            ds = sc * (2 * (D + 4) * E + 2.0 ** -21) * (np.abs(k[:, h]) @ aq.T).max()
            ds += sc * 2.0 ** -25 * aq.max() * np.abs(k[:, h]).sum(-1).max() * (args["k_scale"] is not None)
            want[at[:, 0], h, at[:, 1]] += times * w[:, h]
            lim[at[:, 0], h, at[:, 1]] += times * w[:, h] * (2 * ds + 2 * (n + 32) * E + (G + 1) * E)
    lim = lim + (lim > 0) * (times + 1) * E * np.abs(want)
    err = np.abs(got - want)
    assert np.all(err <= lim), float((err / np.where(lim > 0, lim, 1e-300)).max())


CASES = [  # lens, Hq, H, D, page, dtype, cache, layout
    ([1], 1, 1, 128, 16, "bf16", "bf16", "seq"),
    ([0], 4, 2, 64, 16, "bf16", "e4m3", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 128, 16, "bf16", "bf16", "head"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 64, 32, "bf16", "e4m3", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 6, 2, 128, 48, "bf16", "e2m1", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 4, 2, 64, 16, "fp32", "fp32", "head"),
    ([777, 40], 32, 8, 128, 16, "bf16", "bf16", "head"),
    ([1500, 0, 333], 16, 2, 128, 64, "bf16", "bf16", "seq"),
    ([1500, 0, 333], 16, 1, 64, 64, "bf16", "e2m1", "seq"),
    ([700, 100], 40, 2, 128, 128, "bf16", "e4m3", "head"),       # two groups of heads a kv head
    ([700, 100], 20, 1, 128, 16, "fp32", "e2m1", "seq"),         # three
    ([900, 31], 3, 1, 64, 16, "fp32", "e4m3", "seq"),
    ([900, 31], 1, 1, 128, 16, "fp32", "fp32", "seq"),
    ([4099], 32, 8, 128, 16, "bf16", "bf16", "head"),            # eight warps a CTA: eight CTAs,
    ([2047, 2033], 64, 4, 128, 64, "bf16", "e2m1", "seq"),       # 16 heads a kv head
    ([1000, 0, 900, 512, 1], 24, 4, 64, 48, "bf16", "e4m3", "head"),   # four CTAs
    ([1023, 800], 16, 2, 128, 32, "fp32", "fp32", "seq"),
    ([500 + 13 * i for i in range(20)], 8, 8, 128, 16, "bf16", "bf16", "seq"),   # too many for eight warps: one CTA of four
]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_weights(case, wide):
    lens, Hq, H, D, page, dtype, cache, layout = CASES[case]
    args, rows = make(lens, Hq, H, D, page, dtype, cache, layout, seed=case)
    if wide:
        args = widen(args)
    before = start(args, case)
    w = before.clone()
    o, lse = U.attn_decode(weights=w, **args)
    U.check()
    check_weights(w, before, args, rows)
    # the outputs beside them: the plain call's (a narrow table's clusters add pieces up in another order)
    po, pl = U.attn_decode(**args)
    if wide:
        assert torch.equal(o, po) and torch.equal(lse, pl)
    elif cache == "e2m1":
        check4(o, lse, rows, build4(lens, Hq, H, D, page, dtype, layout, seed=case)[2], dtype, layout)
    else:
        check(o, lse, rows, dtype, cache, layout)
    # and again on top, with a workspace of the caller's
    ws = U.attn_decode_workspace(args["q"], args["k_cache"], args["page_table"], layout=layout, weights=True)
    assert ws.numel() > 0 or not wide
    U.attn_decode(weights=w, workspace=ws, **args)
    U.check()
    check_weights(w, before, args, rows, times=2)
    v = before.clone()
    U.attn_decode(weights=v, **args)
    U.attn_decode(weights=v, **args)
    assert torch.equal(v, w)


@pytest.mark.parametrize("case", [2, 3, 4, 5, 8, 10])
def test_weights_simt(case):
    lens, Hq, H, D, page, dtype, cache, layout = CASES[case]
    args, rows = make(lens, Hq, H, D, page, dtype, cache, layout, seed=20 + case)
    U.set_kernel(U.KERNEL_SIMT)
    try:
        for a in (args, widen(args)):
            before = start(a)
            w = before.clone()
            U.attn_decode(weights=w, scale=0.2, **a)
            U.check()
            check_weights(w, before, a, rows, scale=0.2)
    finally:
        U.set_kernel(U.KERNEL_AUTO)


def test_more_sequences_than_a_launch_takes():
    lens = [(7 * i) % 40 for i in range(2100)]
    args, rows = make(lens, 2, 1, 64, 16, "bf16", "bf16", "seq", seed=9)
    before = start(args)
    w = before.clone()
    U.attn_decode(weights=w, **args)
    U.check()
    check_weights(w, before, args, rows)


@pytest.mark.parametrize("wide", [False, True])
def test_bad_pages_add_nothing(wide):
    args, rows = make([60, 50], 4, 1, 128, 16, "bf16", "bf16", "seq", seed=3)
    tab = args["page_table"]
    hole = int(tab[0, 1])
    tab[0, 1] = -7
    tab[1, 3] = 1 << 29
    if wide:
        args = widen(args)
    before = start(args)
    w = before.clone()
    U.attn_decode(weights=w, **args)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    left = [np.r_[0:16, 32:60], np.arange(48)]
    part = [(q, k[i], v[i]) for (q, k, v), i in zip(rows, left)]
    want, t = f64(before), tab.cpu().numpy()
    for b, (q, k, _) in enumerate(part):
        for j, x in zip(left[b], so.attention_weights(q, k)):
            want[int(t[b][j // 16]), :, j % 16] += x
    assert np.abs(f64(w) - want).max() < 1e-5 and torch.equal(w[hole], before[hole])


def test_shared_pages_gather_from_all():
    args, rows = make([48, 48], 4, 2, 64, 16, "bf16", "bf16", "seq", seed=4)
    args["page_table"][1] = args["page_table"][0]
    (q0, k0, v0), (q1, _, _) = rows
    for a in (args, widen(args)):
        before = start(a)
        w = before.clone()
        U.attn_decode(weights=w, **a)
        U.check()
        check_weights(w, before, a, [(q0, k0, v0), (q1, k0, v0)])


def test_captured_and_replayed_with_growing_lengths():
    args, rows = make([300, 45], 8, 2, 128, 16, "bf16", "e2m1", "seq", seed=6)
    args = widen(args)
    ws = U.attn_decode_workspace(args["q"], args["k_cache"], args["page_table"], weights=True)
    o, lse = torch.empty_like(args["q"]), torch.empty((2, 8), device="cuda")
    w = start(args)
    before = w.clone()
    U.attn_decode(weights=w, workspace=ws, out=o, lse=lse, **args)
    torch.cuda.synchronize()
    w.copy_(before)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        U.attn_decode(weights=w, workspace=ws, out=o, lse=lse, **args)
    want = before.clone()
    for lens in ([20, 45], [0, 0], [300, 1]):
        args["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        eo, el = U.attn_decode(weights=want, **args)
        assert torch.equal(o, eo) and torch.equal(lse, el) and torch.equal(w, want)
    U.check()
