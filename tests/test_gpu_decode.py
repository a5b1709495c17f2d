"""Attention of one new token per sequence over the paged cache
(ulysses_attn_decode) against the fp64 definition.

Element-wise bound.  With e = 2^-24 and keys' weights p_j (they add up to 1),
a score of D products is off by ds_j = (D + 4) e scale sum |q_d k_jd|, so its
weight by p_j (2 max ds + 8 e) with exp2f's 2 ulp; the sums over n keys round
n times: |do| <= (2 max ds + (n + 16) e + u) sum_j p_j |v_j|, plus half a step
of the output's type.  u is the rounding of the weights where the kernel feeds
them to the matrix pipe in 16 bits (with a bf16 cache as a bf16 value and the bf16
rest, 2^-16; f16 2^-11 with an e4m3 cache); in fp32 the operands are pairs of 11-bit parts, 2^-22
each, so u = 2^-21 and scores are off by 2^-21 scale sum |q_d k_jd| more; the
SIMT kernels have u = 0.  With an e4m3 cache the weights carry V's
scale, so f16's smallest step (2^-25 of the largest weighted scale) adds
n 448 2^-25 max_j(p_j scale_j), and q, scaled by a power of two into f16,
2^-25 max|q| in each element of it.  LSE: max ds + (n + 16) e + e |lse|."""
import math

import numpy as np
import pytest
import torch

import oracle
from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
E = 2.0 ** -24


def f64(t):
    return t.detach().float().double().cpu().numpy()


def build(lens, Hq, Hkv, D, page, dtype, cache, layout, seed=0, gain=1.0, slack=2):
    """Random cache in pages of a mixed order; every slot that no sequence owns
    is NaN (codes and scales too), unused table entries hold a wild id.
    Returns the call's tensors and each sequence's q, k, v in fp64."""
    g = torch.Generator().manual_seed(seed)
    per = [-(-n // page) for n in lens]
    total = sum(per) + slack
    order = torch.randperm(total, generator=g)
    tab = torch.full((len(lens), max(per) + 1), 1 << 30, dtype=torch.int32)
    own = torch.zeros((total, page), dtype=torch.bool)
    at = 0
    for b, n in enumerate(lens):
        for i in range(per[b]):
            p = int(order[at])
            at += 1
            tab[b, i] = p
            own[p, :min(page, n - i * page)] = True
    bufs = []
    for _ in range(2):
        x = torch.randn((total, Hkv, page, D), generator=g) * gain
        if cache == "e4m3":
            x = x * torch.exp(torch.randn((total, Hkv, page, 1), generator=g))
            s = x.abs().amax(-1) / 448.0
            c = (x / s[..., None]).to(DT[cache])
            s[~own[:, None].expand_as(s)] = float("nan")
            c.view(torch.uint8)[~own[:, None].expand(total, Hkv, page)] = 0x7F
            bufs.append((c.cuda(), s.cuda()))
        else:
            c = x.to(DT[cache])
            c[~own[:, None].expand(total, Hkv, page)] = float("nan")
            bufs.append((c.cuda(), None))
    B = len(lens)
    q = (torch.randn((B, Hq, D), generator=g) * 2).to(DT[dtype])
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    (kc, ks), (vc, vs) = bufs
    rows = []
    for b, n in enumerate(lens):
        kv = []
        for c, s in bufs:
            r = so.cache_rows(f64(c), tab.numpy(), b, n)
            if s is not None:
                r = r * so.cache_rows(f64(s)[..., None], tab.numpy(), b, n)
            kv.append(r)
        rows.append((f64(q[b]), *kv))
    qd = (q if layout == "seq" else q.transpose(0, 1)).contiguous().cuda()
    return dict(q=qd, k_cache=kc, v_cache=vc, page_table=tab.cuda(), seq_lens=ln, k_scale=ks, v_scale=vs,
                layout=layout), rows


def widen(args, positions=1 << 20):
    """The same call with a table of room for many more positions: its unused
    entries are never read, and the keys are split over the whole launch
    instead of a cluster for each item."""
    tab = args["page_table"]
    wide = torch.full((tab.shape[0], max(tab.shape[1], positions // args["k_cache"].shape[2])), -5, dtype=torch.int32,
                      device="cuda")
    wide[:, :tab.shape[1]] = tab
    return {**args, "page_table": wide}


def check(o, lse, rows, dtype, cache, layout, scale=None, simt=False):
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
        mma = dtype == "bf16" and not simt
        for h in range(Hq):
            K, V = k[:, h // G], v[:, h // G]
            split = dtype == "fp32" and not simt
            ds = sc * ((D + 4) * E + (2.0 ** -21 if split else 0.0)) * (np.abs(K) @ np.abs(q[h])).max()
            if mma and cache == "e4m3":
                ds += sc * 2.0 ** -25 * np.abs(q[h]).max() * np.abs(K).sum(-1).max()
            s = sc * (K @ q[h])
            p = np.exp(s - rl[h])
            u = (2.0 ** -11 if cache == "e4m3" else 2.0 ** -16) if mma else 2.0 ** -21 if split else 0.0
            lim = (2 * ds + (n + 16) * E + u) * (p @ np.abs(V))
            if mma and cache == "e4m3":
                lim = lim + n * 2.0 ** -25 * (p * np.abs(V).max(-1)).max()
            lim = lim + np.abs(ro[h]) * (2.0 ** -8 if dtype == "bf16" else E) * 1.01 + 1e-37
            err = np.abs(o[b, h] - ro[h])
            assert np.all(err <= lim), (b, h, n, float((err / lim).max()))
            assert abs(lse[b, h] - rl[h]) <= ds + (n + 16) * E + 2 * E * abs(rl[h]), (b, h, lse[b, h], rl[h])


CASES = [
    # lens, Hq, Hkv, D, page, dtype, cache, layout
    ([1], 1, 1, 128, 16, "bf16", "bf16", "seq"),
    ([0], 4, 1, 128, 16, "bf16", "bf16", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 128, 16, "bf16", "bf16", "head"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 8, 2, 64, 32, "bf16", "e4m3", "seq"),
    ([0, 1, 2, 15, 16, 17, 31, 33], 4, 2, 64, 16, "fp32", "fp32", "head"),
    ([777], 32, 8, 128, 16, "bf16", "bf16", "head"),
    ([777, 3], 32, 8, 128, 48, "bf16", "e4m3", "head"),
    ([5, 1200, 64, 0, 65], 6, 2, 128, 64, "bf16", "bf16", "seq"),
    ([300, 20], 7, 1, 128, 16, "bf16", "bf16", "seq"),
    ([300, 20], 5, 1, 64, 16, "bf16", "e4m3", "seq"),
    ([513, 127], 16, 1, 128, 128, "bf16", "bf16", "head"),
    ([513, 127], 16, 2, 64, 128, "bf16", "bf16", "head"),
    ([260, 1], 40, 2, 64, 16, "bf16", "e4m3", "seq"),
    ([260, 1], 12, 1, 128, 16, "bf16", "e4m3", "seq"),
    ([100, 1000], 3, 3, 128, 16, "fp32", "fp32", "seq"),
    ([100, 1000], 12, 2, 64, 80, "fp32", "e4m3", "head"),
    ([100, 1000], 4, 2, 128, 256, "fp32", "e4m3", "head"),
    ([4097, 1, 2500], 8, 2, 128, 64, "bf16", "bf16", "head"),
    ([20001], 2, 1, 64, 16, "bf16", "bf16", "seq"),
    ([20001], 4, 1, 128, 32, "bf16", "e4m3", "seq"),
    ([4001, 0, 3, 2048], 20, 2, 128, 32, "fp32", "fp32", "head"),
    ([4001, 0, 3, 2048], 9, 1, 64, 16, "fp32", "e4m3", "seq"),
    ([15, 16, 17, 23, 24, 25], 8, 1, 128, 48, "fp32", "fp32", "seq"),
    ([15, 16, 17, 23, 24, 25], 1, 1, 128, 16, "fp32", "e4m3", "seq"),
    ([3000, 2999], 24, 2, 128, 16, "bf16", "e4m3", "seq"),
    ([3] * 70 + [0] * 3 + [129] * 9, 4, 2, 64, 16, "bf16", "bf16", "seq"),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,dtype,cache,layout", CASES)
def test_against_the_definition(lens, Hq, Hkv, D, page, dtype, cache, layout):
    args, rows = build(lens, Hq, Hkv, D, page, dtype, cache, layout)
    o, lse = U.attn_decode(**args)
    U.check()
    assert o.shape == args["q"].shape and o.dtype == args["q"].dtype and lse.shape == (len(lens), Hq)
    check(o, lse, rows, dtype, cache, layout)
    o2, lse2 = U.attn_decode(**args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)          # no order of the GPU's in it
    args = widen(args)
    assert U.attn_decode_workspace(args["q"], args["k_cache"], args["page_table"], layout=layout).numel() > 0
    o, lse = U.attn_decode(**args)
    U.check()
    check(o, lse, rows, dtype, cache, layout)
    o2, lse2 = U.attn_decode(**args)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32"), ("fp32", "e4m3")])
@pytest.mark.parametrize("Hq,D,lens", [(12, 128, [0, 1, 40, 333]), (6, 64, [17, 2500]), (2, 128, [130])])
def test_simt_kernels(dtype, cache, Hq, D, lens):
    args, rows = build(lens, Hq, 2, D, 16, dtype, cache, "head")
    U.set_kernel(U.KERNEL_SIMT)
    try:
        o, lse = U.attn_decode(**args)
        o2, lse2 = U.attn_decode(**widen(args))
        U.check()
    finally:
        U.set_kernel(U.KERNEL_AUTO)
    check(o, lse, rows, dtype, cache, "head", simt=True)
    check(o2, lse2, rows, dtype, cache, "head", simt=True)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
@pytest.mark.parametrize("order", ["rising", "falling"])
def test_running_maximum(dtype, cache, order):
    """Scores over a range of hundreds, rising or falling along the cache: the
    maximum moves at every tile, or never again; the weights of most keys
    vanish."""
    args, rows = build([700, 90], 8, 2, 128, 16, dtype, cache, "seq", seed=3)
    kc, tab = args["k_cache"], args["page_table"].cpu().numpy()
    step = torch.linspace(0.1, 12.0, 700) if order == "rising" else torch.linspace(12.0, 0.1, 700)
    scaled = args["k_scale"] if cache == "e4m3" else kc
    for b, n in ((0, 700), (1, 90)):
        for i in range(n):
            pg, sl = so.place(tab, 16, b, i)
            scaled[pg, :, sl] = (scaled[pg, :, sl].float() * float(step[i])).to(scaled.dtype)
    new = []
    for b, n in enumerate((700, 90)):
        r = so.cache_rows(f64(kc), tab, b, n)
        if cache == "e4m3":
            r = r * so.cache_rows(f64(args["k_scale"])[..., None], tab, b, n)
        new.append((rows[b][0], r, rows[b][2]))
    for x in (args, widen(args)):
        o, lse = U.attn_decode(**x)
        U.check()
        check(o, lse, new, dtype, cache, "seq")


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3"), ("fp32", "fp32")])
def test_scale_out_lse_workspace_and_strides(dtype, cache):
    args, rows = build([50, 0, 211], 8, 2, 64, 16, dtype, cache, "seq", seed=4)
    wide = torch.full((3, 11, 64), 5.0, dtype=DT[dtype], device="cuda")
    wide[:, :8] = args["q"]
    out = torch.full((3, 9, 64), 9.0, dtype=DT[dtype], device="cuda")
    lse = torch.empty((3, 8), device="cuda")
    args = widen(args)
    ws = U.attn_decode_workspace(wide[:, :8], args["k_cache"], args["page_table"])
    assert ws.numel() > 0
    args["q"] = wide[:, :8]
    o, l2 = U.attn_decode(**args, scale=0.03, out=out[:, :8], lse=lse, workspace=ws)
    U.check()
    assert o.data_ptr() == out.data_ptr() and l2 is lse and bool((out[:, 8] == 9.0).all())
    check(o, lse, rows, dtype, cache, "seq", scale=0.03)


def test_not_finite_values_where_they_count():
    """A NaN or infinite row that a sequence owns shows in its own heads and
    nowhere else; scores of -inf alone have no weight."""
    args, rows = build([40, 40, 40], 4, 2, 128, 16, "bf16", "bf16", "seq", seed=5)
    tab = args["page_table"].cpu().numpy()
    pg, sl = so.place(tab, 16, 1, 17)
    args["v_cache"][pg, 0, sl, 3] = float("nan")
    pg, sl = so.place(tab, 16, 2, 0)                 # the first key: score -inf or +inf by q's sign
    args["k_cache"][pg, 1, sl, :] = 0
    args["k_cache"][pg, 1, sl, 0] = float("-inf")
    args["q"][2, 2:, 0] = 1.0                        # heads 2, 3: -inf
    q2, k2, v2 = rows[2]
    q2 = f64(args["q"][2])
    ro, rl = so.decode(q2, k2[1:], v2[1:])           # as if the key were not there
    for x in (args, widen(args)):
        o, lse = U.attn_decode(**x)
        U.check()
        bad = torch.isnan(o)
        assert bool(bad[1, :2, 3].all()) and int(bad.sum()) == 2
        assert np.max(np.abs(f64(o[2, 2:]) - ro[2:])) <= 0.05 and np.max(np.abs(f64(lse[2, 2:]) - rl[2:])) <= 1e-4


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp32", "fp32")])
def test_bad_pages_and_lengths_are_reported(dtype, cache):
    args, rows = build([40, 40], 2, 1, 64, 16, dtype, cache, "seq", seed=6)
    good = args["page_table"].clone()
    cap = good.shape[1] * 16
    for col, page in ((1, -1), (2, 1 << 20)):
        args["page_table"] = good.clone()
        args["page_table"][1, col] = page
        o, lse = U.attn_decode(**args)
        with pytest.raises(U.UlyssesError) as e:
            U.check()
        assert e.value.code == U.ERR_BAD_PAGES
        check(o[:1], lse[:1], rows[:1], dtype, cache, "seq")
    args["page_table"] = good
    for n in (-1, cap + 1, 2 ** 31 - 1):
        args["seq_lens"] = torch.tensor([40, n], dtype=torch.int32, device="cuda")
        o, lse = U.attn_decode(**args)
        with pytest.raises(U.UlyssesError) as e:
            U.check()
        assert e.value.code == U.ERR_BAD_PAGES
        check(o[:1], lse[:1], rows[:1], dtype, cache, "seq")
    U.check()


@pytest.mark.parametrize("how", ["cluster", "split"])
def test_other_streams_and_captured_graphs(how):
    """One call on a stream of its own, and a captured one replayed with new
    lengths, queries and pages in the same tensors; two graphs with one
    workspace, replayed in turn."""
    a, ra = build([6000, 30], 8, 2, 128, 16, "bf16", "bf16", "seq", seed=7)
    b, rb = build([17, 6000], 8, 2, 128, 16, "bf16", "bf16", "seq", seed=8)
    if how == "split":
        a, b = widen(a), widen(b)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o, lse = U.attn_decode(**a, stream=st)
    st.synchronize()
    check(o, lse, ra, "bf16", "bf16", "seq")
    ws = U.attn_decode_workspace(a["q"], a["k_cache"], a["page_table"])
    assert (ws.numel() > 0) == (how == "split")
    kw = dict(workspace=ws) if ws.numel() else {}
    graphs, outs = [], []
    for args in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(U.attn_decode(**args, **kw))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    check(*outs[0], ra, "bf16", "bf16", "seq")
    check(*outs[1], rb, "bf16", "bf16", "seq")
    # new contents in the captured tensors
    for x in ("q", "k_cache", "v_cache", "seq_lens", "page_table"):
        a[x].copy_(b[x])
    graphs[0].replay()
    U.check()
    check(*outs[0], rb, "bf16", "bf16", "seq")


def test_cache_beyond_32_bit_offsets():
    H, D, page, n = 8, 128, 256, 700
    pages = (1 << 32) // (H * D * page) + 40
    kc = torch.zeros((pages, H, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.zeros_like(kc)
    ks = torch.zeros((pages, H, page), device="cuda")
    vs = torch.zeros_like(ks)
    tab = torch.tensor([[pages - 1, 1, pages - 2]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn((n, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    U.cache_write(k, v, kc, vc, tab, cu[1:], cu_new=cu, k_scale=ks, v_scale=vs)
    q = torch.randn((1, 32, D), generator=g).bfloat16().cuda()
    o, lse = U.attn_decode(q, kc, vc, tab, cu[1:], k_scale=ks, v_scale=vs)
    U.check()
    rk, rv = (so.cache_rows(np.stack([f64(c[i]) for i in (pages - 1, 1, pages - 2)]), [[0, 1, 2]], 0, n) for c in (kc, vc))
    sk, sv = (so.cache_rows(np.stack([f64(c[i]) for i in (pages - 1, 1, pages - 2)])[..., None], [[0, 1, 2]], 0, n) for c in (ks, vs))
    check(o, lse, [(f64(q[0]), rk * sk, rv * sv)], "bf16", "e4m3", "seq")
    del kc, vc, ks, vs
    torch.cuda.empty_cache()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_decode_loop_as_it_is_used(cache):
    """Prompts of two lengths go through the projection, rotary positions, the
    layer's attention and into the cache; then tokens one by one: projection,
    rotary positions in place, cache write, attention over the cache, output
    projection.  Every new token's attention is the last row of the oracle's
    causal attention over the whole sequence."""
    Hq, Hkv, D, hidden, page = 8, 2, 128, 512, 16
    H = Hq + 2 * Hkv
    g = torch.Generator().manual_seed(10)
    wqkv = (torch.randn((H * D, hidden), generator=g) * hidden ** -0.5).bfloat16().cuda()
    wo = (torch.randn((hidden, Hq * D), generator=g) * (Hq * D) ** -0.5).bfloat16().cuda()
    inv, axes = U.rope_frequencies(D, 1e6)
    prompt, steps = [130, 45], 4
    B, T = len(prompt), sum(prompt)
    tab = torch.arange(24, dtype=torch.int32, device="cuda").flip(0).view(2, 12).contiguous()
    kc, vc, ks, vs = U.kv_cache(24, page, Hkv, D, DT[cache])
    x = torch.randn((T, hidden), generator=g).bfloat16().cuda()
    qkv = U.qkv_proj(x, wqkv, Hq, Hkv)                                      # [H, T, D]
    pos = torch.cat([torch.arange(n) for n in prompt]).to(torch.int32).cuda()
    q, k, v = qkv[:Hq], qkv[Hq:Hq + Hkv], qkv[Hq + Hkv:]
    U.rope_fwd(q, k, pos, inv, axes, layout="head", out=(q, k))
    cu = torch.tensor([0, prompt[0], T], dtype=torch.int32, device="cuda")
    o, _ = U.attn_fwd(q[None], k[None], v[None], Hq, Hkv, 1, cu_seqlens=cu)
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    U.cache_write(k, v, kc, vc, tab, lens, cu_new=cu, k_scale=ks, v_scale=vs, layout="head")
    U.check()
    # what the cache holds, unrounded: fp32 from 8-bit rows
    held = torch.bfloat16 if cache == "bf16" else torch.float32
    rk, rv = U.cache_read(kc, vc, tab, cu, T, k_scale=ks, v_scale=vs, layout="head", dtype=held)
    if cache == "bf16":
        assert torch.equal(rk, k) and torch.equal(rv, v)
    keys = [[f64(rk[:, cu[b]:cu[b + 1]]), f64(rv[:, cu[b]:cu[b + 1]])] for b in range(B)]    # [Hkv, n, D]
    for _ in range(steps):
        x = torch.randn((B, hidden), generator=g).bfloat16().cuda()
        qkv = U.qkv_proj(x, wqkv, Hq, Hkv)
        q, k, v = qkv[:Hq], qkv[Hq:Hq + Hkv], qkv[Hq + Hkv:]
        U.rope_fwd(q, k, lens, inv, axes, layout="head", out=(q, k))
        lens += 1
        U.cache_write(k, v, kc, vc, tab, lens, k_scale=ks, v_scale=vs, layout="head")
        o, lse = U.attn_decode(q, kc, vc, tab, lens, k_scale=ks, v_scale=vs, layout="head")
        y = U.out_proj(o, wo)
        U.check()
        assert y.shape == (B, hidden) and bool(torch.isfinite(y).all())
        one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        nk, nv = U.cache_read(kc, vc, tab, one, B, first=lens - 1, k_scale=ks, v_scale=vs, layout="head",
                              dtype=held)
        for b in range(B):
            keys[b] = [np.concatenate([a, f64(n[:, b:b + 1])], 1) for a, n in zip(keys[b], (nk, nv))]
            n = keys[b][0].shape[1]
            full = np.zeros((Hq, n, D))
            full[:, -1] = f64(q[:, b])
            ro, rl = oracle.attn_fwd(full, keys[b][0], keys[b][1], None, True)
            # the bf16 tolerances of the layer's own attention tests
            assert np.max(np.abs(f64(o[:, b]) - ro[:, -1])) <= 2e-2
            assert np.max(np.abs(f64(lse[b]) - rl[:, -1])) <= 1e-3


def test_more_sequences_than_one_launch_takes():
    B = 2100                                          # 2048 a launch
    lens = [(7 * i) % 37 for i in range(B)]
    args, rows = build(lens, 2, 1, 64, 16, "bf16", "bf16", "head", seed=11)
    o, lse = U.attn_decode(**args)
    U.check()
    check(o, lse, rows, "bf16", "bf16", "head")


@pytest.mark.parametrize("spread,gain", [(18.0, 2.0), (30.0, 60.0), (3.0, 1e-4)])
@pytest.mark.parametrize("how", ["cluster", "split"])
def test_e4m3_rows_of_very_different_scales(spread, gain, how):
    """V's scales over 2^-spread .. 2^spread, queries from nearly uniform to
    nearly one-hot weights: f16 weights follow the largest contribution."""
    args, rows = build([333, 40], 6, 2, 128, 16, "bf16", "e4m3", "seq", seed=12)
    g = torch.Generator().manual_seed(13)
    f = torch.exp2((torch.rand(args["v_scale"].shape, generator=g) * 2 - 1) * spread).cuda()
    args["v_scale"] *= f
    args["q"] = (args["q"].float() * gain / 2).bfloat16()
    tab = args["page_table"].cpu().numpy()
    new = []
    for b, n in enumerate((333, 40)):
        v = so.cache_rows(f64(args["v_cache"]), tab, b, n) * so.cache_rows(f64(args["v_scale"])[..., None], tab, b, n)
        new.append((f64(args["q"][b]), rows[b][1], v))
    o, lse = U.attn_decode(**(widen(args) if how == "split" else args))
    U.check()
    check(o, lse, new, "bf16", "e4m3", "seq")


@pytest.mark.parametrize("Hq,D", [(8, 128), (4, 64)])
def test_long_fp32_sums_keep_fp32_precision(Hq, D):
    """20000 keys of nearly equal weights: the 2-norm of the error stays below
    that of one fp32 rounding a key accumulated at random, sqrt(n) 2^-24 of the
    weighted values' 2-norm, plus the products' 2^-21."""
    n = 20000
    args, rows = build([n], Hq, 1, D, 64, "fp32", "fp32", "seq", seed=18)
    args["q"] *= 0.05
    q, k, v = f64(args["q"][0]), rows[0][1], rows[0][2]
    o, _ = U.attn_decode(**widen(args, 1 << 22))
    U.check()
    ro, rl = so.decode(q, k, v)
    p = np.exp(k[:, 0] @ q.T / math.sqrt(D) - rl)                # [n, Hq]
    size = np.sqrt((p ** 2).T @ (v[:, 0] ** 2))                   # [Hq, D]: spread of a sum of n products
    lim = np.linalg.norm(size) * (math.sqrt(n) * E + 2.0 ** -21) + np.linalg.norm(ro) * 2.0 ** -20
    assert np.linalg.norm(f64(o[0]) - ro) <= lim


def test_nothing_outside_outputs_and_workspace_is_written():
    """Windows with guard bytes on both sides, in both ways of a launch."""
    pat, guard, bufs = 0xA5, 4096, []

    def window(shape, dtype):
        n = torch.Size(shape).numel() * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((2 * guard + (n + 255) // 256 * 256,), pat, dtype=torch.uint8, device="cuda")
        bufs.append((raw, n))
        return raw[guard:guard + n].view(dtype).view(shape)

    for dtype, cache, D, Hq in (("bf16", "bf16", 128, 24), ("bf16", "e4m3", 64, 6), ("fp32", "fp32", 64, 10),
                                ("fp32", "fp32", 128, 2)):
        args, rows = build([1, 0, 700, 33], Hq, 2, D, 16, dtype, cache, "head", seed=14)
        for x in (args, widen(args)):
            n = U.attn_decode_workspace(x["q"], x["k_cache"], x["page_table"], layout="head").numel()
            o, lse = U.attn_decode(**x, out=window(x["q"].shape, DT[dtype]), lse=window((4, Hq), torch.float32),
                                   workspace=window((n,), torch.uint8) if n else None)
            U.check()
            check(o, lse, rows, dtype, cache, "head")
    for raw, n in bufs:
        assert bool((raw[:guard] == pat).all()) and bool((raw[guard + n:] == pat).all())


def test_two_calls_at_once_on_two_streams():
    a, ra = build([5000, 100, 1], 8, 2, 128, 16, "bf16", "bf16", "seq", seed=15)
    b, rb = build([31, 4000], 8, 2, 128, 16, "bf16", "e4m3", "seq", seed=16)
    a, b = widen(a), widen(b)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    t.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append((U.attn_decode(**a, stream=s), U.attn_decode(**b, stream=t)))
    torch.cuda.synchronize()
    U.check()
    for x, y in got:
        assert torch.equal(x[0], got[0][0][0]) and torch.equal(y[0], got[0][1][0])
    check(*got[0][0], ra, "bf16", "bf16", "seq")
    check(*got[0][1], rb, "bf16", "e4m3", "seq")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_captured_step_replayed_with_an_empty_place(cache):
    """Rotary positions, cache write and attention of one step in a CUDA graph;
    the lengths grow in it, and one place of the batch is empty.  Replays equal
    the calls one by one."""
    Hq, Hkv, D, page, B = 8, 2, 128, 16, 4
    inv, axes = U.rope_frequencies(D)
    start = torch.tensor([15, 40, 0, 1], dtype=torch.int32, device="cuda")
    used = (start > 0).to(torch.int32)
    tab = torch.arange(B * 6, dtype=torch.int32, device="cuda").view(B, 6)
    g = torch.Generator().manual_seed(17)
    steps = torch.randn((5, B, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()

    def fresh():
        bufs = U.kv_cache(B * 6, page, Hkv, D, DT[cache])
        return bufs, start.clone()

    def step(x, bufs, lens):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q, k = U.rope_fwd(q, k, lens, inv, axes)
        lens.add_(used)
        U.cache_write(k, v, bufs[0], bufs[1], tab, lens, k_scale=bufs[2], v_scale=bufs[3])
        return U.attn_decode(q, bufs[0], bufs[1], tab, lens, k_scale=bufs[2], v_scale=bufs[3])

    bufs, lens = fresh()
    want = [tuple(t.clone() for t in step(x, bufs, lens)) for x in steps]
    bufs2, lens2 = fresh()
    x = steps[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, bufs2, lens2)
    for i in range(5):
        x.copy_(steps[i])
        graph.replay()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1]), i
        assert bool((out[0][2] == 0).all()) and bool(torch.isneginf(out[1][2]).all())
    U.check()
    assert torch.equal(lens, lens2)
    for p, r in zip(bufs, bufs2):
        assert p is None or torch.equal(p.view(torch.uint8), r.view(torch.uint8))
