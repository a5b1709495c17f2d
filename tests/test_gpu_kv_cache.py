"""The paged key-value cache (ulysses_cache_write / _read) against the fp64
definition: which place a row goes to, what is stored there, and that nothing
else is touched.

Stored rows are copies, bit for bit.  8-bit rows: scale and 448 / amax are one
fp32 division each (2^-24), the product another rounding, so code * scale is
off by half an e4m3 step (2^-4 of the value, and 2^-10 scale units below
2^-6 units) plus 3 * 2^-24 of the value that is rounded."""
import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.detach().float().double().cpu().numpy()


def normal(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def table(pages, seed=0, spare=3):
    """Pages in a mixed order; entries of no page hold a wild id."""
    total = sum(pages)
    order = np.random.default_rng(seed).permutation(total + spare)[:total]
    t = np.full((len(pages), max(pages) + 2), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(pages):
        t[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), total + spare


def fill(bufs):
    """Every byte a pattern (a NaN as fp32 or bf16)."""
    for x in bufs:
        if x is not None:
            x.view(torch.uint8).fill_(0xFF)


CASES = [
    # new tokens per sequence, tokens there before, pad rows, H, D, page, dtype, cache, layout
    ([1], [0], 0, 1, 128, 16, "bf16", "bf16", "seq"),
    ([1, 1, 1], [4, 15, 16], 0, 8, 128, 16, "bf16", "e4m3", "head"),
    ([5, 0, 40, 1], [0, 9, 30, 31], 3, 2, 64, 32, "bf16", "e4m3", "seq"),
    ([100, 0, 0, 333], [1, 0, 0, 77], 0, 3, 128, 48, "fp32", "e4m3", "seq"),
    ([17, 64], [0, 0], 1, 4, 64, 64, "fp32", "fp32", "head"),
    ([1500, 700], [100, 3], 5, 8, 128, 64, "bf16", "bf16", "head"),
    ([9000], [17], 0, 2, 128, 256, "bf16", "e4m3", "head"),
    ([130, 1, 258], [0, 0, 0], 0, 5, 64, 16, "fp32", "e4m3", "head"),
]


@pytest.mark.parametrize("new,before,pad,H,D,page,dtype,cache,layout", CASES)
def test_write_then_read(new, before, pad, H, D, page, dtype, cache, layout):
    B, n = len(new), sum(new)
    lens = [a + b for a, b in zip(new, before)]
    tab, pages = table([max(1, -(-x // page)) for x in lens])
    bufs = U.kv_cache(pages, page, H, D, DT[cache])
    fill(bufs)
    kc, vc, ks, vs = bufs
    T = n + pad
    shape = (T, H, D) if layout == "seq" else (H, T, D)
    k, v = normal(shape, 1, dtype), normal(shape, 2, dtype)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    U.cache_write(k, v, kc, vc, tab, ln, cu_new=cu, k_scale=ks, v_scale=vs, layout=layout)
    U.check()
    first = torch.tensor(before, dtype=torch.int32, device="cuda")
    out = [torch.full(shape, 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    got = U.cache_read(kc, vc, tab, cu, T, first=first, k_scale=ks, v_scale=vs, layout=layout, out=out)
    U.check()
    tr = (lambda a: a.transpose(1, 0, 2)) if layout == "head" else (lambda a: a)
    t_np = tab.cpu().numpy()
    for x, c, s, back in ((k, kc, ks, got[0]), (v, vc, vs, got[1])):
        X, R = tr(f64(x)), tr(f64(back))
        raw = c.view(torch.uint8).cpu().numpy().reshape(pages, H, page, -1)
        touched = np.zeros((pages, page), bool)
        codes = c.float().cpu().numpy()
        scales = None if s is None else s.cpu().numpy()
        t = 0
        for b in range(B):
            for i in range(new[b]):
                pg, sl = so.place(t_np, page, b, before[b] + i)
                touched[pg, sl] = True
                if cache != "e4m3":
                    assert np.array_equal(codes[pg, :, sl], X[t])
                else:
                    _, ws = so.quantise(X[t])
                    assert np.allclose(scales[pg, :, sl], ws, rtol=2.0 ** -23)
                    value = codes[pg, :, sl].astype(np.float64) * scales[pg, :, sl, None]
                    lim = np.maximum(np.abs(X[t]) * 2.0 ** -4, ws[:, None] * 2.0 ** -10) + np.abs(X[t]) * 2.0 ** -21
                    assert np.all(np.abs(value - X[t]) <= lim)
                    # the codes themselves: the same two fp32 roundings (448 / amax, x * that), then e4m3
                    x32 = X[t].astype(np.float32)
                    inv = np.float32(448.0) / np.abs(x32).max(-1, keepdims=True)
                    assert np.array_equal(codes[pg, :, sl], so.e4m3(x32 * inv))
                t += 1
        # untouched slots keep their bytes
        assert np.all(raw.transpose(0, 2, 1, 3)[~touched] == 0xFF)
        if s is not None:
            assert np.all(np.isnan(scales.transpose(0, 2, 1)[~touched]))
        # read back: the stored value, rounded once; rows behind the last sequence stay
        assert np.all(R[n:] == 7.0)
        t = 0
        for b in range(B):
            rows = so.cache_rows(c.float().cpu().numpy(), t_np, b, new[b], before[b]).astype(np.float64)
            if s is not None:
                sc = so.cache_rows(scales[..., None], t_np, b, new[b], before[b])[..., 0]
                rows = (rows.astype(np.float32) * sc[..., None]).astype(np.float64)
            if dtype == "bf16":
                rows = f64(torch.from_numpy(rows).float().bfloat16())
            assert np.array_equal(R[t:t + new[b]], rows)
            t += new[b]


def test_one_token_per_sequence_with_empty_places():
    H, D, page, B = 2, 128, 16, 5
    lens = [0, 1, 16, 17, 0]
    tab, pages = table([max(1, -(-x // page)) for x in lens])
    kc, vc, _, _ = U.kv_cache(pages, page, H, D)
    fill((kc, vc))
    k, v = normal((B, H, D), 1, "bf16"), normal((B, H, D), 2, "bf16")
    U.cache_write(k, v, kc, vc, tab, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    U.check()
    t_np = tab.cpu().numpy()
    left = torch.ones((pages, page), dtype=torch.bool)
    for b, n in enumerate(lens):
        if n:
            pg, sl = so.place(t_np, page, b, n - 1)
            left[pg, sl] = False
            assert torch.equal(kc[pg, :, sl], k[b]) and torch.equal(vc[pg, :, sl], v[b])
    for c in (kc, vc):
        assert bool((c.view(torch.uint8).view(pages, H, page, -1).transpose(1, 2).cpu()[left] == 0xFF).all())


def test_rows_that_are_not_ordinary():
    """Zeros, the smallest and the largest numbers, infinities and NaN."""
    D = 64
    x = torch.zeros((8, 1, D), device="cuda")
    x[1] = 1e-45                                     # the smallest subnormal: below the floor of the scale
    x[2] = 3.3e38
    x[3, 0, ::2] = 1e-38
    x[4, 0, 5] = float("inf")
    x[5, 0, 6] = float("nan")
    x[6, 0, 7] = -float("inf")
    x[7, 0, 0], x[7, 0, 1] = -448.0, 1.0
    tab = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    kc, vc, ks, vs = U.kv_cache(1, 16, 1, D, torch.float8_e4m3fn)
    cu = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    U.cache_write(x, x, kc, vc, tab, torch.tensor([8], dtype=torch.int32, device="cuda"), cu_new=cu, k_scale=ks, v_scale=vs)
    k, v = U.cache_read(kc, vc, tab, cu, 8, k_scale=ks, v_scale=vs, dtype=torch.float32)
    U.check()
    assert torch.equal(k[:4], v[:4])
    assert bool((k[0] == 0).all()) and bool(torch.isfinite(k[:4]).all())
    assert bool((k[1].abs() <= 1e-37).all())
    assert bool(((k[2] / 3.3e38 - 1).abs() <= 2.0 ** -4).all())
    # its row's scale is that of 2^-100: 1e-38 is far below one step of it
    assert bool((k[3].abs() <= 2.0 ** -100 / 448).all())
    for r in (4, 5, 6):
        assert bool(torch.isnan(k[r]).all()), r
    assert k[7, 0, 0] == -448 and k[7, 0, 1] == 1


def test_strided_rows_of_a_fused_projection():
    Hq, H, T, D = 4, 2, 37, 128
    x = normal((T, Hq + 2 * H, D), 3, "bf16")
    k, v = x[:, Hq:Hq + H], x[:, Hq + H:]
    tab, pages = table([3])
    kc, vc, _, _ = U.kv_cache(pages, 16, H, D)
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    ln = torch.tensor([T], dtype=torch.int32, device="cuda")
    U.cache_write(k, v, kc, vc, tab, ln, cu_new=cu)
    back = torch.zeros_like(x)
    U.cache_read(kc, vc, tab, cu, T, out=(back[:, Hq:Hq + H], back[:, Hq + H:]))
    U.check()
    assert torch.equal(back[:, Hq:], x[:, Hq:]) and bool((back[:, :Hq] == 0).all())


@pytest.mark.parametrize("what", ["page", "negative", "length", "short"])
def test_bad_places_are_reported_and_skipped(what):
    H, D, page = 1, 64, 16
    tab = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    if what == "page":
        tab[1, 1] = 4
    elif what == "negative":
        tab[1, 1] = -1
    elif what == "length":
        lens[1] = 34                                 # one position past the table, one inside
    else:
        lens[1] = 1                                  # two new tokens, one position
    kc, vc, _, _ = U.kv_cache(4, page, H, D)
    x = normal((4, H, D), 4, "bf16") + 100.0         # no zeros
    U.cache_write(x, x, kc, vc, tab, lens, cu_new=cu)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    U.check()                                        # reported once
    assert torch.equal(kc[1, 0, 2:4], x[:2, 0])
    rows = int((kc[:, 0, :, 0] != 0).sum())
    assert rows == (2 if what in ("page", "negative", "length") else 3)
    out = [torch.full((4, H, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    first = torch.tensor([18, 18 if what in ("page", "negative") else 31], dtype=torch.int32, device="cuda")
    U.cache_read(kc, vc, tab, cu, 4, first=first, out=out)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    assert torch.equal(out[0][:2], x[:2]) and bool((out[0][3] == 7.0).all())


def test_malformed_cu_is_reported():
    tab = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    tab[1] = 1
    kc, vc, _, _ = U.kv_cache(2, 16, 1, 64)
    x = normal((4, 1, 64), 5, "bf16")
    for bad in ([0, 3, 2], [1, 2, 4], [0, 2, 5]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        U.cache_write(x, x, kc, vc, tab, torch.tensor([4, 4], dtype=torch.int32, device="cuda"), cu_new=cu)
        with pytest.raises(U.UlyssesError) as e:
            U.check()
        assert e.value.code in (U.ERR_BAD_SEQLENS, U.ERR_BAD_PAGES)
    U.check()


def test_pages_beyond_32_bit_offsets():
    """A cache of more than 2^32 elements: the last pages are as good as the first."""
    H, D, page = 8, 128, 256
    pages = (1 << 32) // (H * D * page) + 40
    kc = torch.empty((pages, H, page, D), dtype=torch.float8_e4m3fn, device="cuda")
    vc = torch.empty_like(kc)
    ks = torch.empty((pages, H, page), device="cuda")
    vs = torch.empty_like(ks)
    tab = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device="cuda")
    T = 600
    k, v = normal((T, H, D), 6, "bf16"), normal((T, H, D), 7, "bf16")
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    U.cache_write(k, v, kc, vc, tab, cu[1:], cu_new=cu, k_scale=ks, v_scale=vs)
    a, b = U.cache_read(kc, vc, tab, cu, T, k_scale=ks, v_scale=vs)
    U.check()
    for x, y in ((k, a), (v, b)):
        err = (x.float() - y.float()).abs()
        assert bool((err <= x.float().abs() * (2.0 ** -4 + 2.0 ** -8) + x.float().abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10).all())


def test_write_and_read_on_a_stream_of_their_own():
    st = torch.cuda.Stream()
    kc, vc, _, _ = U.kv_cache(8, 16, 2, 64)
    k, v = normal((2, 100, 64), 8, "bf16"), normal((2, 100, 64), 9, "bf16")
    tab = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    st.wait_stream(torch.cuda.current_stream())
    U.cache_write(k, v, kc, vc, tab, cu[1:], cu_new=cu, layout="head", stream=st)
    a, b = U.cache_read(kc, vc, tab, cu, 100, layout="head", stream=st)
    st.synchronize()
    assert torch.equal(a, k) and torch.equal(b, v)


def test_many_heads_and_many_tokens_of_a_block():
    """Blocks of the largest and of the smallest number of tokens."""
    for T, H, D in ((40000, 1, 64), (3, 300, 128)):
        kc, vc, ks, vs = U.kv_cache(-(-T // 64), 64, H, D, torch.float8_e4m3fn)
        k, v = normal((T, H, D), 10, "bf16"), normal((T, H, D), 11, "bf16")
        tab = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None]
        cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        U.cache_write(k, v, kc, vc, tab, cu[1:], cu_new=cu, k_scale=ks, v_scale=vs)
        a, b = U.cache_read(kc, vc, tab, cu, T, k_scale=ks, v_scale=vs, dtype=torch.float32)
        U.check()
        for x, y in ((k, a), (v, b)):
            x = x.float()
            lim = torch.maximum(x.abs() * 2.0 ** -4, x.abs().amax(-1, keepdim=True) / 448 * 2.0 ** -10) + x.abs() * 2.0 ** -21
            assert bool(((x - y).abs() <= lim).all())
