"""The calls of the 4-bit cache, the attention weights and eviction: the C++
marshalling against the Python one, wrong tensors in every place, windows of
memory with guards around, offsets beyond 32 bits, two calls at once."""
import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

from tests.test_gpu_4bit import build4, check4, f64, unpack
from tests.test_gpu_evict import HELD, expect, i32, make, parts

pytestmark = pytest.mark.gpu


def same(a, b):
    a, b = (x if isinstance(x, (tuple, list)) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.dtype == y.dtype and x.stride() == y.stride()
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("layout", ["seq", "head"])
@pytest.mark.parametrize("held", ["bf16", "e4m3", "e2m1"])
def test_cpp_and_python_marshalling_agree(monkeypatch, held, layout):
    U.lib()
    assert U._fast is not None
    B, Hq, H, D, page = 3, 6, 2, 64, 16
    lens, cu = i32([40, 0, 7]), i32([0, 40, 40, 47])
    tab = torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4)
    g = torch.Generator().manual_seed(0)
    x = torch.randn((47, 2 * H, D) if layout == "seq" else (2 * H, 47, D), generator=g).bfloat16().cuda()
    q = torch.randn((B, Hq, D) if layout == "seq" else (Hq, B, D), generator=g).bfloat16().cuda()
    k, v = (x[:, :H], x[:, H:]) if layout == "seq" else (x[:H], x[H:])

    def calls():
        kc, vc, ks, vs = U.kv_cache(12, page, H, D, HELD[held])
        w = U.cache_weights(kc).fill_(5.0)
        kw = dict(k_scale=ks, v_scale=vs)
        assert U.cache_write(k, v, kc, vc, tab, lens, cu_new=cu, layout=layout, weights=w, **kw) is None
        got = [*U.cache_read(kc, vc, tab, cu, 47, layout=layout, **kw)]
        got += U.attn_decode(q, kc, vc, tab, lens, layout=layout, weights=w, **kw)
        got.append(U.cache_evict(kc, vc, w, tab, lens, i32([20, 1, 7]), recent=3, **kw))
        out, ws = i32([0, 0, 0]), U.cache_evict_workspace(kc, tab)
        assert U.cache_evict(kc, vc, w, tab, got[-1], i32([10, 1, 6]), 3, ks, vs, out, ws) is out
        return got + [t.clone() for t in (out, w, kc, vc) + ((ks, vs) if ks is not None else ())]

    with monkeypatch.context() as m:
        m.setattr(U, "_launch", lambda *a: pytest.fail("the plain call went through Python"))
        fast = calls()
    with monkeypatch.context() as m:
        m.setattr(U, "_fast", None)
        same(fast, calls())
    U.check()


def test_wrong_tensors_are_refused():
    a = make([40, 9], 2, 64, 16, "e2m1", seed=0)
    args = dict(a, keep=i32([10, 5]), out=i32([0, 0]), workspace=U.cache_evict_workspace(a["k_cache"], a["page_table"]))
    launches, tried = U.launch_count(), 0
    for name, t in list(args.items()):
        bad = [t[:-1], t.cpu(), torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype, device="cuda")[..., ::2]]
        bad += [t.to(dt) for dt in (torch.int64, torch.float16, torch.uint8, torch.bool) if dt is not t.dtype]
        if name in ("seq_lens", "keep", "out", "workspace"):
            bad = bad[1:] if name == "workspace" else bad
        for b in bad:
            # a cache and scales cut alike would be a smaller cache: one of them alone never is
            with pytest.raises((ValueError, TypeError, U.UlyssesError)):
                U.cache_evict(**{**args, name: b})
            tried += 1
    with pytest.raises(U.UlyssesError):
        U.cache_evict(**args, recent=-1)
    assert U.launch_count() == launches and tried > 50
    q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    kw = {x: a[x] for x in ("k_cache", "v_cache", "page_table", "seq_lens", "k_scale", "v_scale")}
    w = a["weights"]
    for b in (w[:-1], w.double(), w.cpu(), w.transpose(0, 1), w.view(-1)):
        with pytest.raises((ValueError, TypeError, U.UlyssesError)):
            U.attn_decode(q, weights=b, **kw)
        with pytest.raises((ValueError, TypeError, U.UlyssesError)):
            U.cache_write(q[:, :2], q[:, 2:], weights=b, **kw)
    assert U.launch_count() == launches
    U.check()


def test_recent_of_any_size():
    a = make([100], 1, 64, 16, "bf16", seed=2)
    for recent in (1 << 31, 1 << 40):
        b = {x: t.clone() if t is not None else None for x, t in a.items()}
        want, new = expect(b, [100], [30], 1 << 20)
        assert U.cache_evict(keep=i32([30]), recent=recent, **b).tolist() == new
        got = parts(b)
        assert all(np.array_equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("held", ["bf16", "e4m3", "e2m1"])
def test_nothing_outside_the_buffers_is_written(held):
    """Every buffer is a window of a larger one filled with a pattern."""
    guard, pat, B, H, D, page = 4096, 0xC7, 2, 2, 128, 16
    raws = []

    def window(shape, dtype):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((2 * guard + (n + 255) // 256 * 256,), pat, dtype=torch.uint8, device="cuda")
        raws.append((raw, n))
        return raw[guard:guard + n].view(dtype).view(shape)

    width = 9 * D // 16 if held == "e2m1" else D
    kc, vc = (window((8, H, page, width), HELD[held]) for _ in range(2))
    ks, vs = (window((8, H, page), torch.float32) if held != "bf16" else None for _ in range(2))
    w = window((8, H, page), torch.float32)
    for t in (kc, vc, w) + ((ks, vs) if ks is not None else ()):
        t.view(torch.uint8).zero_()
    tab = torch.tensor([[3, 0, 7, 1], [5, 2, 6, 4]], dtype=torch.int32, device="cuda")
    x = torch.randn((100, 2 * H, D), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    lens, kw = i32([61, 39]), dict(k_scale=ks, v_scale=vs)
    U.cache_write(x[:, :H], x[:, H:], kc, vc, tab, lens, cu_new=i32([0, 61, 100]), weights=w, **kw)
    q = x[:B, :1].repeat(1, 8, 1)
    for t in (tab, torch.cat((tab, torch.full((B, 3000), -1, dtype=torch.int32, device="cuda")), 1)):
        n = U.attn_decode_workspace(q, kc, t, weights=True).numel()
        o, lse = window((B, 8, D), torch.bfloat16), window((B, 8), torch.float32)
        U.attn_decode(q, kc, vc, t, lens, weights=w, out=o, lse=lse, workspace=window((n,), torch.uint8) if n else None, **kw)
        n = U.cache_evict_workspace(kc, t).numel()
        U.cache_evict(kc, vc, w, t, lens, i32([50, 39]), recent=7, out=window((B,), torch.int32), workspace=window((n,), torch.uint8), **kw)
    U.check()
    for raw, n in raws:
        assert bool((raw[:guard] == pat).all()) and bool((raw[guard + n:] == pat).all())


def test_cache_beyond_32_bit_offsets():
    """4-bit pages whose bytes, and whose rows' scales, lie beyond 2^32 bytes."""
    H, D, page, n = 8, 128, 256, 700
    pages = (1 << 32) // (H * page * 72) + 40
    kc, vc = (torch.zeros((pages, H, page, 72), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs, w = (torch.zeros((pages, H, page), device="cuda") for _ in range(3))
    at = [pages - 1, 1, pages - 2]
    tab = i32([at])
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn((n, H, D), generator=g).bfloat16().cuda() for _ in range(2))
    cu, sc = i32([0, n]), dict(k_scale=ks, v_scale=vs)
    U.cache_write(k, v, kc, vc, tab, cu[1:], cu_new=cu, weights=w, **sc)
    q = torch.randn((1, 32, D), generator=g).bfloat16().cuda()
    rows = lambda m: [so.cache_rows(so.values4(*unpack(c[at], page, D), f64(s[at])), [[0, 1, 2]], 0, m)   # noqa: E731
                      for c, s in ((kc, ks), (vc, vs))]
    before = rows(n)
    o, lse = U.attn_decode(q, kc, vc, tab, cu[1:], weights=w, **sc)
    U.check()
    check4(o, lse, [(f64(q[0]), *before)], [so.cache_rows(f64(vs[at])[..., None], [[0, 1, 2]], 0, n)[..., 0]], "bf16", "seq")
    got = so.cache_rows(f64(w[at])[..., None], [[0, 1, 2]], 0, n)[..., 0]
    assert np.abs(got - so.attention_weights(f64(q[0]), before[0])).max() < 1e-5
    left = U.cache_evict(kc, vc, w, tab, cu[1:], i32([300]), recent=20, **sc)
    U.check()
    assert left.tolist() == [300]
    for old, new in zip(before, rows(300)):
        for h in range(H):
            assert np.array_equal(new[:, h], old[so.stays(got[:, h], 300, 20), h])
    rk, rv = U.cache_read(kc, vc, tab, i32([0, 300]), 300, dtype=torch.float32, **sc)
    assert np.array_equal(f64(rk), rows(300)[0]) and np.array_equal(f64(rv), rows(300)[1])
    del kc, vc, ks, vs, w
    torch.cuda.empty_cache()


def test_two_evictions_at_once_on_two_streams():
    """Sequences of their own in one cache, a workspace each."""
    lens, keep = [3000, 2500, 2800, 2000], [1500, 2499, 100, 1999]
    a = make(lens, 4, 64, 16, "e4m3", seed=4)
    want, new = expect(a, lens, keep, 50)
    kp, outs, wss, sub = i32(keep), [], [], []
    for i in range(2):
        rows = slice(2 * i, 2 * i + 2)
        sub.append(dict(a, page_table=a["page_table"][rows].contiguous(), seq_lens=a["seq_lens"][rows].contiguous()))
        wss.append(U.cache_evict_workspace(a["k_cache"], sub[i]["page_table"]))
        outs.append(i32([0, 0]))
    keeps = [kp[:2].contiguous(), kp[2:].contiguous()]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        U.cache_evict(keep=keeps[i], recent=50, out=outs[i], workspace=wss[i], stream=streams[i], **sub[i])
    torch.cuda.synchronize()
    U.check()
    got = parts(a)
    assert outs[0].tolist() + outs[1].tolist() == new and all(np.array_equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("held", ["bf16", "fp32", "e4m3"])
def test_written_tokens_begin_at_zero_weight(held):
    dt = torch.float32 if held == "fp32" else torch.bfloat16
    kc, vc, ks, vs = U.kv_cache(6, 16, 3, 64, HELD[held])
    w = U.cache_weights(kc).fill_(2.0)
    x = torch.randn((30, 3, 64), generator=torch.Generator().manual_seed(5)).to(dt).cuda()
    U.cache_write(x, x, kc, vc, i32([[4, 0], [1, 2]]), i32([25, 9]), cu_new=i32([0, 21, 30]), k_scale=ks, v_scale=vs, weights=w)
    want = torch.full((6, 3, 16), 2.0)
    for b, (tab, n, m) in enumerate((([4, 0], 25, 21), ([1, 2], 9, 9))):
        for p in range(n - m, n):
            want[tab[p // 16], :, p % 16] = 0.0
    assert torch.equal(w.cpu(), want)
    # one token a sequence, and an empty place
    w.fill_(2.0)
    U.cache_write(x[:2], x[:2], kc, vc, i32([[4, 0], [1, 2]]), i32([17, 0]), k_scale=ks, v_scale=vs, weights=w)
    U.check()
    want = torch.full((6, 3, 16), 2.0)
    want[0, :, 0] = 0.0
    assert torch.equal(w.cpu(), want)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_bf16_rows_that_are_no_numbers(bad):
    x = torch.randn((3, 2, 128), generator=torch.Generator().manual_seed(6)).bfloat16()
    x[1, 0, 77] = bad
    kc, vc, ks, vs = U.kv_cache(1, 16, 2, 128, torch.uint8)
    xd = x.cuda()
    U.cache_write(xd, xd, kc, vc, i32([[0]]), i32([3]), cu_new=i32([0, 3]), k_scale=ks, v_scale=vs)
    r, _ = U.cache_read(kc, vc, i32([[0]]), i32([0, 3]), 3, k_scale=ks, v_scale=vs)
    U.check()
    assert bool(r[1, 0].isnan().all()) and int(r.isnan().sum()) == 128
    good, _ = U.cache_read(kc, vc, i32([[0]]), i32([0, 1]), 1, k_scale=ks, v_scale=vs)
    codes, block, scale = so.quantise4(f64(x[:1]))
    assert np.array_equal(f64(good), so.values4(codes, block, scale))


def test_a_whole_range_of_bf16_rows():
    """Every exponent, and elements that fall on borders: codes by the definition."""
    rng = np.random.default_rng(7)
    n, D = 4000, 128
    x = rng.integers(-128, 129, (n, 1, D)) * 2.0 ** rng.integers(-6, 1, (n, 1, D)) * 2.0 ** rng.integers(-90, 110, (n, 1, 1))
    t = torch.from_numpy(x).bfloat16()
    page = 64
    kc, vc, ks, vs = U.kv_cache(-(-n // page), page, 1, D, torch.uint8)
    tab = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None].contiguous()
    d = t.cuda()
    U.cache_write(d, d, kc, vc, tab, i32([n]), cu_new=i32([0, n]), k_scale=ks, v_scale=vs)
    U.check()
    codes, block, scale = so.quantise4(f64(t)[:, 0])
    gc, gb = unpack(kc, page, D)
    gc, gb, gs = gc.reshape(-1, D)[:n], gb.reshape(-1, D // 16)[:n], f64(ks).reshape(-1)[:n]
    assert np.array_equal(gs, scale) and np.array_equal(gb, block)
    assert ((gc == codes) | (((gc | codes) & 7) == 0)).all()
    z = np.abs(f64(t)[:, 0] / scale[:, None] / np.repeat(np.where(block > 0, block, 1), 16, -1))
    assert np.isin(z, so.E2M1_BORDERS).sum() > 1000                          # the case is what it is meant to be


EDGES = ["clusters", "split"]


@pytest.mark.parametrize("how", EDGES)
@pytest.mark.parametrize("Hq", [4, 8, 16])
@pytest.mark.parametrize("above", [30.0, 200.0, 2000.0])
def test_one_key_far_above_the_others(above, Hq, how):
    """A late key's score far above all before it: the maximum moves in the middle of a piece."""
    n, D = 300, 128
    args, rows, scales = build4([n], Hq, 1, D, 16, "bf16", "seq", seed=3)
    if how == "split":
        wide = torch.full((1, 1 << 14), -1, dtype=torch.int32, device="cuda")
        wide[:, :args["page_table"].shape[1]] = args["page_table"]
        args["page_table"] = wide
    q, k, v = rows[0]
    j, tab = 233, args["page_table"].cpu().numpy()
    pg, sl = int(tab[0][j // 16]), j % 16
    gain = above / max(np.abs((k[j] @ q.T)).max() * D ** -0.5, 1e-3)
    e = 2.0 ** np.ceil(np.log2(gain))                        # a power of two, as row scales are
    args["k_scale"][pg, 0, sl] *= e
    k = k.copy()
    k[j] *= e
    o, lse = U.attn_decode(**args)
    U.check()
    check4(o, lse, [(q, k, v)], scales, "bf16", "seq")


@pytest.mark.parametrize("how", EDGES)
def test_a_sequence_whose_pages_are_all_bad_is_empty(how):
    args, rows, scales = build4([50, 40], 4, 1, 64, 16, "bf16", "seq", seed=8)
    args["page_table"][0] = -1
    if how == "split":
        wide = torch.full((2, 1 << 14), -1, dtype=torch.int32, device="cuda")
        wide[:, :args["page_table"].shape[1]] = args["page_table"]
        args["page_table"] = wide
    w = U.cache_weights(args["k_cache"])
    o, lse = U.attn_decode(weights=w, **args)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    assert bool((o[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())
    check4(o[1:], lse[1:], rows[1:], scales[1:], "bf16", "seq")
    assert abs(float(w.sum()) - 4.0) < 1e-4
