"""The C++ marshalling (_fastcall.so) and the Python one make the same calls:
same results, and everything that is not plain is left to Python."""
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U

pytestmark = pytest.mark.gpu


@pytest.fixture
def both(monkeypatch):
    """run(call): the results by C++ and by Python marshalling; the first must not need Python's launch."""
    U.lib()
    assert U._fast is not None, "_fastcall.so is not loaded"

    def run(call):
        with monkeypatch.context() as m:
            m.setattr(U, "_launch", lambda *a: pytest.fail("the plain call went through Python"))
            fast = call()
        with monkeypatch.context() as m:
            m.setattr(U, "_fast", None)
            slow = call()
        return fast, slow
    return run


def normal(*shape, seed=0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def same(a, b):
    a, b = (x if isinstance(x, tuple) else (x,) for x in (a, b))
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.dtype == y.dtype and x.stride() == y.stride()
        assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("layout", ["seq", "head"])
@pytest.mark.parametrize("four", [False, True])
def test_rope(both, layout, four):
    T, H, D = 21, 6, 128
    shape = ((2,) if four else ()) + ((T, H, D) if layout == "seq" else (H, T, D))
    x = normal(*shape)
    q, k = (x[..., :4, :], x[..., 4:, :]) if layout == "seq" else (x[..., :4, :, :], x[..., 4:, :, :])
    inv, axes = U.rope_frequencies(96, sections=[20, 28])
    pos = torch.randint(0, 9999, (2,) + ((2,) if four else ()) + (T,), dtype=torch.int32, device="cuda")
    same(*both(lambda: U.rope_fwd(q, k, pos, inv, axes, layout=layout)))
    same(*both(lambda: U.rope_fwd(None, k, pos[0], inv, None, layout=layout, pairs="adjacent")))
    g = x.float()
    same(*both(lambda: U.rope_bwd(g, None, pos, inv, axes, layout=layout, dtype=torch.bfloat16)))
    o = torch.empty_like(x)
    r, _ = both(lambda: U.rope_fwd(x, None, pos, inv, axes, layout=layout, out=o))
    assert r is o
    a, b = torch.empty_like(q), torch.empty_like(k)
    same(*both(lambda: tuple(t.clone() for t in U.rope_fwd(q, k, pos, inv, axes, layout=layout, out=(a, b)))))


@pytest.mark.parametrize("layout", ["seq", "head"])
@pytest.mark.parametrize("held", [torch.bfloat16, torch.float8_e4m3fn])
def test_cache_and_attention(both, layout, held):
    B, Hq, H, D, page = 3, 6, 2, 64, 16
    lens = torch.tensor([40, 0, 7], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 40, 47], dtype=torch.int32, device="cuda")
    tab = torch.arange(12, dtype=torch.int32, device="cuda").view(B, 4)
    x = normal(47, Hq + 2 * H, D) if layout == "seq" else normal(Hq + 2 * H, 47, D)
    k, v = (x[:, Hq:Hq + H], x[:, Hq + H:]) if layout == "seq" else (x[Hq:Hq + H], x[Hq + H:])

    def write():
        bufs = U.kv_cache(12, page, H, D, held)
        assert U.cache_write(k, v, bufs[0], bufs[1], tab, lens, cu_new=cu, k_scale=bufs[2], v_scale=bufs[3],
                             layout=layout) is None
        return tuple(t for t in bufs if t is not None)
    a, b = both(write)
    same(a, b)
    kc, vc, ks, vs = a if len(a) == 4 else (*a, None, None)
    kw = dict(k_scale=ks, v_scale=vs, layout=layout)
    same(*both(lambda: U.cache_read(kc, vc, tab, cu, 47, **kw)))
    first = torch.tensor([3, 0, 0], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, 30, 30, 36], dtype=torch.int32, device="cuda")
    out = [torch.zeros((36, H, D) if layout == "seq" else (H, 36, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    same(*both(lambda: tuple(t.clone() for t in U.cache_read(kc, vc, tab, cut, 36, first=first, out=tuple(out), **kw))))
    q = normal(B, Hq, D, seed=1) if layout == "seq" else normal(Hq, B, D, seed=1)
    wide = torch.full((B, 1 << 14), -1, dtype=torch.int32, device="cuda")
    wide[:, :4] = tab
    for t in (tab, wide):
        same(*both(lambda: U.attn_decode(q, kc, vc, t, lens, **kw)))
        ws = U.attn_decode_workspace(q, kc, t, layout=layout)
        o, lse = torch.empty_like(q), torch.empty((B, Hq), device="cuda")
        r, _ = both(lambda: U.attn_decode(q, kc, vc, t, lens, scale=0.2, workspace=ws if ws.numel() else None, out=o,
                                          lse=lse, **kw))
        assert r[0] is o and r[1] is lse
    U.check()


def test_errors_are_python_s_or_the_library_s():
    x = normal(4, 2, 128)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(128)
    U.rope_fwd(x, None, pos, inv, axes)
    assert U._fast is not None
    # left to Python: None, whatever is not plain
    for bad in (dict(q=x.cpu()), dict(positions=pos.long()), dict(positions=pos[:3]), dict(inv_freq=inv.float()),
                dict(layout="x"), dict(layout=None), dict(pairs=3), dict(q=x[..., ::2]), dict(q=x.half()), dict(out=[x]),
                dict(out=(x, x)), dict(q="x"), dict(q=x[:0])):
        a = {**dict(q=x, k=None, positions=pos, inv_freq=inv, axes=axes, layout="seq", pairs="half", dtype=None, out=None),
             **bad}
        assert U._fast.rope(False, *a.values()) is None, bad
    # the library's refusal, as its code
    with pytest.raises(U.UlyssesError) as e:
        U.rope_fwd(x, x, pos, inv, axes, out=(x, x))
    assert e.value.code == U.ERR_INVALID
    with pytest.raises(U.UlyssesError) as e:
        U.rope_fwd(x, None, pos, inv, torch.full((64,), 3, dtype=torch.int32))
    assert e.value.code == U.ERR_INVALID
    with pytest.raises(TypeError):
        U._fast.rope(False)
    torch.cuda.synchronize()
