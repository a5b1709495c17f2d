"""Host-side refusals of the rotary, paged-cache and single-token attention
calls (no GPU: every call is refused, or is empty, before any launch)."""
import ctypes

import pytest
import torch

from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U


@pytest.fixture(scope="module")
def L():
    B.build()
    return U.lib()


P = ctypes.c_void_p
X, Y, Z, W = (P(i << 32) for i in (1, 2, 3, 4))     # far apart, aligned, never dereferenced


def _rope(L, items=None, n=None, pos=X, n_axes=1, freq=(1.0,) * 64, axes=None, rot=128, pairs=0, S=4, B=1, D=128,
          dt=U.BF16, out=U.BF16, fn="fwd"):
    items = [U.RopeItem(X.value, Y.value, 2, 0, 256, 128, 0, 256, 128)] if items is None else items
    arr = (U.RopeItem * max(1, len(items)))(*items)
    f = (ctypes.c_double * len(freq))(*freq)
    ax = None if axes is None else (ctypes.c_int32 * len(axes))(*axes)
    return getattr(L, f"ulysses_rope_{fn}")(arr, len(items) if n is None else n, pos, n_axes, f, ax, rot, pairs, S, B, D,
                                            dt, out, None)


def test_rope_refusals(L):
    launches = L.ulysses_launch_count()
    item = lambda **k: U.RopeItem(**{**dict(src=X.value, dst=Y.value, H=2, src_b=0, src_s=256, src_h=128, dst_b=0,  # noqa: E731
                                            dst_s=256, dst_h=128), **k})
    assert _rope(L, dt=7) == U.ERR_INVALID
    assert _rope(L, dt=U.BF16, out=U.FP32) == U.ERR_UNSUPPORTED
    assert _rope(L, dt=U.E4M3, out=U.E4M3) == U.ERR_INVALID
    assert _rope(L, D=96, rot=96) == U.ERR_UNSUPPORTED
    for rot in (0, 8, 24, 144):
        assert _rope(L, rot=rot) == U.ERR_INVALID
    assert _rope(L, pairs=2) == U.ERR_INVALID
    assert _rope(L, n_axes=0) == U.ERR_INVALID and _rope(L, n_axes=5) == U.ERR_INVALID
    assert _rope(L, axes=[1] * 64) == U.ERR_INVALID and _rope(L, axes=[-1] * 64) == U.ERR_INVALID
    assert _rope(L, freq=(float("inf"),) * 64) == U.ERR_INVALID
    assert _rope(L, freq=(float("nan"),) * 64, fn="bwd") == U.ERR_INVALID
    assert _rope(L, n=5) == U.ERR_INVALID and _rope(L, n=-1) == U.ERR_INVALID
    assert _rope(L, S=-1) == U.ERR_INVALID and _rope(L, B=0) == U.ERR_INVALID
    assert _rope(L, S=1 << 31) == U.ERR_UNSUPPORTED
    assert _rope(L, pos=None) == U.ERR_INVALID
    assert _rope(L, [item(H=0)]) == U.ERR_INVALID
    assert _rope(L, [item(src=0)]) == U.ERR_INVALID
    assert _rope(L, [item(src=X.value + 8)]) == U.ERR_INVALID               # not 16-byte aligned
    assert _rope(L, [item(src_h=132)]) == U.ERR_UNSUPPORTED                 # strides of 16 bytes
    assert _rope(L, [item(src_s=-256)]) == U.ERR_UNSUPPORTED
    assert _rope(L, [item(src_s=1 << 60)]) == U.ERR_UNSUPPORTED
    assert _rope(L, [item(dst_s=0)]) == U.ERR_INVALID                       # rows written over each other
    assert _rope(L, [item(dst_s=128)]) == U.ERR_INVALID
    assert _rope(L, [item(dst=X.value + 256)]) == U.ERR_INVALID             # overlap that is not in place
    assert _rope(L, [item(dst=X.value, dst_s=512)]) == U.ERR_INVALID        # in place with other strides
    one = item(dst=X.value)
    assert _rope(L, [one], dt=U.FP32, out=U.BF16) == U.ERR_INVALID          # in place with another type
    assert _rope(L, [one, item(src=Z.value, dst=X.value)]) == U.ERR_INVALID  # two outputs in one place
    assert _rope(L, [item(dst=Z.value), item(src=Z.value, dst=W.value)]) == U.ERR_INVALID
    # K's heads overlapping Q's in one row: q 2 heads at 0, k 1 head at 1 of rows of 4
    q = item(dst=X.value, src_s=512, dst_s=512)
    k = item(src=X.value + 256, dst=X.value + 256, H=1, src_s=512, dst_s=512)
    assert _rope(L, [q, k]) == U.ERR_INVALID
    assert b"overlaps" in L.ulysses_last_error()
    # nothing to do
    assert _rope(L, S=0) == U.OK and _rope(L, n=0) == U.OK
    assert L.ulysses_launch_count() == launches


def _write(L, k=X, v=Y, k_s=256, k_h=128, v_s=256, v_h=128, T=4, B=4, cu=None, table=X, cols=8, lens=X, kc=Z, vc=W,
           ks=None, vs=None, pages=64, page=16, H=2, D=128, dt=U.BF16, cd=U.BF16):
    return L.ulysses_cache_write(k, v, k_s, k_h, v_s, v_h, T, B, cu, table, cols, lens, kc, vc, ks, vs, pages, page, H, D,
                                 dt, cd, None)


def _read(L, k=X, v=Y, k_s=256, k_h=128, v_s=256, v_h=128, T=4, B=4, cu=X, table=X, cols=8, first=None, kc=Z, vc=W,
          ks=None, vs=None, pages=64, page=16, H=2, D=128, dt=U.BF16, cd=U.BF16):
    return L.ulysses_cache_read(kc, vc, ks, vs, table, cols, cu, first, k, v, k_s, k_h, v_s, v_h, T, B, pages, page, H, D,
                                dt, cd, None)


def test_cache_refusals(L):
    launches = L.ulysses_launch_count()
    for f in (_write, _read):
        assert f(L, dt=U.E4M3, cd=U.E4M3, ks=X, vs=X) == U.ERR_INVALID      # rows are bf16 or fp32
        assert f(L, dt=U.BF16, cd=U.FP32) == U.ERR_UNSUPPORTED
        assert f(L, cd=9) == U.ERR_INVALID
        assert f(L, cd=U.E4M3) == U.ERR_INVALID                             # no scales
        assert f(L, cd=U.E4M3, ks=X) == U.ERR_INVALID
        assert f(L, ks=X, vs=X) == U.ERR_INVALID                            # scales without codes
        assert f(L, D=80) == U.ERR_UNSUPPORTED
        for page in (0, 8, 24, -16, 1 << 21):
            assert f(L, page=page) == U.ERR_UNSUPPORTED
        assert f(L, cols=(1 << 26) + 1) == U.ERR_UNSUPPORTED                # positions above 2^30
        assert f(L, H=0) == U.ERR_INVALID and f(L, pages=-1) == U.ERR_INVALID and f(L, B=-1) == U.ERR_INVALID
        assert f(L, T=-1) == U.ERR_INVALID
        assert f(L, kc=None) == U.ERR_INVALID and f(L, k=None) == U.ERR_INVALID and f(L, table=None) == U.ERR_INVALID
        assert f(L, k=P(X.value + 4)) == U.ERR_INVALID and f(L, vc=P(W.value + 8)) == U.ERR_INVALID
        assert f(L, k_s=260) == U.ERR_UNSUPPORTED and f(L, v_h=-128) == U.ERR_UNSUPPORTED
        assert f(L, k=Z) == U.ERR_INVALID                                   # rows inside the cache
        assert f(L, T=0, cu=X) == U.OK and f(L, B=0, T=0) == U.OK
    assert _write(L, T=5) == U.ERR_INVALID                                  # one token per sequence
    assert _write(L, lens=None) == U.ERR_INVALID
    assert _write(L, vc=Z) == U.ERR_INVALID                                 # one buffer for both caches
    assert _read(L, cu=None) == U.ERR_INVALID
    assert _read(L, k_s=0) == U.ERR_INVALID                                 # rows written over each other
    assert _read(L, v=X) == U.ERR_INVALID
    assert L.ulysses_launch_count() == launches


def _decode(L, q=X, q_b=512, q_h=128, kc=Z, vc=W, ks=None, vs=None, table=X, cols=8, lens=X, o=Y, o_b=512, o_h=128,
            lse=X, B=4, Hq=4, Hkv=2, D=128, pages=64, page=16, scale=0.0, dt=U.BF16, cd=U.BF16, ws=None, n=None):
    need = L.ulysses_attn_decode_workspace(B, Hq, Hkv, D, cols, page, dt, cd) if n is None else n
    return L.ulysses_attn_decode(q, q_b, q_h, kc, vc, ks, vs, table, cols, lens, o, o_b, o_h, lse, B, Hq, Hkv, D, pages,
                                 page, scale, dt, cd, P(256) if ws is None and need else ws, need, None)


def test_decode_refusals(L):
    launches = L.ulysses_launch_count()
    assert _decode(L, Hq=5) == U.ERR_INVALID
    assert _decode(L, Hq=0) == U.ERR_INVALID
    assert _decode(L, D=96) == U.ERR_UNSUPPORTED
    assert _decode(L, cd=U.FP32) == U.ERR_UNSUPPORTED
    assert _decode(L, cd=U.E4M3) == U.ERR_INVALID
    assert _decode(L, page=20) == U.ERR_UNSUPPORTED
    assert _decode(L, B=1 << 23) == U.ERR_UNSUPPORTED
    for k in ("q", "o", "lens", "table"):
        assert _decode(L, **{k: None}) == U.ERR_INVALID
    assert _decode(L, q=P(X.value + 2)) == U.ERR_INVALID
    assert _decode(L, q_h=100) == U.ERR_UNSUPPORTED
    assert _decode(L, o_b=128) == U.ERR_INVALID                             # rows written over each other
    assert _decode(L, o=X) == U.ERR_INVALID                                 # O over Q
    need = L.ulysses_attn_decode_workspace(4, 4, 2, 128, 8, 16, U.BF16, U.BF16)
    if need:
        assert _decode(L, n=need - 1) == U.ERR_INVALID
        assert _decode(L, ws=P(264)) == U.ERR_INVALID
    # more units of 16 keys in one sequence's table than 31 bits count
    assert _decode(L, Hq=64, Hkv=64, q_b=64 * 128, o_b=64 * 128, o=P(1 << 40), cols=1 << 26) == U.ERR_UNSUPPORTED
    assert _decode(L, B=0) == U.OK
    assert L.ulysses_launch_count() == launches


def test_binding_refuses_on_the_host():
    t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    f, ax = U.rope_frequencies(128, sections=[16, 24, 24])
    assert f.shape == (64,) and ax.tolist() == [0] * 16 + [1] * 24 + [2] * 24
    with pytest.raises(ValueError):
        U.rope_frequencies(128, sections=[16, 24])
    with pytest.raises(ValueError, match="CUDA"):
        U.rope_fwd(t, None, torch.zeros(4, dtype=torch.int32), f)
    with pytest.raises(ValueError):
        U.rope_fwd(None, None, torch.zeros(4, dtype=torch.int32), f)
    kc, vc, ks, vs = U.kv_cache(4, 16, 2, 128, torch.float8_e4m3fn, device="cpu")
    assert kc.shape == (4, 2, 16, 128) and ks.shape == (4, 2, 16) and ks.dtype == torch.float32
    with pytest.raises(ValueError, match="CUDA"):
        U.cache_write(t, t, kc, vc, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32),
                      k_scale=ks, v_scale=vs)
    with pytest.raises(ValueError, match="one shape"):
        U.cache_write(t, t[:2], kc, vc, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="heads or D"):
        U.cache_write(t[:, :1], t[:, :1], kc, vc, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        U.attn_decode(t, kc, vc, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32))
    with pytest.raises(ValueError, match="layout"):
        U.attn_decode(t, kc, vc, torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32), layout="bshd")
