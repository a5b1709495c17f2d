"""Host-side refusals of the 4-bit cache, the attention weights of cached tokens
and eviction (no GPU: every call is refused, or is empty, before any launch)."""
import ctypes

import pytest
import torch

from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U

P = ctypes.c_void_p
KC, VC, KS, VS, W, TAB, LENS, KEEP, OUT, WS, X, Y = (P(i << 36) for i in range(1, 13))   # far apart, aligned, never read


@pytest.fixture(scope="module")
def L():
    B.build()
    return U.lib()


def _evict(L, kc=KC, vc=VC, ks=None, vs=None, w=W, table=TAB, cols=8, lens=LENS, keep=KEEP, recent=4, out=OUT, B=4, pages=64,
           page=16, H=2, D=128, cd=U.BF16, ws=WS, n=None):
    n = L.ulysses_cache_evict_workspace(B, H, cols, page) if n is None else n
    return L.ulysses_cache_evict(kc, vc, ks, vs, w, table, cols, lens, keep, recent, out, B, pages, page, H, D, cd, ws, n, None)


def test_evict_refusals(L):
    launches = L.ulysses_launch_count()
    assert _evict(L, cd=9) == U.ERR_INVALID
    for cd in (U.E4M3, U.E2M1):
        assert _evict(L, cd=cd) == U.ERR_INVALID                             # no scales
        assert _evict(L, cd=cd, ks=KS) == U.ERR_INVALID
    assert _evict(L, ks=KS, vs=VS) == U.ERR_INVALID                          # scales without codes
    assert _evict(L, D=96) == U.ERR_UNSUPPORTED
    for page in (0, 8, 24, -16, 1 << 21):
        assert _evict(L, page=page, n=1 << 30) == U.ERR_UNSUPPORTED
    assert _evict(L, cols=(1 << 26) + 1, n=1 << 30) == U.ERR_UNSUPPORTED
    assert _evict(L, cols=1 << 22, B=2048, H=8, n=1 << 60) == U.ERR_UNSUPPORTED   # more chunks than 30 bits count
    assert _evict(L, H=0, n=0) == U.ERR_INVALID and _evict(L, pages=-1) == U.ERR_INVALID and _evict(L, B=-1, n=0) == U.ERR_INVALID
    assert _evict(L, recent=-1) == U.ERR_INVALID
    for k in ("kc", "vc", "w", "table", "lens", "keep", "out"):
        assert _evict(L, **{k: None}) == U.ERR_INVALID, k
    assert _evict(L, vc=KC) == U.ERR_INVALID and _evict(L, cd=U.E4M3, ks=KS, vs=KS) == U.ERR_INVALID
    assert _evict(L, w=P(KC.value + 64)) == U.ERR_INVALID                    # weights inside the cache
    assert _evict(L, w=P(W.value + 4)) == U.ERR_INVALID                      # not 16-byte aligned
    for k, p in (("lens", LENS), ("keep", KEEP), ("out", OUT), ("table", TAB)):
        assert _evict(L, **{k: P(p.value + 2)}) == U.ERR_INVALID
    need = L.ulysses_cache_evict_workspace(4, 2, 8, 16)
    assert need > 0
    assert _evict(L, n=need - 1) == U.ERR_INVALID and _evict(L, ws=None) == U.ERR_INVALID
    assert _evict(L, ws=P(WS.value + 128)) == U.ERR_INVALID
    assert _evict(L, B=0) == U.OK
    assert L.ulysses_cache_evict_workspace(0, 2, 8, 16) == 0 and L.ulysses_cache_evict_workspace(4, 2, 8, 20) == 0
    assert L.ulysses_launch_count() == launches


def _write(L, w=W, T=4, B=4, k=X, v=Y, kc=KC, vc=VC, ks=KS, vs=VS, dt=U.BF16, cd=U.E2M1, D=128, lens=LENS):
    return L.ulysses_cache_write_weights(k, v, 256, 128, 256, 128, T, B, None, TAB, 8, lens, kc, vc, ks, vs, w, 64, 16, 2, D,
                                         dt, cd, None)


def test_write_refusals(L):
    launches = L.ulysses_launch_count()
    assert _write(L, ks=None) == U.ERR_INVALID and _write(L, vs=None) == U.ERR_INVALID
    assert _write(L, dt=U.E2M1) == U.ERR_INVALID and _write(L, D=80) == U.ERR_UNSUPPORTED
    assert _write(L, w=None) == U.ERR_INVALID and _write(L, w=P(W.value + 8)) == U.ERR_INVALID
    assert _write(L, w=P(KS.value + 16)) == U.ERR_INVALID and _write(L, w=P(X.value + 16)) == U.ERR_INVALID
    assert _write(L, k=P(KC.value + 32)) == U.ERR_INVALID                    # rows inside the cache
    assert _write(L, T=5) == U.ERR_INVALID and _write(L, lens=None) == U.ERR_INVALID
    assert _write(L, T=0, B=0) == U.OK
    # rows right behind a 4-bit cache of 64 pages x 2 heads x 16 rows of 72 bytes are outside it, one word before not
    end = KC.value + 64 * 2 * 16 * 72
    assert _write(L, k=P(end - 16)) == U.ERR_INVALID
    assert L.ulysses_launch_count() == launches


def _decode(L, w=W, q=X, o=Y, ks=KS, vs=VS, cd=U.E2M1, dt=U.BF16, B=4, Hq=4, cols=1 << 16, ws=WS, n=None, D=128):
    n = L.ulysses_attn_decode_weights_workspace(B, Hq, 2, D, cols, 16, dt, cd) if n is None else n
    return L.ulysses_attn_decode_weights(q, Hq * D, D, KC, VC, ks, vs, TAB, cols, LENS, o, Hq * D, D, None, w, B, Hq, 2, D, 64,
                                         16, 0.0, dt, cd, ws, n, None)


def test_decode_refusals(L):
    launches = L.ulysses_launch_count()
    assert _decode(L, ks=None) == U.ERR_INVALID and _decode(L, cd=U.FP32, ks=None, vs=None) == U.ERR_UNSUPPORTED
    assert _decode(L, w=None) == U.ERR_INVALID and _decode(L, w=P(W.value + 4)) == U.ERR_INVALID
    assert _decode(L, w=X) == U.ERR_INVALID and _decode(L, w=Y) == U.ERR_INVALID and _decode(L, w=KC) == U.ERR_INVALID
    need = L.ulysses_attn_decode_weights_workspace(4, 4, 2, 128, 1 << 16, 16, U.BF16, U.E2M1)
    plain = L.ulysses_attn_decode_workspace(4, 4, 2, 128, 1 << 16, 16, U.BF16, U.E2M1)
    assert need >= plain + 4 * 4 * 4 * (1 << 20) and plain > 0               # the scores of every position
    assert _decode(L, n=need - 1) == U.ERR_INVALID and _decode(L, ws=None) == U.ERR_INVALID
    assert _decode(L, ws=P(WS.value + 64)) == U.ERR_INVALID
    assert _decode(L, B=0, n=0) == U.OK
    assert L.ulysses_launch_count() == launches


def test_binding_refuses_on_the_host():
    kc, vc, ks, vs = U.kv_cache(4, 16, 2, 128, torch.uint8, device="cpu")
    assert kc.shape == (4, 2, 16, 72) and kc.dtype == torch.uint8 and ks.shape == (4, 2, 16)
    w = U.cache_weights(kc)
    assert w.shape == (4, 2, 16) and w.dtype == torch.float32 and not w.any()
    tab, lens = torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    t = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    kw = dict(k_scale=ks, v_scale=vs)
    for call in (lambda: U.cache_write(t, t, kc, vc, tab, lens, weights=w, **kw),
                 lambda: U.cache_read(kc, vc, tab, torch.zeros(5, dtype=torch.int32), 4, **kw),
                 lambda: U.attn_decode(t, kc, vc, tab, lens, weights=w, **kw),
                 lambda: U.cache_evict(kc, vc, w, tab, lens, lens, **kw)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="9 D / 16"):
        U.cache_write(t, t, kc[..., :70].contiguous(), vc[..., :70].contiguous(), tab, lens, **kw)
    with pytest.raises(ValueError, match="heads or D"):
        U.cache_write(t[..., :64], t[..., :64], kc, vc, tab, lens, **kw)
    with pytest.raises(ValueError, match="scales"):
        U.cache_evict(kc, vc, w, tab, lens, lens, k_scale=ks[:2], v_scale=vs)
