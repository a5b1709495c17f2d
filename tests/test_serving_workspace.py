"""Workspace refusals of single-token attention where a workspace is needed (a
table too wide for the launch without one).  No GPU: refused before any launch."""
import ctypes

import pytest

from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    B.build()
    return U.lib()


def _call(L, ws, n, B, Hq, Hkv, D, cols, page, dt, cd):
    at = [P(i << 40) for i in range(1, 9)]            # far apart, aligned, never dereferenced
    ks, vs = (at[6], at[7]) if cd == U.E4M3 else (None, None)
    return L.ulysses_attn_decode(at[0], Hq * D, D, at[1], at[2], ks, vs, at[3], cols, at[4], at[5], Hq * D, D, None, B, Hq,
                                 Hkv, D, 64, page, 0.0, dt, cd, ws, n, None)


@pytest.mark.parametrize("dt,cd", [(U.BF16, U.BF16), (U.BF16, U.E4M3), (U.FP32, U.FP32), (U.FP32, U.E4M3)])
@pytest.mark.parametrize("B,Hq,Hkv,D,cols,page", [(4, 4, 2, 128, 1 << 16, 16), (1, 32, 8, 128, 1 << 14, 64),
                                                  (300, 8, 8, 64, 4, 16), (5, 40, 1, 64, 1 << 16, 16)])
def test_workspace_refusals(L, B, Hq, Hkv, D, cols, page, dt, cd):
    shape = (B, Hq, Hkv, D, cols, page, dt, cd)
    need = L.ulysses_attn_decode_workspace(*shape)
    assert need > 0
    launches = L.ulysses_launch_count()
    ws = P(1 << 50)
    assert _call(L, ws, need - 1, *shape) == U.ERR_INVALID
    assert b"workspace too small" in L.ulysses_last_error()
    assert _call(L, ws, 0, *shape) == U.ERR_INVALID
    assert _call(L, None, need, *shape) == U.ERR_INVALID
    assert _call(L, P((1 << 50) + 128), need, *shape) == U.ERR_INVALID
    assert b"256-byte aligned" in L.ulysses_last_error()
    assert L.ulysses_launch_count() == launches
