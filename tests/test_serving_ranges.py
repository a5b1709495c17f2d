"""Ranges that the rotary and cache calls refuse.  No GPU: refused before any launch."""
import ctypes

import pytest

from long_context_sequence_seq_gb300 import build as B
from long_context_sequence_seq_gb300 import ulysses as U

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    B.build()
    return U.lib()


@pytest.mark.parametrize("fn", ["fwd", "bwd"])
@pytest.mark.parametrize("f", [2.0 ** 40 * (1 + 2.0 ** -52), -2.0 ** 41, 1e300])
def test_frequencies_above_2_40(L, fn, f):
    launches = L.ulysses_launch_count()
    items = (U.RopeItem * 1)(U.RopeItem(1 << 32, 2 << 32, 2, 0, 128, 64, 0, 128, 64))
    freq = (ctypes.c_double * 32)(*[1.0] * 31, f)
    assert getattr(L, f"ulysses_rope_{fn}")(items, 1, P(3 << 32), 1, freq, None, 64, 0, 4, 1, 64, U.BF16, U.BF16,
                                            None) == U.ERR_UNSUPPORTED
    assert b"inv_freq[31]" in L.ulysses_last_error() and L.ulysses_launch_count() == launches
