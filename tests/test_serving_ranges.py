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


def test_pointers_of_32_bit_elements_are_aligned(L):
    launches = L.ulysses_launch_count()
    x, y, z, w, i = (P(n << 40) for n in range(1, 6))
    for odd in (P((5 << 40) + 1), P((5 << 40) + 2)):
        items = (U.RopeItem * 1)(U.RopeItem(1 << 32, 2 << 32, 2, 0, 128, 64, 0, 128, 64))
        freq = (ctypes.c_double * 32)(*[1.0] * 32)
        assert L.ulysses_rope_fwd(items, 1, odd, 1, freq, None, 64, 0, 4, 1, 64, U.BF16, U.BF16, None) == U.ERR_INVALID
        for cu, table, lens in ((odd, i, i), (i, odd, i), (i, i, odd)):
            assert L.ulysses_cache_write(x, y, 256, 128, 256, 128, 4, 4, cu, table, 8, lens, z, w, None, None, 64, 16, 2, 128,
                                         U.BF16, U.BF16, None) == U.ERR_INVALID
            assert L.ulysses_cache_read(z, w, None, None, table, 8, cu, lens, x, y, 256, 128, 256, 128, 4, 4, 64, 16, 2, 128,
                                        U.BF16, U.BF16, None) == U.ERR_INVALID
        for table, lens, lse in ((odd, i, i), (i, odd, i), (i, i, odd)):
            assert L.ulysses_attn_decode(x, 512, 128, z, w, None, None, table, 8, lens, y, 512, 128, lse, 4, 4, 2, 128, 64, 16,
                                         0.0, U.BF16, U.BF16, None, 0, None) == U.ERR_INVALID
            assert b"4-byte" in L.ulysses_last_error()
    assert L.ulysses_launch_count() == launches


@pytest.mark.parametrize("dt,Hkv,G,kernel", [(U.BF16, 32, 16, "AUTO"), (U.BF16, 16, 17, "AUTO"), (U.FP32, 32, 8, "AUTO"),
                                             (U.FP32, 16, 9, "AUTO"), (U.FP32, 16, 16, "AUTO"), (U.BF16, 16, 5, "SIMT"),
                                             (U.FP32, 16, 3, "SIMT"), (U.FP32, 32, 1, "AUTO")])
def test_units_of_one_sequence(L, dt, Hkv, G, kernel):
    """2^30 positions, as many heads as make 2^35 with the groups the header names."""
    n = 16 if dt == U.BF16 else 8
    if kernel == "SIMT":
        n = 2 if G == 3 else 4
    assert (1 << 30) * Hkv * -(-G // n) == 1 << 35
    launches = L.ulysses_launch_count()
    x, y, z, w, i, ws = (P(m << 44) for m in range(1, 7))
    Hq = Hkv * G
    assert L.ulysses_set_kernel(getattr(U, f"KERNEL_{kernel}")) == U.OK
    try:
        rc = L.ulysses_attn_decode(x, Hq * 128, 128, z, w, None, None, i, 1 << 26, i, y, Hq * 128, 128, None, 1, Hq, Hkv, 128,
                                   64, 16, 0.0, dt, dt, ws, 1 << 40, None)
    finally:
        L.ulysses_set_kernel(U.KERNEL_AUTO)
    assert rc == U.ERR_UNSUPPORTED and b"2^35" in L.ulysses_last_error()
    assert L.ulysses_launch_count() == launches
