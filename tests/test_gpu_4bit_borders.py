"""4-bit rows with elements on the borders between codes and right beside them,
for every block scale: codes equal the definition's in fp64, with none left out.

A border m (3 bits) times an e4m3 scale b (4 bits) is a number of 7 bits, so both
types hold it and its two neighbours.  A neighbour is a step of m b away, so its
quotient by b a step of m over b's significand (or twice that), which is below 2:
more than half a step of m, so that rounding to nearest does not reach m.  (Below a
product that is a power of two steps are half as wide; then m and b are powers of
two, and the quotient is the float below m.)  A quotient rounded once therefore falls
on its side of the border; products by the reciprocal of b fail for one in seven.
"""
import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

from tests.test_gpu_4bit import f64, same_codes, unpack

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def scales():
    """Every positive e4m3 value."""
    return torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def beside(x, dtype, by):
    """The float `by` places above x > 0."""
    ints = {"bf16": torch.int16, "fp32": torch.int32}[dtype]
    return float((torch.tensor(x, dtype=torch.float64).to(DT[dtype]).view(ints) + by).view(DT[dtype]).double())


def border_rows(dtype, e):
    """A row of 128 for every block scale b: a block that fixes the row's scale at 2^e, then borders times b and
    their neighbours, of either sign, beside the 6 b that fixes b."""
    rows = []
    for b in scales():
        x = [beside(m * b * 2.0 ** e, dtype, by) for m in so.E2M1_BORDERS for by in (-1, 0, 1)]
        row = np.zeros((8, 16))
        row[0, 3] = 2688.0 * 2.0 ** e
        for i, sign in ((1, 1.0), (3, -1.0)):
            row[i, :11], row[i + 1, :10] = sign * np.array(x[:11]), sign * np.array(x[11:])
            row[i, 15] = row[i + 1, 15] = 6.0 * b * 2.0 ** e
        rows.append(row.reshape(128))
    return np.array(rows)


@pytest.mark.parametrize("dtype", list(DT))
def test_the_rows_are_what_they_are_meant_to_be(dtype):
    for e in (-111, -60, 0, 40, 116):
        rows = border_rows(dtype, e)
        assert np.array_equal(f64(torch.from_numpy(rows).to(DT[dtype])), rows)
        _, block, scale = so.quantise4(rows)
        assert (scale == 2.0 ** e).all() and np.array_equal(block[:, 1:5], np.tile(scales()[:, None], (1, 4)))
        z = np.abs(rows[:, 16:80].reshape(-1, 4, 16)) / (scales()[:, None, None] * 2.0 ** e)
        on = np.isin(z, so.E2M1_BORDERS)
        assert on.sum() == 2 * 7 * 126
        near = np.min(np.abs(z[..., None] / np.array(so.E2M1_BORDERS) - 1), -1)
        assert ((near > 0) & (near <= {"bf16": 2.0 ** -7, "fp32": 2.0 ** -23}[dtype])).sum() == 2 * 2 * 7 * 126


def written(x, dtype):
    """(codes, block scales, row scales) of rows [T, H, D], as K's and as V's."""
    T, H, D = x.shape
    t = torch.from_numpy(x).to(DT[dtype]).cuda()
    kc, vc, ks, vs = U.kv_cache(-(-T // 64), 64, H, D, torch.uint8)
    tab = torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None].contiguous()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")   # noqa: E731
    U.cache_write(t, -t, kc, vc, tab, i32([T]), cu_new=i32([0, T]), k_scale=ks, v_scale=vs)
    U.check()
    for cache, scale in ((kc, ks), (vc, vs)):
        c, b = unpack(cache, 64, D)
        yield tuple(y.swapaxes(1, 2).reshape(-1, H, *y.shape[3:])[:T] for y in (c, b, f64(scale)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("e", [-111, -60, 0, 40, 116])
def test_borders_and_their_neighbours(e, dtype):
    x = border_rows(dtype, e)[:, None]
    for (c, b, s), sign in zip(written(x, dtype), (1.0, -1.0)):
        codes, block, scale = so.quantise4(sign * x)
        assert np.array_equal(s, scale) and np.array_equal(b, block)
        ok = same_codes(c, codes)
        assert ok.all(), (int((~ok).sum()), np.argwhere(~ok)[:5])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_fp32_elements(D):
    """None left out for lying near a border."""
    rng = np.random.default_rng(D)
    x = (rng.standard_normal((4096, 8, D)) * np.exp(rng.standard_normal((4096, 8, 1)))).astype(np.float32).astype(np.float64)
    for (c, b, s), sign in zip(written(x, "fp32"), (1.0, -1.0)):
        codes, block, scale = so.quantise4(sign * x)
        assert np.array_equal(s, scale) and np.array_equal(b, block)
        assert same_codes(c, codes).all()
