"""Rotary positions with large frequencies."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U

pytestmark = pytest.mark.gpu

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.parametrize("top", [2.0 ** 10, 2.0 ** 20, 2.0 ** 40])
def test_angles_of_large_frequencies(top):
    """Frequencies of many turns a position, at positions up to 2^31.  The turn
    is pos * f / 2 pi mod 1 with f / 2 pi cut to 2^-64 of a turn: off by |pos| 2^-64,
    cut to 2^-32 and rounded to fp32 (pi 2^-25 radians); sincospif is within
    2^-23, products and sums round by 2^-24 each."""
    half = 32
    inv = torch.tensor([top * 10.0 ** (-0.37 * i) for i in range(half)], dtype=torch.float64)
    pos = [2 ** 31 - 1, -2 ** 31, 123456789, 1, 0, -77]
    x = torch.randn((len(pos), 2, 64), generator=torch.Generator().manual_seed(30)).cuda()
    got = U.rope_fwd(x, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), inv)
    U.check()
    turns = [[float(Fraction(float(f)) * p / (2 * PI) % 1) for f in inv.tolist()] for p in pos]
    a = 2 * math.pi * np.array(turns)[:, None]
    X, G = x.double().cpu().numpy(), got.double().cpu().numpy()
    u, v = X[..., :half], X[..., half:]
    want = np.concatenate([u * np.cos(a) - v * np.sin(a), u * np.sin(a) + v * np.cos(a)], -1)
    c = math.pi * 2.0 ** -25 + 2 * math.pi * (2.0 ** -32 + 2.0 ** -33) + 2.0 ** -23 + 2 * 2.0 ** -24
    lim = np.tile(np.abs(u) + np.abs(v), 2) * c + 1e-38
    err = np.abs(G - want)
    assert np.all(err <= lim), float((err / lim).max())
