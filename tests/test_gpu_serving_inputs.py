"""Rotary positions with large frequencies, and offsets that do not fit the
tokens of a cache call."""
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


@pytest.mark.parametrize("cu,lens", [([0, 2, 7], [2, 5]), ([-3, 2, 4], [5, 2])])
def test_sequences_whose_offsets_do_not_fit_are_skipped(cu, lens):
    """A sequence that begins before the first token or ends behind the last is
    reported and none of its tokens is stored or read; the other one's are."""
    T, good = 4, 0 if cu[0] == 0 else 1
    tab = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    kc, vc, _, _ = U.kv_cache(2, 16, 1, 64)
    x = torch.randn((T, 1, 64), generator=torch.Generator().manual_seed(31)).add(100.0).bfloat16().cuda()
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    U.cache_write(x, x, kc, vc, tab, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu_new=c)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_SEQLENS
    mine = slice(0, 2) if good == 0 else slice(2, 4)
    for cache in (kc, vc):
        assert torch.equal(cache[good, 0, :2], x[mine, 0]) and bool((cache[1 - good] == 0).all())
    kc.fill_(5.0)
    vc.fill_(5.0)
    out = [torch.full((T, 1, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    U.cache_read(kc, vc, tab, c, T, out=out)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_SEQLENS
    for y in out:
        assert bool((y[mine] == 5.0).all()) and int((y == 7.0).sum()) == 2 * 64
