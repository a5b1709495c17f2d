"""Pins of the fp64 definitions that the rotary, paged-cache and single-token
attention tests compare with."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_oracle as so


def test_rope_quarter_turn_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = [math.pi / 2, math.pi]                     # position 1: a quarter and a half turn
    half = so.rope(x, [1], f)
    assert np.allclose(half, [[[-3.0, -2.0, 1.0, -4.0, 5.0]]], atol=1e-15)
    adj = so.rope(x, [1], f, pairs="adjacent")
    assert np.allclose(adj, [[[-2.0, 1.0, -3.0, -4.0, 5.0]]], atol=1e-15)
    two = so.rope(x, [[1], [0]], f, axes=[1, 0])   # pair 0 stays (axis 1 is at 0), pair 1 turns
    assert np.allclose(two, [[[1.0, -2.0, 3.0, -4.0, 5.0]]], atol=1e-15)


def test_rope_scores_depend_on_distance_and_adjoint_is_inverse():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    f = [0.7 ** i for i in range(8)]
    dots = [float(np.sum(so.rope(q, [a], f) * so.rope(k, [b], f))) for a, b in ((5, 3), (105, 103), (2, 0))]
    assert np.allclose(dots, dots[0])
    y = so.rope(q, [9], f)
    assert np.allclose(so.rope(y, [9], f, inverse=True), q)
    # <R x, g> = <x, R^T g>
    g = rng.standard_normal((1, 1, 16))
    assert np.isclose(np.sum(y * g), np.sum(q * so.rope(g, [9], f, inverse=True)))


def test_e4m3_matches_torch_on_every_kind_of_value():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 2.0 ** rng.integers(-12, 8, 20000),
                        [0.0, 448.0, -448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 0.0146484375, 17.0, 19.0]])
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(so.e4m3(x).astype(np.float32), want)


def test_quantised_rows_err_by_half_a_step():
    rng = np.random.default_rng(2)
    rows = rng.standard_normal((64, 128)) * np.exp(rng.uniform(-20, 20, (64, 1)))
    codes, scale = so.quantise(rows)
    assert np.max(np.abs(codes)) == so.E4M3_MAX
    err = np.abs(codes * scale[:, None] - rows)
    # 2^-4 relative for normal codes, half of 2^-9 scale units below 2^-6
    assert np.all(err <= np.maximum(np.abs(rows) * 2.0 ** -4, scale[:, None] * 2.0 ** -10) * (1 + 1e-12))
    codes, scale = so.quantise(np.zeros((1, 8)))
    assert np.all(codes == 0) and scale[0] > 0


@pytest.mark.parametrize("G", [1, 3])
def test_decode_is_the_last_row_of_causal_attention(G):
    rng = np.random.default_rng(3)
    n, Hkv, D = 13, 2, 8
    q = rng.standard_normal((Hkv * G, n, D))
    k, v = rng.standard_normal((Hkv, n, D)), rng.standard_normal((Hkv, n, D))
    ro, rl = oracle.attn_fwd(q, k, v, None, True)
    o, lse = so.decode(q[:, -1], k.transpose(1, 0, 2), v.transpose(1, 0, 2))
    assert np.allclose(o, ro[:, -1]) and np.allclose(lse, rl[:, -1])
    o, lse = so.decode(q[:, -1], np.zeros((0, Hkv, D)), np.zeros((0, Hkv, D)))
    assert np.all(o == 0) and np.all(np.isneginf(lse))


def test_cache_rows_follow_the_table():
    cache = np.arange(3 * 1 * 16 * 1, dtype=np.float64).reshape(3, 1, 16, 1)
    got = so.cache_rows(cache, [[2, 0]], 0, 4, first=14)[:, 0, 0]
    assert got.tolist() == [2 * 16 + 14, 2 * 16 + 15, 0, 1]
