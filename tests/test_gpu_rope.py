"""Rotary positions (ulysses_rope_fwd / _bwd) against the fp64 definition.

Element-wise bound, for a pair (x1, x2) and fp32 arithmetic: the turn is
rounded to fp32 (2^-25 half turns = pi 2^-25) after a truncation of 2^-32
turns and freq's own 2^-53 * |pos| turns; sincospif is within 2 ulp (2^-23);
each product and sum rounds by 2^-24.  So |dy| <= (|x1| + |x2|) *
(pi 2^-25 + 2 pi (2^-32 + 2^-53 |pos| ) + 2^-23 + 2 * 2^-24), and a bf16
result adds half a bf16 step, 2^-8 |y|.
"""
import math

import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def bound(x, y, rot, far, out, pairs):
    ax = np.abs(x)
    s = ax.copy()
    h = rot // 2
    if pairs == "half":
        s[..., :h] += ax[..., h:rot]
        s[..., h:rot] += ax[..., :h]
    else:
        s[..., 0:rot:2] += ax[..., 1:rot:2]
        s[..., 1:rot:2] += ax[..., 0:rot:2]
    c = math.pi * 2.0 ** -25 + 2 * math.pi * (2.0 ** -32 + 2.0 ** -53 * far) + 2.0 ** -23 + 2 * 2.0 ** -24
    return s * c + (np.abs(y) * 2.0 ** -8 if out == "bf16" else 0.0) * (1 + 2.0 ** -6) + 1e-38


def normal(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


CASES = [
    # T, Hq, Hkv, D, rot, axes (sections or None), span, layout, pairs, dtype, out
    (1, 4, 1, 128, 128, None, 1 << 20, "seq", "half", "bf16", "bf16"),
    (1, 32, 8, 128, 128, None, 1 << 30, "head", "half", "bf16", "bf16"),
    (17, 8, 2, 64, 64, None, 100, "head", "adjacent", "bf16", "bf16"),
    (333, 6, 2, 128, 64, None, 4096, "seq", "half", "fp32", "fp32"),
    (333, 3, 3, 128, 48, None, 4096, "seq", "adjacent", "fp32", "fp32"),
    (1000, 8, 8, 64, 48, [10, 14], 1 << 20, "head", "half", "bf16", "bf16"),
    (2049, 5, 1, 128, 128, [16, 24, 24], 300, "seq", "half", "bf16", "bf16"),
    (77, 32, 8, 128, 128, [16, 16, 16, 16], 1 << 20, "head", "adjacent", "fp32", "fp32"),
    (130, 2, 1, 64, 16, None, 7, "seq", "half", "bf16", "bf16"),
    (10007, 8, 2, 128, 128, None, 1 << 20, "head", "half", "fp32", "fp32"),
]


def _given(T, Hq, Hkv, D, rot, sections, span, layout, dtype):
    shape = lambda H: (T, H, D) if layout == "seq" else (H, T, D)  # noqa: E731
    q, k = normal(shape(Hq), 1, dtype), normal(shape(Hkv), 2, dtype)
    inv, axes = U.rope_frequencies(rot, 10000.0, sections)
    n = len(sections) if sections else 1
    pos = torch.randint(-span, span, (n, T), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    return q, k, (pos[0].contiguous() if n == 1 else pos), inv, axes


def _check(got, x, pos, inv, axes, rot, span, layout, pairs, out, inverse):
    tr = (lambda a: a.transpose(1, 0, 2)) if layout == "head" else (lambda a: a)
    X, G = tr(f64(x)), tr(f64(got))
    want = so.rope(X, pos.cpu().numpy(), inv.numpy(), axes.numpy(), pairs, inverse)
    err = np.abs(G - want)
    lim = bound(X, want, rot, span, out, pairs)
    assert np.all(err <= lim), (float((err / lim).max()), float(err.max()))
    assert np.array_equal(G[..., rot:], X[..., rot:] if out != "bf16" else f64(torch.from_numpy(X[..., rot:].copy()).bfloat16()))


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,sections,span,layout,pairs,dtype,out", CASES)
def test_forward_and_adjoint(T, Hq, Hkv, D, rot, sections, span, layout, pairs, dtype, out):
    q, k, pos, inv, axes = _given(T, Hq, Hkv, D, rot, sections, span, layout, dtype)
    for fn, inverse in ((U.rope_fwd, False), (U.rope_bwd, True)):
        a, b = fn(q, k, pos, inv, axes, layout=layout, pairs=pairs)
        U.check()
        assert a.dtype == q.dtype and a.shape == q.shape and b.shape == k.shape
        _check(a, q, pos, inv, axes, rot, span, layout, pairs, out, inverse)
        _check(b, k, pos, inv, axes, rot, span, layout, pairs, out, inverse)


@pytest.mark.parametrize("layout,pairs", [("seq", "half"), ("head", "adjacent")])
def test_gradients_in_bf16_from_fp32(layout, pairs):
    q, k, pos, inv, axes = _given(515, 8, 2, 128, 96, None, 1 << 16, layout, "fp32")
    a, b = U.rope_bwd(q, k, pos, inv, axes, layout=layout, pairs=pairs, dtype=torch.bfloat16)
    U.check()
    assert a.dtype == b.dtype == torch.bfloat16
    _check(a, q, pos, inv, axes, 96, 1 << 16, layout, pairs, "bf16", True)
    _check(b, k, pos, inv, axes, 96, 1 << 16, layout, pairs, "bf16", True)


def test_backward_against_differences():
    """The forward is linear, so (f(x + h e) - f(x)) / h is its derivative at
    any h; <g, that> must be <bwd(g), e>."""
    q, _, pos, inv, axes = _given(65, 4, 1, 128, 128, None, 1 << 12, "seq", "fp32")
    g, e = normal(q.shape, 7, "fp32"), normal(q.shape, 8, "fp32")
    f = lambda x: f64(U.rope_fwd(x, None, pos, inv, axes))  # noqa: E731
    left = np.sum(f64(g) * (f(q + 4 * e) - f(q)) / 4)
    right = np.sum(f64(U.rope_bwd(g, None, pos, inv, axes)) * f64(e))
    # every element of each side is off by at most ~3.4e-7 of values of size <= 10 (the bound above, and the
    # rounding of q + 4 e, 2^-24 of it), added over n elements weighted by the other tensor
    lim = 3.4e-7 * 20 * (np.abs(f64(g)).sum() + np.abs(f64(e)).sum())
    assert abs(left - right) <= lim, (left, right, lim)


@pytest.mark.parametrize("layout", ["seq", "head"])
@pytest.mark.parametrize("B", [1, 2])
def test_in_place_on_slices_of_a_fused_projection(layout, B):
    """Q and K are head ranges of one [.., H_q + 2 H_kv, ..] tensor, turned in
    place; V and the other tokens stay as they are."""
    Hq, Hkv, S, D = 6, 2, 45, 128
    H = Hq + 2 * Hkv
    x = normal((B, S, H, D) if layout == "seq" else (B, H, S, D), 5, "bf16")
    keep = x.clone()
    cut = (lambda t, a, b: t[:, :, a:b]) if layout == "seq" else (lambda t, a, b: t[:, a:b])
    pos = torch.randint(0, 9999, (B, S), dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(D)
    q, k = cut(x, 0, Hq), cut(x, Hq, Hq + Hkv)
    U.rope_fwd(q, k, pos, inv, axes, layout=layout, out=(q, k))
    U.check()
    want_q, want_k = U.rope_fwd(cut(keep, 0, Hq).contiguous(), cut(keep, Hq, Hq + Hkv).contiguous(), pos, inv, axes,
                                layout=layout)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)
    assert torch.equal(cut(x, Hq + Hkv, H), cut(keep, Hq + Hkv, H))


def test_broadcast_source_and_four_dimensions_agree_with_three():
    S, H, D = 33, 4, 64
    x = normal((S, 1, D), 9, "fp32").expand(S, H, D)
    pos = torch.arange(S, dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(D)
    a = U.rope_fwd(x, None, pos, inv, axes, out=torch.empty((S, H, D), device="cuda"))
    b = U.rope_fwd(x.contiguous()[None], None, pos[None], inv, None)
    U.check()
    assert torch.equal(a, b[0])


def test_far_positions_keep_their_angles():
    """At position 2^31 - 1 an fp32 angle is off by a hundred turns."""
    x = normal((3, 2, 128), 10, "fp32")
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(128, 1e6)
    got = U.rope_fwd(x, None, pos, inv, axes)
    U.check()
    _check(got, x, pos, inv, axes, 128, 2 ** 31, "seq", "half", "fp32", False)


def test_not_finite_elements_stay_in_their_pair():
    x = normal((2, 1, 64), 11, "fp32")
    x[0, 0, 3] = float("nan")
    x[1, 0, 40] = float("inf")
    pos = torch.ones(2, dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(64)
    y = U.rope_fwd(x, None, pos, inv, axes)
    bad = ~torch.isfinite(y)
    assert bad.nonzero().tolist() == [[0, 0, 3], [0, 0, 35], [1, 0, 8], [1, 0, 40]]


def test_binding_refusals():
    x = normal((4, 2, 128), 12, "bf16")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    inv, axes = U.rope_frequencies(128)
    for bad, err in ((dict(positions=pos.long()), TypeError), (dict(positions=pos[:3]), ValueError),
                     (dict(inv_freq=inv.float()), ValueError), (dict(inv_freq=inv.cuda()), ValueError),
                     (dict(axes=axes.long()), ValueError), (dict(layout="x"), ValueError),
                     (dict(pairs="x"), ValueError), (dict(q=x.transpose(1, 2)), ValueError),
                     (dict(q=x.half()), TypeError), (dict(out=x[:2]), ValueError),
                     (dict(out=(x, x)), ValueError), (dict(k=x[:3]), ValueError)):
        with pytest.raises(err):
            U.rope_fwd(**{**dict(q=x, k=None, positions=pos, inv_freq=inv, axes=axes), **bad})
    with pytest.raises(U.UlyssesError):
        U.rope_fwd(x, x, pos, inv, axes, out=(x, x))
