"""Eviction that moves so many rows that each CTA's ring in shared memory goes
round several times, for every kind of row, and selections whose clusters do not
all run at once.  Rows are moved, not computed, so everything is compared whole.

The definition is the oracle's, ordered by sorts of whole arrays (held to the
oracle's own on small ones)."""
import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U
from oracle import serving_oracle as so

from tests.test_gpu_evict import i32, make, parts

CTAS = 2 * 152                         # of the kernel that moves rows
RINGS = {                              # chunks whose places a CTA knows, and rows of a chunk
    ("bf16", 128): (5, 64), ("bf16", 64): (5, 128), ("fp32", 128): (5, 32), ("fp32", 64): (5, 64),
    ("e4m3", 128): (4, 128), ("e4m3", 64): (7, 128), ("e2m1", 128): (6, 128), ("e2m1", 64): (8, 128)}


def stays(w, keep, recent):
    """so.stays by one sort: NaN first, then by falling weight, then by rising position."""
    n = len(w)
    m = n if keep < 0 else min(n, keep)
    if m == n:
        return np.arange(n)
    r = min(m, recent)
    old, nan = w[:n - r], np.isnan(w[:n - r])
    order = np.lexsort((np.arange(n - r), np.where(nan, 0.0, -old), ~nan))
    return np.concatenate((np.sort(order[:m - r]), np.arange(n - r, n)))


def test_the_sorted_definition_is_the_oracles():
    rng = np.random.default_rng(0)
    for n in (1, 2, 7, 50, 200):
        for keep in (-1, 0, 1, n // 2, n - 1, n, n + 3):
            for recent in (0, 1, n // 3, n + 5):
                w = np.floor(rng.standard_normal(n) * 2) / 2
                w[rng.random(n) < 0.1] = np.nan
                w[rng.random(n) < 0.1] = np.inf
                w[rng.random(n) < 0.1] = -np.inf
                w[rng.random(n) < 0.2] = -0.0
                assert stays(w, keep, recent).tolist() == so.stays(w, keep, recent)


def run(a, lens, keep, recent):
    buf, tab, page = parts(a), a["page_table"].cpu().numpy(), a["weights"].shape[2]
    w = a["weights"].double().cpu().numpy()
    new, moved = [], 0
    for b, n in enumerate(lens):
        m = n if keep[b] < 0 else min(n, keep[b])
        new.append(m)
        p = np.arange(n)
        pg, sl = tab[b][p // page], p % page
        for h in range(w.shape[1] if m < n else 0):
            src = stays(w[pg, h, sl], keep[b], recent)
            moved += int((src != np.arange(m)).sum())
            for x in buf.values():
                x[pg[:m], h, sl[:m]] = x[pg[src], h, sl[src]]
    out = U.cache_evict(keep=i32(keep), recent=recent, **a)
    U.check()
    assert out.tolist() == new
    got = parts(a)
    for x in buf:
        assert np.array_equal(got[x], buf[x]), x
    return moved


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["any", "by a little", "by a lot"])
@pytest.mark.parametrize("held,D", list(RINGS))
def test_every_ring_goes_round(held, D, kind):
    """Three times a CTA and more.  Weights in any order, or rising with the position,
    so that every row moves, by less than a chunk or by many."""
    ring, chunk = RINGS[held, D]
    B, H, page = 8, 8, 64
    keep = -(-3 * ring * CTAS * chunk // (B * H)) + 100
    lens = [keep + (40 if kind == "by a little" else 1500) + 3 * b for b in range(B)]
    a = make(lens, H, D, page, held, seed=len(held) + D)
    if kind != "any":
        tab, w = a["page_table"].cpu().numpy(), a["weights"].cpu().numpy()
        for b, n in enumerate(lens):
            p = np.arange(n)
            w[tab[b][p // page], :, p % page] = p[:, None]
        a["weights"].copy_(torch.from_numpy(w))
    moved = run(a, lens, [keep] * B, 100)
    assert moved >= 0.9 * keep * B * H or kind == "any"


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,n", [(37, 1, 20000), (19, 2, 40000), (19, 2, 70000), (18, 4, 9000), (25, 3, 20000), (19, 4, 20000),
                                   (19, 4, 34000)])
def test_selections_that_do_not_all_run_at_once(B, H, n):
    """As many heads as there are clusters at once, and one or two more."""
    lens = [n - 17 * b for b in range(B)]
    run(make(lens, H, 64, 64, "e2m1", seed=B), lens, [900 + b for b in range(B)], 64)
