"""Eviction: calls beside the ordinary ones.  Rows are moved, not computed, so
everything is compared whole."""
import numpy as np
import pytest
import torch

from long_context_sequence_seq_gb300 import ulysses as U

from tests.test_gpu_evict import expect, i32, make, parts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("keep", [100, 130, -1])
@pytest.mark.parametrize("column", [0, 3, 6])
def test_a_bad_page_of_a_sequence_that_loses_nothing_is_reported(column, keep):
    """All of its tokens stay, so nothing would move: its pages are looked at all the same."""
    lens = [100, 60]
    a = make(lens, 2, 64, 16, "bf16", seed=1)
    a["page_table"][0, column] = -1 if column else a["k_cache"].shape[0]
    want, _ = expect(a, [0, 60], [0, 30], 8)
    out = U.cache_evict(keep=i32([keep, 30]), recent=8, **a)
    with pytest.raises(U.UlyssesError) as e:
        U.check()
    assert e.value.code == U.ERR_BAD_PAGES
    assert out.tolist() == [100, 30]
    got = parts(a)
    assert all(np.array_equal(got[x], want[x]) for x in want)


def test_entries_behind_the_last_page_are_not_looked_at():
    """Whole pages, empty sequences and wide tables, nothing to take out: no report."""
    lens = [96, 0, 1, 16]
    a = make(lens, 1, 64, 16, "bf16", seed=2)          # entries behind a sequence's pages hold a wild id
    wide = torch.full((4, 5000), -9, dtype=torch.int32, device="cuda")
    wide[:, :a["page_table"].shape[1]] = a["page_table"]
    for table in (a["page_table"], wide):
        out = U.cache_evict(keep=i32([-1, 0, 1, 20]), **dict(a, page_table=table))
        U.check()
        assert out.tolist() == lens


def test_a_bad_page_far_down_a_wide_table():
    """More pages than a selecting CTA's threads look at before the lengths are there."""
    n = 16 * 2100
    a = make([n, 50], 1, 64, 16, "e2m1", seed=3, slack=1)
    a["page_table"][0, 2099] = 1 << 29
    want, _ = expect(a, [0, 50], [0, 20], 0)
    for keep in (n, 100):
        b = {x: t.clone() if t is not None else None for x, t in a.items()}
        out = U.cache_evict(keep=i32([keep, 20]), **b)
        with pytest.raises(U.UlyssesError):
            U.check()
        assert out.tolist() == [n, 20]
        got = parts(b)
        assert all(np.array_equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("B", [3, 2100])
def test_new_lengths_in_the_place_of_the_budgets(B):
    lens = [(13 * i + 30) % 50 for i in range(B)]
    keep = [(7 * i + 5) % 40 for i in range(B)]
    a = make(lens, 1, 64, 16, "bf16", seed=4)
    want, new = expect(a, lens, keep, 2)
    kp = i32(keep)
    assert U.cache_evict(keep=kp, recent=2, out=kp, **a) is kp
    U.check()
    got = parts(a)
    assert kp.tolist() == new and all(np.array_equal(got[x], want[x]) for x in want)


@pytest.mark.parametrize("recent", [-1, -(1 << 31), -(1 << 32), 5 - (1 << 32), -(1 << 63), -(1 << 70)])
def test_recent_below_zero_is_refused_whatever_its_size(recent):
    """Python's numbers have no end: cut to 32 bits some of these would be 0 or more."""
    a = make([100], 1, 64, 16, "bf16", seed=5)
    before, launches = parts(a), U.launch_count()
    with pytest.raises(U.UlyssesError, match="recent"):
        U.cache_evict(keep=i32([30]), recent=recent, **a)
    assert U.launch_count() == launches
    got = parts(a)
    assert all(np.array_equal(got[x], before[x]) for x in before)
