"""Pins of the page plan's oracle where requests start behind another one's tokens."""
import numpy as np
import pytest

from oracle import serving as sv


@pytest.mark.parametrize("ctx,prefix,common", [
    (191, 192, 5), (64, 96, 2), (31, 200, 0), (0, 64, 0), (96, 96, 3), (200, 2**31 - 1, 6)])
def test_pages_in_front_of_all_new_tokens_are_shared(ctx, prefix, common):
    """A parent of 200 tokens, pages of 32: no new token goes to a page of two rows."""
    table = np.full((2, 9), -1)
    table[0, :7] = np.arange(7)
    refs = np.where(np.arange(20) < 7, 1, 0)
    t, r, starts, slots, _, _ = sv.plan(table, refs, [200, ctx], [30, 30], 31, 32, parents=[-1, 0], prefix=[0, prefix])
    assert starts.tolist() == [200, ctx]
    assert (r == 2).sum() == common and t[1, :common].tolist() == list(range(common))
    live = slots[slots >= 0]
    assert (r[live // 32] == 1).all() and len(set(live.tolist())) == len(live)


def test_a_parent_that_ends_bounds_nothing():
    table = np.array([[0, 1, 2, 3], [-1] * 4])
    t, r, *_ = sv.plan(table, [1, 1, 1, 1, 0, 0], [-1, 96], [0, 0], 1, 32, parents=[-1, 0], prefix=[0, 100])
    assert t.tolist() == [[-1] * 4, [0, 1, 2, 3]] and r.tolist() == [1, 1, 1, 1, 0, 0]


@pytest.mark.parametrize("row,window,flags", [
    ([0, 1, 2, 3, 4, 5], 0, 0),
    ([0, 1, -1, 3, 4, 5], 0, sv.NO_PREFIX),
    ([0, 99, 2, 3, 4, 5], 0, sv.NO_PREFIX | sv.BAD_PAGE),
    ([0, 1, 2, 3, 4, -1], 0, 0),            # behind the whole pages
    ([-1, -1, 2, 3, 4, 5], 40, 0),          # behind the window
    ([-1, -1, -1, 3, 4, 5], 40, sv.NO_PREFIX),
])
def test_pages_that_a_parent_lacks_are_told(row, window, flags):
    """128 tokens of a parent at 165; pages of 32."""
    table = np.array([row, [-1] * 6])
    t, r, starts, _, _, got = sv.plan(table, np.r_[np.ones(6, int), np.zeros(20, int)], [165, 128], [0, 0], 1, 32,
                                      window=window, parents=[-1, 0], prefix=[0, 128])
    assert got == flags and starts.tolist() == [165, 128]
    need = sv.needed_pages(128, 1, 32, window)
    for i in need:
        assert (t[1, i] == row[i]) == (i < 4 and 0 <= row[i] < 26)
