"""Pins of the serving oracle: page plans worked by hand and their invariants,
rotations against complex numbers and known angles, visible positions."""
import numpy as np
import pytest

from oracle import serving as sv


def test_a_plan_worked_by_hand():
    """Pages of 32, a pool of 6, three slots of 3 pages."""
    table = np.array([[4, 1, -1], [2, -1, -1], [-1, -1, -1]])
    refs = np.array([0, 1, 1, 0, 1, 0])
    # 0 grows into its third page, 1 ends, 2 starts with 33 tokens.
    t, r, starts, slots, pos, flags = sv.plan(table, refs, [63, -1, 0], [3, 0, 32], 33, 32)
    assert t.tolist() == [[4, 1, 0], [-1, -1, -1], [2, 3, -1]]
    assert r.tolist() == [1, 1, 1, 1, 1, 0] and flags == 0
    assert starts.tolist() == [63, -1, 0]
    assert slots[0, :5].tolist() == [1 * 32 + 31, 0, 1, 2, -1]
    assert pos[0, :5].tolist() == [63, 64, 65, 66, -1]
    assert slots[2].tolist() == list(range(64, 96)) + [96] and (slots[1] == -1).all()
    # Two pages are wanted by 0 and 1, which is one too many for 1.
    t, r, starts, slots, _, flags = sv.plan(t, r, [63, 0, 95], [3, 0, 0], 33, 32)
    # Slot 1 took the last page first: 2 gets nothing and keeps what it has.
    assert starts.tolist() == [63, 0, -1] and t.tolist() == [[4, 1, 0], [5, -1, -1], [2, 3, -1]]
    assert flags == sv.NO_PAGES


def test_shared_prefixes_count_their_holders():
    table = np.array([[3, 0, 2], [-1, -1, -1], [-1, -1, -1]])
    refs = np.array([1, 0, 1, 1])
    t, r, starts, slots, _, flags = sv.plan(table, refs, [80, 64, 40], [0, 0, 0], 1, 32,
                                            parents=[-1, 0, 0], prefix=[0, 64, 63])
    assert t.tolist() == [[3, 0, 2], [3, 0, 1], [3, -1, -1]]
    assert r.tolist() == [2, 1, 1, 3]
    assert starts.tolist() == [80, 64, -1] and flags == sv.NO_PAGES
    # The parent ends: its pages stay with the others.
    t, r, *_ = sv.plan(t, r, [-1, 65, -1], [0, 0, 0], 1, 32)
    assert t.tolist() == [[-1, -1, -1], [3, 0, 1], [-1, -1, -1]] and r.tolist() == [1, 1, 0, 1]


def test_a_parent_with_a_parent_is_refused():
    table = np.array([[0, -1], [-1, -1], [-1, -1]])
    *_, flags = sv.plan(table, [1, 0, 0, 0], [5, 33, 33], [0] * 3, 1, 32, parents=[-1, 0, 1], prefix=[0, 32, 32])
    assert flags == sv.BAD_PARENT


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (40, 0), (40, 5), (64, 33), (500, 70)])
def test_needed_pages_are_those_that_rows_see(window, sinks):
    rng = np.random.default_rng(window)
    for _ in range(50):
        ctx, n = int(rng.integers(0, 400)), int(rng.integers(1, 9))
        rows = {j // 32 for t in range(n) for j in sv.visible(ctx + t, window, sinks)}
        assert sv.needed_pages(ctx, n, 32, window, sinks) == rows
        # Nothing that a later step's rows see has been given up.
        later = {j // 32 for j in sv.visible(ctx + 50, window, sinks) if j < ctx + n}
        assert later <= rows


def test_holders_are_counted_right_over_many_steps():
    rng = np.random.default_rng(1)
    B, width, page, pages, T = 6, 8, 32, 30, 4
    table, refs = np.full((B, width), -1), np.zeros(pages, int)
    ctx = np.full(B, -1)
    for _ in range(60):
        ends = rng.random(B) < 0.2
        ctx = np.where(ends, -1, np.where(ctx < 0, rng.integers(0, 150, B), ctx + rng.integers(0, T + 1, B)))
        ctx = np.where(ctx + T > width * page, -1, ctx)
        table, refs, starts, slots, _, flags = sv.plan(table, refs, ctx, rng.integers(0, T, B), T, page)
        held = table[table >= 0]
        assert np.array_equal(np.bincount(held, minlength=pages), refs) and len(set(held)) == len(held)
        live = slots[slots >= 0]
        assert len(set(live.tolist())) == len(live)
        assert not ((starts < 0) & (ctx >= 0)).any() or flags & sv.NO_PAGES


def test_rotation_is_a_turn_of_pairs():
    x = np.zeros(8)
    x[1] = 2.0
    # A quarter turn of pair 1: half pairing puts channel 1 on channel 1 + 4.
    quarter = [0.0, np.pi / 2, 0.0, 0.0]
    y, _ = sv.rotate(x, 1, quarter)
    assert np.allclose(y, np.eye(8)[5] * 2)
    y, _ = sv.rotate(x, 3, [np.pi / 2, 0, 0, 0], interleaved=True)      # (x0, x1) = (0, 2), three quarters
    assert np.allclose(y, np.eye(8)[0] * 2)
    # Scores of rotated rows depend on the distance alone.
    rng = np.random.default_rng(0)
    q, k, f = rng.normal(size=16), rng.normal(size=16), rng.random(8)
    s = [sv.rotate(q, p, f)[0] @ sv.rotate(k, p - 7, f)[0] for p in (7, 100, 5000)]
    assert np.allclose(s, s[0])


def test_norm_gives_rows_of_unit_mean_square():
    x = np.random.default_rng(0).normal(size=(3, 64)) * 7
    y, _ = sv.rotate(x, np.arange(3), None, np.ones(64), eps=0.0)
    assert np.allclose((y ** 2).mean(-1), 1)


def test_visible_positions():
    assert sv.visible(5) == [0, 1, 2, 3, 4, 5]
    assert sv.visible(5, window=2) == [4, 5]
    assert sv.visible(5, window=2, sinks=1) == [0, 4, 5]
    assert sv.visible(1, window=1, sinks=10) == [0, 1]
