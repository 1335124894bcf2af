"""Page tables and slot maps on the GPU against the oracle's plan, request by
request: whole numbers, compared for equality."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import PageTables, binding as sb
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _log(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _same(got, want):
    return np.array_equal(got.cpu().numpy(), np.asarray(want))


class Steps:
    """Page tables on the GPU and the oracle's, taken through the same steps."""

    def __init__(self, B, width, pages, page, T, window=0, sinks=0):
        self.__dict__.update(B=B, width=width, pages=pages, page=page, T=T, window=window, sinks=sinks)
        self.gpu = PageTables(DEV, B, width, pages, page)
        self.table, self.refs = np.full((B, width), -1), np.zeros(pages, int)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def set(self):
        self.gpu.table.copy_(_i32(self.table))
        self.gpu.refs.copy_(_i32(self.refs))

    def step(self, ctx, budgets, parents=None, prefix=None, **kw):
        self.status.zero_()
        starts, slots, positions = self.gpu.plan(
            _i32(ctx), None if budgets is None else _i32(budgets), self.T, self.window, self.sinks,
            None if parents is None else _i32(parents), None if prefix is None else _i32(prefix),
            status=self.status, **kw)
        self.table, self.refs, *want, flags = sv.plan(self.table, self.refs, ctx, budgets, self.T, self.page,
                                                      self.window, self.sinks, parents, prefix)
        assert _same(self.gpu.table, self.table)
        assert _same(self.gpu.refs, self.refs)
        assert _same(starts, want[0]) and _same(slots, want[1]) and _same(positions, want[2])
        assert int(self.status) == flags
        return flags


@pytest.mark.parametrize("B,width,pages,page,T,window,sinks", [
    (1, 1, 1, 32, 1, 0, 0),
    (1, 3, 9, 4096, 5, 0, 0),
    (7, 9, 70, 32, 6, 0, 0),
    (7, 9, 40, 32, 6, 0, 0),             # too few pages
    (33, 300, 5000, 32, 9, 0, 0),        # rows of more than one round of threads
    (12, 40, 300, 32, 40, 100, 5),
    (12, 40, 300, 64, 1, 1, 0),
    (12, 40, 90, 32, 9, 300, 70),
    (5, 700, 3000, 32, 2049, 3000, 33),  # chunks of prompts
    (12, 200, 2000, 32, 2000, 0, 0),     # one workgroup's table, more tokens than it writes itself
    (40, 500, 9000, 32, 9, 0, 0),        # a workgroup a row, several chunks of the pool
    (40, 500, 5500, 32, 9, 700, 40),     # too few pages
    (7, 3000, 17000, 32, 2100, 0, 0),    # tokens by a kernel of their own
    (3, 40, 70000, 32, 9, 0, 0),         # a small table over a large pool
    (1024, 16, 16384, 32, 16, 0, 0),     # the largest table of one workgroup
])
def test_steps(B, width, pages, page, T, window, sinks):
    _log(f"[pages] B={B} width={width} pages={pages} page={page} T={T} window={window} sinks={sinks}")
    rng = np.random.default_rng(B + T)
    s = Steps(B, width, pages, page, T, window, sinks)
    most = max(1, width * page - 2 * T)
    ctx = np.where(rng.random(B) < 0.3, -1, rng.integers(0, most, B))
    seen = 0
    for _ in range(8):
        budgets = rng.integers(0, T, B)
        parents, prefix = np.full(B, -1), rng.integers(-40, most, B)
        fresh = np.flatnonzero((s.table < 0).all(1))
        roots = np.setdiff1d(np.arange(B), fresh)
        if len(roots):
            some = fresh[rng.random(len(fresh)) < 0.6]
            parents[some] = rng.choice(roots, len(some))
        seen |= s.step(ctx, budgets, parents, prefix)
        ctx = np.where(rng.random(B) < 0.2, -1, np.where(ctx < 0, rng.integers(0, most, B), ctx + rng.integers(0, T + 1, B)))
        ctx = np.where(ctx + T > width * page, -1, ctx)
    held = s.table[s.table >= 0]
    assert np.array_equal(np.bincount(held, minlength=pages), s.refs)


def test_more_requests_than_a_round_of_the_sum():
    """2,500 requests: the sums over requests and over pages take several rounds."""
    rng = np.random.default_rng(3)
    s = Steps(2500, 3, 5200, 32, 2)
    ctx = rng.integers(-30, 90, 2500)
    for _ in range(3):
        s.step(ctx, rng.integers(0, 2, 2500))
        ctx = np.where(ctx < 0, 5, np.where(ctx > 90, -1, ctx + 20))


def test_a_pool_of_millions_of_pages():
    """Chunks of the pool that take a workgroup several rounds; free pages far apart."""
    s = Steps(3, 9, 5_000_000, 32, 2)
    s.refs[:] = 1
    s.refs[[0, 4095, 4096, 8191, 8192, 12345, 4_999_999, 4_500_000]] = 0
    s.set()
    assert s.step([60, 10, 100], [1, 1, 1]) == 0
    assert s.step([96, 40, 130], [1, 1, 1]) == sb.SV_FLAG_NO_PAGES
    s.step([-1, 40, 130], [1, 1, 1])


def test_the_largest_lengths():
    """Lengths at the ends of int32, the longest row, windows past every position."""
    width = sb.SV_MAX_CONTEXT // 4096
    s = Steps(5, width, 9000, 4096, 3, 2**31 - 1, 2**31 - 1)
    top = sb.SV_MAX_CONTEXT
    assert s.step([2**31 - 1, -2**31, top - 3, top - 2, 0], [2, 2, 2, 2, 0]) == sb.SV_FLAG_BAD_LENGTH
    s.window, s.sinks = 1, 0
    s.step([top - 1, -1, top - 3, 4095, 4094], [0, 0, 2, 0, 1])


def test_no_budgets_means_the_whole_block():
    s = Steps(3, 4, 12, 32, 5)
    s.step([0, 30, -1], None)
    s.step([3, 35, 120], None)


def test_flags_and_what_stays():
    s = Steps(4, 3, 10, 32, 4)
    s.step([70, 10, 31, -1], [3, 0, 1, 2])
    # A budget past the block, one below it; a block that does not fit keeps its pages.
    assert s.step([70, 12, 94, -1], [9, -5, 3, 0]) == sb.SV_FLAG_BAD_BUDGET | sb.SV_FLAG_BAD_LENGTH
    # Entries outside the pool are dropped and replaced.
    s.table[0, 1], s.table[3, 2], s.table[1, 2] = 10, 2**31 - 1, -2**31
    s.set()
    assert s.step([71, 12, 40, -1], [0, 0, 0, 0]) == sb.SV_FLAG_BAD_PAGE
    # Parents outside the batch, of itself, with a parent.
    assert s.step([71, 12, 40, 20], [0] * 4, [4, 1, -1, -9], [64] * 4) == sb.SV_FLAG_BAD_PARENT
    assert s.step([71, -1, -1, 20], [0] * 4) == 0
    assert s.step([71, 40, 64, 20], [0] * 4, [-1, 0, 1, -1], [64] * 4) == sb.SV_FLAG_BAD_PARENT


def test_no_status_and_given_outputs():
    t = PageTables(DEV, 2, 2, 3, 32)
    out = tuple(torch.full(s, 9, dtype=torch.int32, device=DEV) for s in ((2,), (2, 4), (2, 4)))
    got = t.plan(_i32([0, 90]), _i32([3, 77]), 4, out=out)
    assert all(a is b for a, b in zip(got, out))
    assert out[0].tolist() == [0, -1] and out[1].tolist() == [[0, 1, 2, 3], [-1] * 4]


def test_bad_arguments_are_refused():
    t = PageTables(DEV, 2, 2, 3, 32)
    with pytest.raises(ValueError):
        t.plan(_i32([0]), length=1)
    with pytest.raises(ValueError):
        t.plan(_i32([0, 0]), length=0)
    with pytest.raises(ValueError):
        t.plan(_i32([0, 0]).cpu())
    with pytest.raises(ValueError):
        t.plan(_i32([0, 0]), _i32([0, 0]).long())
    with pytest.raises(ValueError):
        t.plan(_i32([0, 0]), parents=_i32([-1, 0]))
    with pytest.raises(ValueError):
        t.plan(_i32([0, 0]), window=-1)
    for bad in (dict(page_size=48), dict(max_pages=0), dict(num_pages=0), dict(num_pages=1 << 26)):
        with pytest.raises(ValueError):
            PageTables(DEV, **{**dict(B=2, max_pages=2, num_pages=3, page_size=32), **bad})
    with pytest.raises(ValueError):
        PageTables(DEV, 2, 2, 3, 32, refs=torch.zeros(4, dtype=torch.int32, device=DEV))
    empty = PageTables(DEV, 0, 2, 3, 32)
    assert empty.plan(_i32([]), length=4)[1].shape == (0, 4)


def test_a_captured_step_replays():
    """Two graphs captured one after another, replayed in turn with eager steps between."""
    rng = np.random.default_rng(4)
    s = Steps(9, 10, 60, 32, 3)
    ctx, budgets = _i32(rng.integers(0, 200, 9)), _i32(rng.integers(0, 3, 9))
    graphs = []
    s.gpu.plan(ctx, budgets, 3)
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = s.gpu.plan(ctx, budgets, 3)
        graphs.append((g, out))
    s.table, s.refs = s.gpu.table.cpu().numpy().astype(int), s.gpu.refs.cpu().numpy().astype(int)
    for i in range(6):
        now = np.where(rng.random(9) < 0.3, -1, rng.integers(0, 250, 9))
        ctx.copy_(_i32(now))
        g, out = graphs[i % 2]
        g.replay()
        torch.cuda.synchronize()
        s.table, s.refs, *want, _ = sv.plan(s.table, s.refs, now, budgets.cpu().numpy(), 3, 32)
        assert _same(s.gpu.table, s.table) and _same(s.gpu.refs, s.refs)
        assert all(_same(a, b) for a, b in zip(out, want))
        s.step(rng.integers(0, 250, 9), rng.integers(0, 3, 9))


def test_on_another_stream():
    s = Steps(9, 10, 60, 32, 3)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ctx = _i32(np.arange(9) * 20)
    torch.cuda.synchronize()
    starts, slots, positions = s.gpu.plan(ctx, None, 3, stream=side)
    side.synchronize()
    want = sv.plan(s.table, s.refs, np.arange(9) * 20, None, 3, 32)
    assert _same(starts, want[2]) and _same(slots, want[3]) and _same(positions, want[4])
