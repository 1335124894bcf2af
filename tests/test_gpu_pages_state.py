"""Page tables that go on from a given state."""
import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, PageTables
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("pages", [20, 20000])
def test_the_pages_of_a_table_given_alone_are_counted(pages):
    table = np.array([[4, 1, -1], [4, 2, -7], [-1, pages, 2**31 - 1]])
    refs = np.bincount([4, 1, 4, 2], minlength=pages)
    t = PageTables(DEV, 3, 3, pages, 32, table=_i32(table))
    assert t.refs.dtype is torch.int32 and np.array_equal(t.refs.cpu().numpy(), refs)
    for ctx in ([60, 70, 0], [-1, 71, 40], [-1, -1, -1]):
        starts, slots, _ = t.plan(_i32(ctx), length=2)
        table, refs, *want, _ = sv.plan(table, refs, ctx, None, 2, 32)
        assert np.array_equal(t.table.cpu().numpy(), table) and np.array_equal(t.refs.cpu().numpy(), refs)
        assert np.array_equal(starts.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[1])
    assert not t.refs.any()


def test_counts_that_are_given_stay():
    """Pages that the caller keeps for itself, with and without a table."""
    refs = _i32([1, 0, 0, 1, 0, 0])
    t = PageTables(DEV, 1, 2, 6, 32, refs=refs)
    assert t.plan(_i32([0]), length=40)[1][0, [0, 39]].tolist() == [32, 2 * 32 + 7] and t.refs is refs
    t = PageTables(DEV, 1, 2, 6, 32, table=_i32([[5, -1]]), refs=_i32([1, 0, 0, 1, 0, 1]))
    assert t.plan(_i32([0]), length=40)[1][0, [0, 39]].tolist() == [5 * 32, 32 + 7]


def test_what_is_made_on_a_busy_stream_is_ready_on_another():
    """Page tables and a cache made behind a long queue, used on a side stream at once."""
    side, big = torch.cuda.Stream(), torch.randn(8192, 8192, device=DEV)
    ctx, want = _i32([0, 40, -1]), sv.plan(np.full((3, 4), -1), np.zeros(12, int), [0, 40, -1], None, 5, 32)
    q, kv = (torch.randn(3, 5, h, 64, device=DEV).bfloat16() for h in (4, 2))
    torch.cuda.synchronize()
    for _ in range(8):
        big @ big
    tables, cache = PageTables(DEV, 3, 4, 12, 32), BlockCache(DEV, 12, 2, 64, 32)
    starts, slots, positions = tables.plan(ctx, length=5, stream=side)
    cache.write_rotated(q, kv, kv, slots, positions, stream=side)
    torch.cuda.synchronize()
    for got, ref in zip((tables.table, tables.refs, starts, slots, positions), want):
        assert np.array_equal(got.cpu().numpy(), ref)
    keys, values = cache.read(tables.table, starts, _i32([5, 5, 0]), 5)
    plain = BlockCache(DEV, 12, 2, 64, 32)
    plain.write(kv, kv, tables.table, starts)
    assert torch.equal(cache.pool, plain.pool) and bool(keys[:2].any()) and torch.equal(keys, values)


def test_made_in_a_capture():
    ctx = _i32([33, -1])
    PageTables(DEV, 2, 3, 6, 32).plan(ctx, length=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tables = PageTables(DEV, 2, 3, 6, 32)
        out = tables.plan(ctx, length=2)
    for at in (33, 0, 64):
        ctx[0] = at
        graph.replay()
        torch.cuda.synchronize()
        table, refs, *want, _ = sv.plan(np.full((2, 3), -1), np.zeros(6, int), [at, -1], None, 2, 32)
        assert np.array_equal(tables.table.cpu().numpy(), table) and np.array_equal(tables.refs.cpu().numpy(), refs)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, want))
