"""Page tables that go on from a given state."""
import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import PageTables
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
