"""A prefix that is not, or no longer, in the parent's row: the plan says so."""
import pytest
import torch

from draft_verify_sampling_spec_amd import PageTables, binding as sb

from tests.test_gpu_pages import Steps, _i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

SIZES = pytest.mark.parametrize("width,pages", [(16, 60), (300, 20000)])    # one workgroup; a workgroup a row


@SIZES
def test_a_parent_whose_window_has_gone_on(width, pages):
    s = Steps(3, width, pages, 32, 2, window=64, sinks=20)
    for at in range(0, 171, 10):
        assert s.step([at, -1, -1], [1, 0, 0]) == 0
    # At 170 it holds pages 0 (sinks) and 3 on, which is what a request at 160 needs.
    assert s.step([170, 160, -1], [1, 1, 0], [-1, 0, -1], [0, 160, 0]) == 0
    assert s.table[1, [0, 3, 4]].tolist() == s.table[0, [0, 3, 4]].tolist()
    for at in range(180, 261, 10):
        s.step([at, -1, -1], [1, 0, 0])
    # At 260 it holds pages 0 and 6 on: of 0, 3 and 4 two are gone, and new ones hold nothing yet.
    assert s.step([260, -1, 160], [1, 0, 1], [-1, -1, 0], [0, 0, 160]) == sb.SV_FLAG_NO_PREFIX
    assert s.table[2, 0] == s.table[0, 0] and (s.refs[s.table[2, [3, 4]]] == 1).all()
    # The next step's pages are there.
    assert s.step([261, -1, 161], [1, 0, 1], [-1, -1, 0], [0, 0, 160]) == 0


@SIZES
def test_a_parent_that_has_no_pages(width, pages):
    """It never ran, starts in this very call, or has ended."""
    s = Steps(3, width, pages, 32, 200)
    assert s.step([-1, 64, -1], [0, 1, 0], [-1, 0, -1], [0, 64, 0]) == sb.SV_FLAG_NO_PREFIX
    assert s.step([-1, -1, -1], [0, 0, 0]) == 0
    assert s.step([0, 64, -1], [99, 1, 0], [-1, 0, -1], [0, 64, 0]) == sb.SV_FLAG_NO_PREFIX
    assert s.step([100, -1, -1], [1, 0, 0]) == 0
    assert s.step([100, 96, -1], [60, 1, 0], [-1, 0, -1], [0, 96, 0]) == 0
    assert s.step([-1, 97, -1], [0, 1, 0]) == 0
    assert s.step([-1, 98, 96], [0, 1, 0], [-1, -1, 0], [0, 0, 96]) == sb.SV_FLAG_NO_PREFIX


def test_a_parent_that_was_refused():
    s = Steps(2, 8, 4, 32, 200)
    assert s.step([0, -1], [150, 0]) == sb.SV_FLAG_NO_PAGES
    assert s.step([-1, 64], [0, 0], [-1, 0], [0, 64]) == sb.SV_FLAG_NO_PREFIX


@SIZES
def test_pages_that_are_held_or_not_needed_do_not_count(width, pages):
    s = Steps(2, width, pages, 32, 100)
    assert s.step([0, -1], [99, 0]) == 0
    assert s.step([100, 96], [1, 1], [-1, 0], [0, 99]) == 0
    assert s.step([-1, 97], [0, 1], [-1, 0], [0, 99]) == 0         # held; the parent ends
    assert s.step([-1, 97], [0, 1], [-1, 0], [0, 99]) == 0
    w = Steps(2, width, pages, 32, 4, window=40)
    for at in (0, 4, 8, 60, 64, 100, 130):
        w.step([at, -1], [3, 0])
    # Behind the window nothing is needed.
    assert w.step([130, 128], [3, 0], [-1, 0], [0, 128]) == 0
    # No tokens, no whole page, no parent.
    assert w.step([130, -1], [3, 0], [-1, -1], [0, 128]) == 0
    assert w.step([130, 31], [3, 0], [-1, 0], [0, 128]) == 0
    assert w.step([130, 128], [3, 0], [-1, -1], [0, 128]) == 0


def test_without_a_status_the_plan_is_the_same():
    t, u = (PageTables(DEV, 2, 8, 30, 32) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    args = dict(ctx_lens=_i32([-1, 64]), parents=_i32([-1, 0]), prefix_lens=_i32([0, 64]), length=3)
    got, want = t.plan(**args, status=status), u.plan(**args)
    assert int(status) == sb.SV_FLAG_NO_PREFIX and all(torch.equal(a, b) for a, b in zip(got, want))
