"""Requests that start behind another one's tokens: no call gives out a slot in a
page that more than one row holds, whatever lengths the caller names."""
import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import PageTables

from tests.test_gpu_pages import Steps, _i32

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

SMALL, LARGE = (16, 400), (300, 20000)      # one workgroup's table and pool; a workgroup a row


def _alone(tables, slots):
    """Every slot's page has one holder, and no slot is given out twice."""
    live = slots[slots >= 0]
    assert bool((tables.refs[live.long() // tables.page_size] == 1).all())
    assert torch.unique(live).numel() == live.numel()


@pytest.mark.parametrize("width,pages", [SMALL, LARGE])
@pytest.mark.parametrize("ctx,prefix", [
    (191, 192),         # a prompt matched in full, its last token run again
    (64, 96), (31, 200), (0, 64), (96, 96),
    (200, 2**31 - 1),
])
def test_own_tokens_never_go_to_a_parents_pages(width, pages, ctx, prefix):
    t = PageTables(DEV, 3, width, pages, 32)
    t.plan(_i32([0, -1, -1]), _i32([199, 0, 0]), 200)
    lens = _i32([200, ctx, ctx])
    starts, slots, _ = t.plan(lens, _i32([30, 30, 7]), 31, parents=_i32([-1, 0, 0]), prefix_lens=_i32([0, prefix, prefix]))
    assert torch.equal(starts, lens)
    _alone(t, slots)
    common = min(ctx, prefix) // 32
    table = t.table.cpu().numpy()
    assert np.array_equal(table[1, :common], table[0, :common]) and np.array_equal(table[2, :common], table[0, :common])


@pytest.mark.parametrize("width,pages", [SMALL, LARGE])
def test_a_parent_that_ends_in_the_call_leaves_its_pages(width, pages):
    """Its row, as it was, is what the others start behind."""
    t = PageTables(DEV, 2, width, pages, 32)
    t.plan(_i32([0, -1]), _i32([99, 0]), 100)
    before = t.table.clone()
    _, slots, _ = t.plan(_i32([-1, 96]), _i32([0, 4]), 5, parents=_i32([-1, 0]), prefix_lens=_i32([0, 100]))
    assert torch.equal(t.table[1, :3], before[0, :3]) and bool((t.table[0] == -1).all())
    _alone(t, slots)


@pytest.mark.parametrize("B,width,pages", [(40, 12, 700), (90, 200, 20000)])
def test_random_forks(B, width, pages):
    """Against the oracle, with prefixes up to the parent's length that have nothing to do with
    the request's own."""
    rng = np.random.default_rng(B)
    T = 40
    s = Steps(B, width, pages, 32, T)
    most = min(width * 32, 700) - T
    ctx = np.where(np.arange(B) % 3 == 0, rng.integers(0, most, B), -1)
    for _ in range(4):
        fresh = ctx < 0
        s.step(ctx, rng.integers(0, T, B))
        roots = np.flatnonzero(~fresh)
        parents = np.where(fresh & (rng.random(B) < 0.7), rng.choice(roots, B), -1)
        ctx = np.where(fresh, rng.integers(0, most, B), np.minimum(ctx + rng.integers(0, 3, B), most))
        prefix = np.minimum(rng.integers(-40, most, B), ctx[parents])
        s.step(ctx, rng.integers(0, T, B), parents, prefix)
        # Forked rows go on alone.
        starts, slots, _ = s.gpu.plan(_i32(ctx), _i32(np.full(B, T - 1)), T)
        assert bool((starts >= 0).all())
        _alone(s.gpu, slots)
        s.table, s.refs = s.gpu.table.cpu().numpy().astype(int), s.gpu.refs.cpu().numpy().astype(int)
        ctx = np.where(rng.random(B) < 0.5, -1, ctx)
        if (ctx < 0).all():
            ctx[0] = 0
