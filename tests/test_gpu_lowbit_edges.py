"""Edges of the low-bit operators on the GPU: bytes that no row sees, NaN
groups and bad pages in every way the attention's work is cut, three row tiles,
NaN blocks in the head's largest tiles, and the calls' limits."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, binding as sb
from oracle import lowbit as lb
from tests import test_gpu_attention as ta

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _log(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("K,Hq,Hkv,window,ctx", [
    (2, 4, 2, 40, [100, 70, 45]),            # one row tile, short
    (8, 8, 2, 40, [100, 71, 300]),           # three row tiles (two of 256 channels)
    (8, 16, 2, 7, [77, 1000, 40]),           # four row tiles and more row blocks
    (4, 8, 2, 3000, [9001, 3100, 5017]),     # split over workgroups
])
def test_bytes_before_every_window_are_not_read(D, K, Hq, Hkv, window, ctx):
    """The positions of a tile in front of every row's window may never have
    been written: whatever bytes stand there, outputs are the same bits."""
    _log(f"[attend] before the window D={D} K={K} Hq={Hq} window={window}")
    c = ta.Case(len(ctx), K, Hq, Hkv, D, 32, np.array(ctx), np.full(len(ctx), K), window=window, seed=31)
    clean = c.run()
    c.check(clean)
    kc, vc, ks, vs = lb.tile_addresses(D)
    for byte in (252, 253, 254, 255):
        for b in range(len(ctx)):
            lo = ctx[b] - window + 1         # a window that starts a tile has nothing in front
            tile = c.pool[int(c.table[b, lo // 32]), :, 0]
            for tok in range(lo % 32):
                for at in (kc, vc):
                    tile[:, at[tok]] = 0x7f
                for at in (ks, vs):
                    tile[:, at[tok]] = byte
        got = c.run()
        assert torch.equal(got, clean), byte
        assert int(c.status) == 0


def test_calls_use_the_pool_that_the_cache_holds_now():
    """A pool replaced, or given other storage, between calls; one of another
    shape, type or place is refused."""
    g = torch.Generator(device=DEV).manual_seed(3)
    shape = (4, 2, 1, 34 * 64)
    first, second = (torch.zeros(shape, dtype=torch.uint8, device=DEV) for _ in range(2))
    c = BlockCache(DEV, 4, 2, 64, 32, pool=first)
    k, v = (torch.randn(1, 40, 2, 64, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(1, 3, 4, 64, generator=g, device=DEV).bfloat16()
    table, zero, n = _i32([[3, 1]]), _i32([0]), _i32([40])
    c.write(k, v, table, zero)
    values = c.read(table, None, n, 40)
    out = c.attend(q, table, _i32([37]))
    assert first.any() and out.any()
    c.pool = second
    assert not any(x.any() for x in c.read(table, None, n, 40))
    assert not c.attend(q, table, _i32([37])).any()
    kept = first.clone()
    c.write(k, v, table, zero)
    assert torch.equal(second, kept) and torch.equal(first, kept)
    third = kept.clone()
    second.zero_()
    second.set_(third)                                     # the same tensor, other storage
    assert all(torch.equal(x, y) for x, y in zip(c.read(table, None, n, 40), values))
    assert torch.equal(c.attend(q, table, _i32([37])), out)
    for bad in (kept[:3], kept.to(torch.int8), kept.cpu(), kept.transpose(0, 1)):
        c.pool = bad
        for call in (lambda: c.write(k, v, table, zero), lambda: c.read(table, None, n, 40),
                     lambda: c.attend(q, table, _i32([37]))):
            with pytest.raises(ValueError):
                call()


@pytest.mark.parametrize("K,Hq,ctx", [(3, 4, 90), (8, 16, 90), (4, 8, 5000)])
def test_the_largest_and_smallest_numbers_of_a_request(K, Hq, ctx):
    """Budgets and contexts at the ends of int32, beside a request that is in
    order, under a window and without: flagged, and otherwise what the clamped
    budgets and empty slots give."""
    far = 2**31 - 1
    for window in (0, 50, far):
        c = ta.Case(3, K, Hq, 2, 64, 32, np.array([ctx, ctx - 7, ctx - 20]), np.full(3, K), window=window, seed=5)
        for budgets, lens, clamped, held, flag in (
                ([K, far, -far - 1], c.ctx, [K, K, 0], c.ctx, sb.SV_FLAG_BAD_BUDGET),
                ([K, K, K], [ctx, far, -far - 1], [K, K, K], [ctx, -1, -1], sb.SV_FLAG_BAD_LENGTH)):
            c.budgets, c.ctx = np.array(clamped), np.array(held)
            want = c.run()
            c.check(want)
            c.budgets, c.ctx = np.array(budgets), np.array(lens)
            got = c.run()
            assert int(c.status) == flag
            assert torch.equal(got, want)
    cache = BlockCache(DEV, 3, 2, 64, 32)
    k = torch.ones(3, 4, 2, 64, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache.write(k, k, _i32([[0], [1], [2]]), _i32([0, 0, 0]), _i32([far, -far - 1, 3]), status=status)
    assert int(status) == sb.SV_FLAG_BAD_BUDGET
    one = cache.read(_i32([[0], [1], [2]]), None, _i32([4, 4, 4]), 4)[0]
    assert bool((one[0] == 1).all()) and bool((one[1, 0] == 1).all()) and not one[1, 1:].any() and bool((one[2] == 1).all())


def test_many_shapes_leave_little_behind():
    """A table width and batch per call, as a server has them: what is kept of
    the shapes stays bounded, and the sizes stay those of the shapes."""
    c = BlockCache(DEV, 1, 1, 64, 32)
    q = torch.zeros(0, 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    for width in range(1, 1500):
        c.attend(q, torch.zeros(0, width, dtype=torch.int32, device=DEV), _i32([]))
    held = [len(x) for x in vars(c).values() if isinstance(x, (dict, list, set))]
    assert max(held, default=0) <= 1024
    for width in (1, 700, 1499, 1, 5000):
        assert sb._attention_bytes(2, 3, 4, 1, 64, 32, width, 0) == \
            sb.spec_verify_attention_workspace_bytes(2, 3, 4, 1, 64, 32, width, 0)
    assert sb._attention_bytes.cache_info().currsize <= 1024
