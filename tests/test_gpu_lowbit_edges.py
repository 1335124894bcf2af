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
