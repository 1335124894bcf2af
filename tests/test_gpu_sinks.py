"""Attention under a window with sinks against the fp64 oracle on the same bytes.

Tolerance: as for the attention without sinks. With A = sum_j p_j |v_j| and S the
largest sum_i |scale q_i k_i| of a row's positions, a score is off by at most
(D + 2) 2^-24 S, its probability by twice that and by 2^-20 for the exponential
and the sums (up to 4,096 terms); probabilities and outputs are rounded to bf16,
half a step of 2^-8 each:
|got - ref| <= (2^-8 + 2 (D + 2) 2^-24 S + 2^-20 (1 + n / 4096)) A + 2^-8 (1 + 2^-7) |ref|."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, binding as sb
from oracle import lowbit as lb, serving as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _log(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _bound(ref, mag, reach, D, n):
    rel = 2.0 ** -8 + 2 * (D + 2) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20 * (1 + n / 4096)
    return rel * mag + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(ref) + 1e-30


class Case:
    """A filled cache with NaN scales everywhere that no row sees (behind the
    blocks, between sinks and windows), and no page where none is needed."""

    def __init__(self, Hq, Hkv, D, page, ctx, budgets, window, sinks, K=None, seed=0):
        rng = np.random.default_rng(seed)
        self.ctx, self.budgets = np.asarray(ctx), np.asarray(budgets)
        B, K = len(self.ctx), int(self.budgets.max()) if K is None else K
        self.__dict__.update(B=B, K=K, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window, sinks=sinks)
        total = np.where(self.ctx < 0, 0, self.ctx + self.budgets + 1)
        width = max(1, -(-int(total.max()) // page)) + 1
        need = [sorted(sv.needed_pages(int(c), int(k) + 1, page, window, sinks)) for c, k in zip(self.ctx, self.budgets)]
        self.pages = sum(map(len, need)) + 2
        order = iter(rng.permutation(self.pages))
        self.table = np.full((B, width), -7)
        n = (self.pages, Hkv, page // 32)
        self.pool = rng.integers(0, 256, n + (34 * D,)).astype(np.uint8)
        self.pool[..., 32 * D:] = rng.integers(123, 129, n + (2 * D,))
        _, _, ks, vs = lb.tile_addresses(D)
        for b in range(B):
            seen = {j for t in range(self.budgets[b] + 1) for j in sv.visible(int(self.ctx[b]) + t, window, sinks)} \
                if self.ctx[b] >= 0 else set()
            for i in need[b]:
                self.table[b, i] = next(order)
                for pos in range(i * page, (i + 1) * page):
                    if pos not in seen:
                        for at in (ks, vs):
                            self.pool[self.table[b, i], :, pos % page // 32, at[pos % 32]] = 255 if pos % 3 else 0
        self.q = torch.tensor(rng.normal(size=(B, K + 1, Hq, D))).bfloat16()

    def run(self, **kw):
        self.cache = BlockCache(DEV, self.pages, self.Hkv, self.D, self.page, pool=torch.tensor(self.pool).to(DEV))
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        return self.cache.attend(self.q.to(DEV), _i32(self.table), _i32(self.ctx), _i32(self.budgets),
                                 window=self.window, sinks=self.sinks, status=self.status, **kw)

    def check(self, got, scale=None, fill=0.0):
        got = got.double().cpu().numpy()
        scale = self.D ** -0.5 if scale is None else scale
        for b in range(self.B):
            n = 0 if self.ctx[b] < 0 else self.budgets[b] + 1
            assert np.all(got[b, n:] == fill), b
            if not n:
                continue
            total = int(self.ctx[b]) + n
            row = np.where(self.table[b] < 0, 0, self.table[b])
            k, v = lb.read(self.pool, row, 0, total, self.D, self.page)
            ref, mag, reach = sv.attend(self.q[b, :n].double().numpy(), k, v, int(self.ctx[b]), scale, self.window, self.sinks)
            err, tol = np.abs(got[b, :n] - ref), _bound(ref, mag, reach, self.D, total)
            assert np.all(err <= tol), (b, float(np.nanmax(err / tol)))
        assert int(self.status) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 4), (33, 32), (40, 33), (64, 64), (100, 150), (300, 5), (2000, 70)])
def test_windows_and_sinks(D, window, sinks):
    """Sinks that end inside a tile, at its end, behind the window's start; windows
    that reach position 0, blocks inside the sinks."""
    _log(f"[sinks] D={D} window={window} sinks={sinks}")
    ctx = np.array([0, 1, 31, 32, 63, 97, -1, 160, 300, 700, 1023])
    rng = np.random.default_rng(window)
    c = Case(4, 2, D, 32, ctx, rng.integers(0, 7, ctx.size), window, sinks, K=6, seed=window + D)
    c.check(c.run())


@pytest.mark.parametrize("K,Hq,Hkv,D,page", [(0, 4, 4, 128, 64), (8, 8, 1, 64, 128), (32, 4, 2, 128, 32),
                                             (32, 6, 2, 256, 64), (2, 3, 1, 256, 256), (15, 16, 4, 64, 32)])
def test_heads_and_blocks(K, Hq, Hkv, D, page):
    _log(f"[sinks] K={K} Hq={Hq} Hkv={Hkv} D={D} page={page}")
    ctx = np.array([5, 250, 77, 1300])
    c = Case(Hq, Hkv, D, page, ctx, np.array([K, K, K // 2, 0]), 90, 41, K=K, seed=K)
    c.check(c.run())


@pytest.mark.parametrize("Hq,Hkv,D,window,sinks", [(8, 2, 128, 9000, 3000), (4, 1, 64, 5000, 12001), (2, 2, 256, 3000, 40)])
def test_long_spans_split_over_workgroups(Hq, Hkv, D, window, sinks):
    _log(f"[sinks] long Hq={Hq} Hkv={Hkv} D={D} window={window} sinks={sinks}")
    c = Case(Hq, Hkv, D, 64, np.array([20011, 3, 511, 13000]), np.array([4, 0, 4, 2]), window, sinks, seed=7)
    c.check(c.run())


def test_a_window_over_everything_is_the_attention_without_one():
    """Bit for bit where the tiles are taken in the same order: sinks in the window's reach add nothing."""
    c = Case(8, 2, 128, 64, np.array([200, 31, 900]), np.array([4, 2, 0]), 5000, 100)
    got = c.run()
    plain = c.cache.attend(c.q.to(DEV), _i32(c.table), _i32(c.ctx), _i32(c.budgets))
    assert torch.equal(got, plain)
    # And no sinks, or no window, is the call without them.
    w = Case(8, 2, 128, 64, np.array([200, 31, 900]), np.array([4, 2, 0]), 70, 0)
    got = w.run()
    assert torch.equal(got, w.cache.attend(w.q.to(DEV), _i32(w.table), _i32(w.ctx), _i32(w.budgets), window=70))
    assert torch.equal(c.cache.attend(c.q.to(DEV), _i32(c.table), _i32(c.ctx), _i32(c.budgets), sinks=9), plain)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_sink_reaches_the_rows_that_see_it_and_no_others(D):
    """A NaN group of a value, then of a key, in a sink, behind the sinks, in the window."""
    window, sinks, K = 40, 37, 5
    base = Case(4, 2, D, 32, np.array([33, 300]), np.array([K, K]), window, sinks, seed=3)
    clean = base.run().double().cpu().numpy()
    _, _, ks, vs = lb.tile_addresses(D)
    g = D // 32 - 1
    for b, where in ((0, 36), (0, 38), (1, 0), (1, 36), (1, 37), (1, 262), (1, 303)):
        for side in ("value", "key"):
            c = Case(4, 2, D, 32, np.array([33, 300]), np.array([K, K]), window, sinks, seed=3)
            c.pool[int(c.table[b, where // 32]), 1, 0, (vs if side == "value" else ks)[where % 32, g]] = 255
            got = c.run().double().cpu().numpy()
            want = clean.copy()
            for t in range(K + 1):
                if where in sv.visible(int(c.ctx[b]) + t, window, sinks):
                    if side == "value":
                        want[b, t, 2:, 32 * g:] = np.nan
                    else:
                        want[b, t, 2:] = np.nan
            assert np.array_equal(np.isnan(got), np.isnan(want)), (D, b, where, side)
            assert np.array_equal(got, want, equal_nan=True)


def test_pages_between_sinks_and_windows_are_not_needed_and_others_are_flagged():
    c = Case(4, 2, 64, 32, np.array([500, 40]), np.array([3, 1]), 50, 40, seed=4)
    good = c.run()
    c.check(good)
    keep = c.table.copy()
    for i in (0, 1, 15):
        c.table = keep.copy()
        c.table[0, i] = c.pages
        got = c.run()
        assert int(c.status) == sb.SV_FLAG_BAD_PAGE and torch.equal(got[1], good[1])


def test_the_ends_of_the_numbers():
    """Windows and sinks of 2^31 - 1, lengths at the ends of int32."""
    c = Case(4, 2, 64, 32, np.array([70, -2**31, 5]), np.array([3, 0, 1]), 2**31 - 1, 2**31 - 1, seed=5)
    got = c.run()
    c.check(got)
    c.window = 3
    again = c.run()
    c.check(again)                           # all sinks
    c.ctx[1] = 2**31 - 1
    assert torch.equal(c.run(), again) and int(c.status) == sb.SV_FLAG_BAD_LENGTH
    for bad in (dict(window=-1), dict(sinks=-1), dict(sinks=2**31), dict(window=2**31)):
        with pytest.raises(ValueError):
            c.cache.attend(c.q.to(DEV), _i32(c.table), _i32(c.ctx), **{**dict(window=3, sinks=4), **bad})


def test_replayed_on_another_stream_and_with_what_stays():
    c = Case(8, 2, 128, 64, np.array([5000, 100, -1, 17]), np.array([4, 2, 0, 0]), 3000, 70, seed=6)
    want = c.run(out=torch.full((4, 5, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV))
    c.check(want, fill=3.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(stream=side, out=torch.full_like(want, 3.0))
    side.synchronize()
    assert torch.equal(got, want)
    args = c.q.to(DEV), _i32(c.table), _i32(c.ctx), _i32(c.budgets)
    outs, graphs = [torch.full_like(want, 3.0) for _ in range(2)], []
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.cache.attend(*args, window=c.window, sinks=c.sinks, out=out)
        graphs.append(graph)
    for _ in range(3):
        for graph, out in zip(graphs, outs):
            out.fill_(3.0)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
