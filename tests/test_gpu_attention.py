"""Attention of drafted blocks over the 4-bit cache against the fp64 oracle on
the same bytes.

Tolerance, from the arithmetic. With A = sum_j p_j |v_j| and S the largest
sum_i |scale q_i k_i| of a row's positions:
  - a score is an fp32 sum of D exact products, then one fp32 product: off by
    at most (D + 2) 2^-24 S; its probability (numerator and denominator) by
    twice that, and by 2^-21 for exp2 and the sums' rounding per 4096 terms;
  - probabilities are rounded to bf16 for the value product: half a step,
    2^-8, relative each;
  - the output is rounded to bf16: 2^-8 of itself.
So |got - ref| <= (2^-8 + 2 (D + 2) 2^-24 S + 2^-20 (1 + n / 4096)) A + 2^-8 |ref|
(1 + 2^-7)."""
import math
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, binding as sb
from oracle import lowbit as lb
from tests.test_gpu_cache import make_table

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
    """A filled cache (random bytes with sane scales, 255 and garbage behind
    every request's end) and queries."""

    def __init__(self, B, K, Hq, Hkv, D, page, ctx, budgets, window=0, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.__dict__.update(B=B, K=K, Hq=Hq, Hkv=Hkv, D=D, page=page, window=window)
        self.ctx, self.budgets = np.asarray(ctx), np.asarray(budgets)
        self.total = np.where(self.ctx < 0, 0, self.ctx + self.budgets + 1)
        need = int((-(-self.total // page)).sum())
        width = max(1, -(-int(self.total.max()) // page)) + 1
        self.pages = need + spare
        self.table = make_table(rng, self.total, page, width, self.pages)
        n = (self.pages, Hkv, page // 32)
        pool = rng.integers(0, 256, n + (34 * D,)).astype(np.uint8)
        pool[..., 32 * D:] = rng.integers(123, 129, n + (2 * D,))
        # Behind the last token of every request: every kind of byte, NaN scales.
        kc, vc, ks, vs = lb.tile_addresses(D)
        for b in range(B):
            t = int(self.total[b])
            if t % page:
                pg = int(self.table[b, t // page])
                for pos in range(t, -(-t // page) * page):
                    for at in (ks, vs):
                        pool[pg, :, pos % page // 32, at[pos % 32]] = 255 if pos % 3 else 0
        self.pool = pool
        # Pages before a window are never needed.
        if window:
            for b in range(B):
                first = max(0, self.ctx[b] - window + 1) // page
                self.table[b, :first] = -7
        self.q = torch.tensor(rng.normal(size=(B, K + 1, Hq, D))).bfloat16()

    def run(self, out=None, scale=None, q=None, status=None, **kw):
        self.cache = BlockCache(DEV, self.pages, self.Hkv, self.D, self.page,
                                pool=torch.tensor(self.pool).to(DEV))
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV) if status is None else status
        return self.cache.attend(self.q.to(DEV) if q is None else q, _i32(self.table),
                                 _i32(self.ctx), _i32(self.budgets), scale=scale,
                                 window=self.window, out=out, status=self.status, **kw)

    def reference(self, b, scale=None):
        scale = self.D ** -0.5 if scale is None else scale
        first = max(0, int(self.ctx[b]) - self.window + 1) if self.window else 0
        n = int(self.total[b]) - first
        k, v = lb.read(self.pool, self.table[b], first, n, self.D, self.page)
        q = self.q[b, :self.budgets[b] + 1].double().numpy()
        return lb.attend(q, k, v, first, int(self.ctx[b]), scale, self.window), n

    def check(self, got, scale=None, fill=0.0):
        got = got.double().cpu().numpy()
        for b in range(self.B):
            n_rows = 0 if self.ctx[b] < 0 else self.budgets[b] + 1
            assert np.all(got[b, n_rows:] == fill), b
            if not n_rows:
                continue
            (ref, mag, reach), n = self.reference(b, scale)
            err = np.abs(got[b, :n_rows] - ref)
            tol = _bound(ref, mag, reach, self.D, n)
            assert np.all(err <= tol), (b, float(np.nanmax(err / tol)))
        assert int(self.status) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("K,Hq,Hkv", [(0, 4, 4), (5, 8, 2), (8, 8, 1), (2, 3, 1), (32, 4, 2)])
@pytest.mark.parametrize("page", [32, 128])
def test_shapes(D, K, Hq, Hkv, page):
    _log(f"[attend] D={D} K={K} Hq={Hq} Hkv={Hkv} page={page}")
    rng = np.random.default_rng(K)
    ctx = np.array([0, 1, 31, 32, 33, 95, -1, 300])
    budgets = rng.integers(0, K + 1, ctx.size)
    budgets[0], budgets[4] = 0, K
    c = Case(ctx.size, K, Hq, Hkv, D, page, ctx, budgets, seed=D + K)
    c.check(c.run())


@pytest.mark.parametrize("D,window", [(64, 1), (64, 40), (128, 7), (128, 33), (128, 64), (256, 100)])
def test_sliding_windows(D, window):
    _log(f"[attend] D={D} window={window}")
    ctx = np.array([0, 5, 64, 97, 700, 1023])
    c = Case(ctx.size, 6, 6, 2, D, 32, ctx, np.array([6, 0, 3, 6, 6, 2]), window=window, seed=window)
    c.check(c.run())


@pytest.mark.parametrize("D,Hq,Hkv,K", [(128, 8, 2, 4), (64, 16, 1, 8), (256, 2, 2, 0)])
def test_long_contexts_split_over_workgroups(D, Hq, Hkv, K):
    """Few requests and long contexts of very different lengths: the two-launch
    form, with splits that only some requests have."""
    ctx = np.array([20011, 3, 511, 9000])
    c = Case(4, K, Hq, Hkv, D, 64, ctx, np.array([K, 0, K, K // 2]), seed=7)
    _log(f"[attend] long D={D} Hq={Hq} Hkv={Hkv} K={K}")
    c.check(c.run())


def test_many_requests_in_one_launch():
    rng = np.random.default_rng(5)
    B = 300
    ctx = rng.integers(-1, 200, B)
    c = Case(B, 3, 8, 4, 64, 32, ctx, rng.integers(0, 4, B), seed=8)
    c.check(c.run())


def _check_on_gpu(cache, q, got, table, ctx, budgets, window=0):
    """Every row against fp64 products on the GPU of the values that the cache
    reads back (which are exact, tested on their own): for batches too large
    for the CPU."""
    B, T, Hq, D = q.shape
    Hkv = cache.kv_heads
    for b in range(B):
        c, k = int(ctx[b]), int(budgets[b])
        if c < 0:
            assert not got[b].any()
            continue
        first = max(0, c - window + 1) if window else 0
        n = c + k + 1 - first
        keys, values = cache.read(table[b:b + 1], _i32([first]), _i32([n]), n, dtype=torch.float32)
        keys, values = (x[0].double().permute(1, 0, 2).contiguous() for x in (keys, values))
        rows = q[b, :k + 1].double().unflatten(1, (Hkv, Hq // Hkv)).permute(1, 0, 2, 3).flatten(1, 2)
        z = rows @ keys.transpose(1, 2) * D ** -0.5
        pos = torch.arange(first, first + n, device=DEV)
        row = (c + torch.arange(k + 1, device=DEV)).repeat_interleave(Hq // Hkv)[:, None]
        hidden = (pos > row) | ((pos <= row - window) if window else False)
        p = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
        ref, mag = p @ values, p @ values.abs()
        reach = (rows.abs() @ keys.abs().transpose(1, 2)).amax(-1, keepdim=True) * D ** -0.5
        tol = (2.0 ** -8 + 2 * (D + 2) * 2.0 ** -24 * reach + 2.0 ** -20 * (1 + n / 4096)) * mag \
            + 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 1e-30
        mine = got[b, :k + 1].double().unflatten(1, (Hkv, Hq // Hkv)).permute(1, 0, 2, 3).flatten(1, 2)
        assert bool(((mine - ref).abs() <= tol).all()), (b, float(((mine - ref).abs() / tol).max()))
        assert not got[b, k + 1:].any()


@pytest.mark.parametrize("B,K,Hq,Hkv,D,lo,hi,window", [
    (8, 8, 224, 32, 64, 3000, 15000, 0),       # ragged, long: equal shares, units in several parts
    (140, 2, 16, 8, 128, 300, 9000, 0),        # more units than workgroups
    (500, 1, 16, 16, 64, 30, 1500, 0),         # a workgroup per unit, many of them
    (6, 8, 64, 1, 128, 2000, 9000, 0),         # 576 rows a request: row blocks of one unit
    (3, 32, 16, 2, 256, 1500, 6000, 0),        # 264 rows a head of 256 channels
    (24, 5, 16, 8, 256, 200, 5000, 1024),      # windows, units of nearly one size
    (2, 3, 8, 2, 128, 30000, 60000, 0),        # few units, many parts
])
def test_every_way_the_work_is_cut(B, K, Hq, Hkv, D, lo, hi, window):
    _log(f"[attend] B={B} K={K} Hq={Hq} Hkv={Hkv} D={D} ctx {lo}..{hi} window={window}")
    g = torch.Generator(device=DEV).manual_seed(B + K)
    ctx = torch.randint(lo, hi + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    ctx[B // 2] = lo
    ctx[0] = hi
    budgets = torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    if B > 2:
        ctx[1] = -1
    page = 64
    need = (ctx.clamp_min(0) + budgets + page) // page
    first = torch.cumsum(need, 0) - need
    width, pages = int(need.max()), int(need.sum())
    col = torch.arange(width, device=DEV)
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp_max(pages - 1)], -1).int()
    cache = BlockCache(DEV, pages, Hkv, D, page)
    cache.pool.random_(0, 256, generator=g)
    cache.pool[..., 32 * D:].random_(122, 129, generator=g)
    q = torch.randn(B, K + 1, Hq, D, generator=g, device=DEV).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = cache.attend(q, table, ctx, budgets, window=window, status=status)
    _check_on_gpu(cache, q, got, table, ctx.tolist(), budgets.tolist(), window)
    assert int(status) == 0
    assert torch.equal(cache.attend(q, table, ctx, budgets, window=window), got)


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_and_sharp_softmax(scale):
    c = Case(3, 4, 4, 2, 128, 64, np.array([100, 0, 1000]), np.array([4, 4, 2]), seed=3)
    c.check(c.run(scale=scale), scale=scale)


def test_rows_behind_the_budget_and_empty_slots_keep_their_values():
    c = Case(4, 5, 4, 2, 64, 32, np.array([40, -1, 3, -2**31]), np.array([2, 5, 0, 3]), seed=2)
    out = torch.full((4, 6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    got = c.run(out=out)
    assert got is out
    c.check(got, fill=3.0)


def test_queries_as_a_slice_of_a_fused_projection():
    c = Case(3, 4, 8, 2, 128, 64, np.array([70, 5, 129]), np.array([4, 1, 3]), seed=4)
    fused = torch.full((3, 5, 12 * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[..., :8 * 128] = c.q.to(DEV).flatten(2)
    got = c.run(q=fused[..., :8 * 128].unflatten(-1, (8, 128)))
    c.check(got)
    assert torch.equal(got, c.run())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 3])
def test_a_nan_token_reaches_the_rows_that_see_it_and_no_others(D, window):
    """A drafted token whose value group, then whose key, is NaN; with a window
    also a context token that only the first rows see."""
    K, ctx, page = 5, 45, 32
    for where, side in ((ctx + 3, "value"), (ctx + 3, "key"), (ctx - 1, "value"), (ctx, "key")):
        c = Case(1, K, 4, 2, D, page, np.array([ctx]), np.array([K]), window=window, seed=11)
        clean = c.run().double().cpu().numpy()
        kc, vc, ks, vs = lb.tile_addresses(D)
        g = D // 32 - 1
        at = (vs if side == "value" else ks)[where % 32, g]
        c.pool[int(c.table[0, where // page]), 1, where % page // 32, at] = 255
        got = c.run().double().cpu().numpy()
        want = clean.copy()
        for t in range(K + 1):
            p = ctx + t
            if where <= p and (not window or where > p - window):
                if side == "value":
                    want[0, t, 2:, 32 * g:] = np.nan       # heads of kv head 1, its group
                else:
                    want[0, t, 2:] = np.nan
        assert np.array_equal(np.isnan(got), np.isnan(want)), (D, where, side)
        assert np.array_equal(got, want, equal_nan=True)


def test_bad_budgets_lengths_and_pages_are_flagged():
    c = Case(2, 3, 2, 1, 64, 32, np.array([40, 10]), np.array([3, 2]), seed=6)
    good = c.run()
    c.check(good)
    keep = c.table.copy()
    for bad in (-1, c.pages, 2**31 - 1):
        c.table = keep.copy()
        c.table[0, 1] = bad
        got = c.run()
        assert int(c.status) == sb.SV_FLAG_BAD_PAGE
        assert torch.equal(got[1], good[1])                # the other request is untouched
    c.table = keep
    c.ctx = np.array([32 * keep.shape[1] - 3, 10])
    got = c.run()
    assert int(c.status) == sb.SV_FLAG_BAD_LENGTH
    assert torch.equal(got[1], good[1]) and not got[0].any()
    c.ctx = np.array([40, 10])
    c.budgets = np.array([77, -4])
    got = c.run()
    assert int(c.status) == sb.SV_FLAG_BAD_BUDGET
    assert torch.equal(got[0], good[0]) and torch.equal(got[1, 0], good[1, 0])
    assert not got[1, 1:].any()


def test_no_budgets_means_the_whole_block():
    c = Case(2, 3, 4, 2, 64, 32, np.array([40, 10]), np.array([3, 3]), seed=6)
    want = c.run()
    got = c.cache.attend(c.q.to(DEV), _i32(c.table), _i32(c.ctx))
    assert torch.equal(got, want)


def test_a_pool_past_32_bit_offsets():
    Hkv, D, page = 8, 128, 128
    per = Hkv * (page // 32) * 34 * D
    pages = (1 << 32) // per + 16
    pool = torch.zeros((pages, Hkv, page // 32, 34 * D), dtype=torch.uint8, device=DEV)
    big = BlockCache(DEV, pages, Hkv, D, page, pool=pool)
    small = BlockCache(DEV, 4, Hkv, D, page)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = (torch.randn(1, 300, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(1, 3, 16, D, generator=g, device=DEV).bfloat16()
    got = []
    for c, row in ((big, [pages - 1, 3, pages - 2]), (small, [0, 1, 2])):
        c.write(k, v, _i32([row]), _i32([0]))
        got.append(c.attend(q, _i32([row]), _i32([297])))
    assert torch.equal(got[0], got[1]) and got[0].any()


def test_the_result_does_not_depend_on_the_run_the_stream_or_a_replay():
    """Bit-equal on a second run, on another stream, and in a captured graph
    replayed between eager calls, with two graphs captured one after another."""
    c = Case(3, 4, 8, 2, 128, 64, np.array([5000, 100, 17]), np.array([4, 2, 0]), seed=12)
    want = c.run()
    assert torch.equal(c.run(), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    table, ctx, budgets, q = _i32(c.table), _i32(c.ctx), _i32(c.budgets), c.q.to(DEV)
    outs = [torch.zeros_like(want) for _ in range(2)]
    graphs = []
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.cache.attend(q, table, ctx, budgets, out=out)
        graphs.append(graph)
    for _ in range(4):
        for graph, out in zip(graphs, outs):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert torch.equal(c.cache.attend(q, table, ctx, budgets), want)
    # New lengths under the same graph.
    ctx.copy_(_i32([4000, -1, 18]))
    eager = c.cache.attend(q, table, ctx, budgets)
    outs[0].zero_()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager)


def test_python_refusals():
    c = BlockCache(DEV, 4, 2, 64, 32)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    table, one = _i32([[0]]), _i32([0])
    for bad in (q.float(), q[..., :32], q[:, :, :3], q.transpose(1, 2)):
        with pytest.raises(ValueError):
            c.attend(bad, table, one)
    with pytest.raises(ValueError):
        c.attend(q, table, one, window=-1)
    with pytest.raises(RuntimeError):
        c.attend(q, table, one, scale=math.nan)
    with pytest.raises(ValueError):
        c.attend(q, table, one, out=torch.zeros(1, 2, 4, 64, device=DEV))
    with pytest.raises(ValueError):
        c.attend(torch.zeros(1, 40, 4, 64, dtype=torch.bfloat16, device=DEV), table, one)


def test_two_streams_at_once_over_shared_pages():
    """Requests that share the pages of a prefix, attended on two streams at
    the same time: each call has its own workspace."""
    Hq, Hkv, D, page = 16, 4, 128, 64
    g = torch.Generator(device=DEV).manual_seed(14)
    cache = BlockCache(DEV, 220, Hkv, D, page)
    cache.pool.random_(0, 256, generator=g)
    cache.pool[..., 32 * D:].random_(122, 129, generator=g)
    table = torch.arange(200, device=DEV).repeat(4, 1).int()
    table[:, 199] = _i32([200, 201, 202, 203])               # every request's own last page
    ctx, budgets = _i32([12736, 12790, 12750, 7000]), _i32([4, 4, 0, 2])
    q = [torch.randn(4, 5, Hq, D, generator=g, device=DEV).bfloat16() for _ in range(2)]
    want = [cache.attend(x, table, ctx, budgets) for x in q]
    _check_on_gpu(cache, q[0], want[0], table, ctx, budgets)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append(cache.attend(q[i], table, ctx, budgets, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


@pytest.mark.parametrize("K,window", [(0, 0), (3, 0), (3, 2**31 - 1)])
def test_the_longest_context(K, window):
    """2^24 positions over eight pages of 4,096 tokens in turn. Rows at the end
    see every position before the block's first exactly as often, so K = 0 is
    attention over the 32,768 distinct tokens."""
    D, page, per = 64, 4096, 8
    n = 1 << 24
    _log(f"[attend] {n} positions, K={K} window={window}")
    g = torch.Generator(device=DEV).manual_seed(15)
    cache = BlockCache(DEV, per, 1, D, page)
    cache.pool.random_(0, 256, generator=g)
    cache.pool[..., 32 * D:].random_(122, 129, generator=g)
    table = (torch.arange(n // page, device=DEV) % per).int()[None]
    q = torch.randn(1, K + 1, 2, D, generator=g, device=DEV).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = cache.attend(q, table, _i32([n - 1 - K]), window=window, status=status)
    assert int(status) == 0
    keys, values = cache.read(table[:, :per], None, _i32([per * page]), per * page, dtype=torch.float32)
    keys, values = keys[0, :, 0].double(), values[0, :, 0].double()
    rows = q[0].double().flatten(0, 1)                       # (t, head)
    z = rows @ keys.t().contiguous() * D ** -0.5
    # How often row t sees each token: the last K - t positions are hidden.
    seen = torch.full((K + 1, per * page), float(n // (per * page)), device=DEV).double()
    for t in range(K):
        seen[t, per * page - K + t:] -= 1.0
    seen = seen.repeat_interleave(2, 0)
    w = seen * torch.exp(z - z.amax(1, keepdim=True))
    p = w / w.sum(1, keepdim=True)
    ref, mag = p @ values, p @ values.abs()
    reach = (rows.abs() @ keys.abs().t().contiguous()).amax(1, keepdim=True) * D ** -0.5
    tol = (2.0 ** -8 + 2 * (D + 2) * 2.0 ** -24 * reach + 2.0 ** -20 * (1 + n / 4096)) * mag \
        + 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 1e-30
    err = (got[0].double().flatten(0, 1) - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    # A position more does not fit.
    cache.attend(q, table, _i32([n - K]), status=status)
    assert int(status) == sb.SV_FLAG_BAD_LENGTH


def test_the_largest_batch():
    """16,384 single tokens, 256 heads that share nothing."""
    B, heads, D = 16384, 256, 64
    g = torch.Generator(device=DEV).manual_seed(16)
    cache = BlockCache(DEV, 2, heads, D, 32)
    cache.pool.random_(0, 256, generator=g)
    cache.pool[..., 32 * D:].random_(122, 129, generator=g)
    table = torch.tensor([[0, 1], [1, 0]], device=DEV).repeat(B // 2, 1).int()
    ctx = torch.arange(B, device=DEV, dtype=torch.int32) % 61 - 1       # -1..59, in turn
    q = torch.randn(61 * 2, 1, heads, D, generator=g, device=DEV).bfloat16()
    q = q.repeat(B // 122 + 1, 1, 1, 1)[:B].contiguous()
    got = cache.attend(q, table, ctx)
    period = 122
    _check_on_gpu(cache, q[:period], got[:period], table, ctx, torch.zeros(period, dtype=torch.int32))
    whole = B // period * period
    assert torch.equal(got[:whole].view(-1, period, heads * D),
                       got[:period].view(1, period, heads * D).expand(B // period, -1, -1))
    assert torch.equal(got[whole:], got[:B - whole])
    none = cache.attend(q[:0], table[:0], ctx[:0])
    assert none.shape == (0, 1, heads, D)


def test_windows_beyond_32_bits_are_refused():
    c = BlockCache(DEV, 4, 2, 64, 32)
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16, device=DEV)
    for window in (2**31, 2**32, 2**32 + 5, -2**32):
        with pytest.raises(ValueError):
            c.attend(q, _i32([[0]]), _i32([0]), window=window)


def test_scales_near_the_largest():
    """A scale whose product with log2(e) is no longer finite: equal scores
    still share the weight, a larger one takes it all."""
    c = BlockCache(DEV, 1, 1, 64, 32)
    k, v = (torch.zeros(1, 4, 1, 64, device=DEV) for _ in range(2))
    k[0, 2, 0, 0] = 1.0
    v[0, :, 0, 0] = torch.tensor([1.0, 2.0, 4.0, 3.0], device=DEV)
    table = _i32([[0]])
    c.write(k, v, table, _i32([0]))
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 3, 0, 0] = 2.0 ** -100
    got = c.attend(q, table, _i32([0]), scale=3.0e38)[0, :, 0, 0].tolist()
    assert got[0] == 1.0 and got[1] == 1.5 and abs(got[2] - 7 / 3) <= 2.0 ** -7 * 7 / 3 and got[3] == 4.0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,K,Hq,Hkv,ctx,window", [
    (1, 0, 16, 1, [900], 0), (4, 0, 8, 8, [0, 990, -1, 31], 0), (32, 1, 16, 8, None, 0),
    (33, 1, 16, 8, None, 0),                    # past 256 units: fewer wavefronts
    (5, 3, 8, 2, [700, 1, 32, 512, 63], 65),
])
def test_few_short_units(B, K, Hq, Hkv, ctx, window, D):
    """Short contexts of few units, whose workgroups have twice the wavefronts:
    more of them than tiles, tiles in two and more rounds, windows."""
    rng = np.random.default_rng(B + D)
    ctx = rng.integers(0, 600, B) if ctx is None else np.array(ctx)
    c = Case(B, K, Hq, Hkv, D, 32, ctx, rng.integers(0, K + 1, B), window=window, seed=21)
    got = c.run()
    c.check(got)
    assert torch.equal(c.run(), got)
