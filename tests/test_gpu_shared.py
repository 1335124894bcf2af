"""Attention behind shared prefixes against fp64 products on the GPU of the values
that the cache reads back (which are exact, tested on their own), and against
the attention that shares nothing.

Tolerance: as for the attention itself. With A = sum_j p_j |v_j| and S the
largest sum_i |scale q_i k_i| of a row's positions, a score is off by at most
(D + 2) 2^-24 S, its probability by twice that and by 2^-20 (1 + n / 4096) for
the exponential, the sums and their joins; probabilities and outputs are rounded
to bf16, half a step of 2^-8 each:
|got - ref| <= (2^-8 + 2 (D + 2) 2^-24 S + 2^-20 (1 + n / 4096)) A + 2^-8 (1 + 2^-7) |ref|."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, binding as sb
from oracle import lowbit as lb

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _log(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


class Case:
    """Requests with group numbers; those of a group hold the pages that lie
    wholly in its first lens[g] tokens in common. Behind every request's end the
    cache holds NaN scales."""

    def __init__(self, groups, lens, ctx, budgets, K, Hq, Hkv, D, page, seed=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.groups, self.lens = np.asarray(groups), np.asarray(lens)
        self.ctx, self.budgets = np.asarray(ctx), np.asarray(budgets)
        B = len(self.ctx)
        self.__dict__.update(B=B, K=K, Hq=Hq, Hkv=Hkv, D=D, page=page)
        total = np.where(self.ctx < 0, 0, self.ctx + self.budgets + 1)
        width = max(1, -(-int(total.max()) // page)) + 1
        self.pages = int((-(-total // page)).sum()) + 3
        order = iter(rng.permutation(self.pages))
        self.table, common = np.full((B, width), -1), {}
        ends = []
        for b in range(B):
            grp = int(self.groups[b])
            for i in range(-(-int(total[b]) // page)):
                if 0 <= grp < len(self.lens) and (i + 1) * page <= min(self.lens[grp], self.ctx[b]):
                    if (grp, i) not in common:
                        common[grp, i] = next(order)
                    self.table[b, i] = common[grp, i]
                else:
                    self.table[b, i] = next(order)
            if total[b] > 0 and total[b] % page:
                ends.append((self.table[b, total[b] // page], int(total[b]) % page))
        self.cache = BlockCache(DEV, self.pages, Hkv, D, page)
        pool = self.cache.pool
        pool.random_(0, 256, generator=g)
        pool[..., 32 * D:].random_(122, 129, generator=g)
        _, _, ks, vs = lb.tile_addresses(D)
        for pg, n in ends:
            for tile in range(n // 32, page // 32):
                at = np.concatenate([a[t].ravel() for a in (ks, vs) for t in range(32) if 32 * tile + t >= n])
                pool[int(pg), :, tile, torch.tensor(at, device=DEV)] = 255
        self.q = torch.randn(B, K + 1, Hq, D, generator=g, device=DEV).bfloat16()
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, **kw):
        self.status.zero_()
        return self.cache.attend_shared(self.q, _i32(self.table), _i32(self.ctx), _i32(self.groups), _i32(self.lens),
                                        _i32(self.budgets), status=self.status, **kw)

    def plain(self, **kw):
        return self.cache.attend(self.q, _i32(self.table), _i32(self.ctx), _i32(self.budgets), **kw)

    def check(self, got, fill=0.0, scale=None):
        D, Hkv, group = self.D, self.Hkv, self.Hq // self.Hkv
        scale = D ** -0.5 if scale is None else scale
        for b in range(self.B):
            c, k = int(self.ctx[b]), int(self.budgets[b])
            if c < 0:
                assert bool((got[b] == fill).all())
                continue
            n = c + k + 1
            keys, values = self.cache.read(_i32(self.table[b:b + 1]), None, _i32([n]), n, dtype=torch.float32)
            keys, values = (x[0].double().permute(1, 0, 2).contiguous() for x in (keys, values))
            by_head = lambda x: x.unflatten(1, (Hkv, group)).permute(1, 0, 2, 3).flatten(1, 2)
            rows = by_head(self.q[b, :k + 1].double())
            z = rows @ keys.transpose(1, 2).contiguous() * scale
            row = (c + torch.arange(k + 1, device=DEV)).repeat_interleave(group)[:, None]
            p = torch.softmax(z.masked_fill(torch.arange(n, device=DEV) > row, -float("inf")), -1)
            ref, mag = p @ values, p @ values.abs()
            reach = (rows.abs() @ keys.abs().transpose(1, 2).contiguous()).amax(-1, keepdim=True) * abs(scale)
            tol = (2.0 ** -8 + 2 * (D + 2) * 2.0 ** -24 * reach + 2.0 ** -20 * (1 + n / 4096)) * mag \
                + 2.0 ** -8 * (1 + 2.0 ** -7) * ref.abs() + 1e-30
            err = (by_head(got[b, :k + 1].double()) - ref).abs()
            assert bool((err <= tol).all()), (b, float((err / tol).max()))
            assert bool((got[b, k + 1:] == fill).all())
        assert int(self.status) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 128])
@pytest.mark.parametrize("K,Hq,Hkv", [(0, 4, 4), (5, 8, 2), (8, 8, 1), (2, 3, 1), (32, 4, 2)])
def test_shapes(D, page, K, Hq, Hkv):
    """Two groups and loners, empty slots in front of and inside groups, contexts
    that end at the shared tokens, groups that share no whole tile."""
    _log(f"[shared] D={D} page={page} K={K} Hq={Hq} Hkv={Hkv}")
    groups = [0, 1, 0, -1, 0, 1, 1, 2, 2, 7, 0]
    ctx = np.array([-1, 300, 400, 77, 391, 257, 513, 40, 31, 5, 384])
    rng = np.random.default_rng(K)
    budgets = rng.integers(0, K + 1, ctx.size)
    c = Case(groups, [384, 256, 40, 500], ctx, budgets, K, Hq, Hkv, D, page, seed=D + K)
    c.check(c.run())


@pytest.mark.parametrize("lens", [0, 31, 32, 33, 64, 95, 96, 2**31 - 1, -5, -2**31])
def test_lengths_of_the_prefix(lens):
    """What is shared is cut to whole tiles and to the shortest context."""
    c = Case([0] * 5, [128], np.array([128, 140, 131, 128, 200]), np.array([2, 0, 1, 2, 2]), 2, 4, 2, 128, 32, seed=3)
    c.lens = np.array([lens])
    if lens > 128:
        c.ctx = np.array([128, 140, 131, 128, 200])
    c.check(c.run())


@pytest.mark.parametrize("B,G,K,Hq,Hkv,D,prefix,tail", [
    (70, 1, 3, 16, 2, 128, 3000, 300),      # several row blocks, parts of the prefix
    (3, 1, 0, 8, 8, 128, 40000, 90),        # few rows, many parts
    (2, 1, 0, 4, 1, 64, 60000, 50),         # eight rows, hundreds of parts each
    (2, 1, 1, 2, 1, 256, 20000, 9000),
    (40, 9, 1, 12, 4, 64, 1500, 700),       # groups of unlike sizes
    (33, 2, 8, 8, 1, 256, 2500, 1100),
    (300, 1, 0, 8, 8, 64, 700, 40),
    (6, 3, 8, 64, 1, 128, 5000, 3000),      # long tails, split themselves
])
def test_every_way_the_work_is_cut(B, G, K, Hq, Hkv, D, prefix, tail):
    _log(f"[shared] B={B} G={G} K={K} Hq={Hq} Hkv={Hkv} D={D} prefix={prefix} tail={tail}")
    rng = np.random.default_rng(B)
    lens = rng.integers(prefix // 2, prefix + 1, G)
    lens = lens // 64 * 64 + lens % 32          # whole pages are in common, and less than a tile more
    groups = np.minimum(rng.integers(0, G + 1, B), rng.integers(0, G + 1, B)) if G > 1 else np.zeros(B, int)
    ctx = lens[np.minimum(groups, G - 1)] + rng.integers(0, tail, B)
    if B > 3:
        ctx[B // 2] = -1
    c = Case(groups, lens, ctx, rng.integers(0, K + 1, B), K, Hq, Hkv, D, 64, seed=B + K)
    got = c.run()
    c.check(got)
    assert torch.equal(c.run(), got)


def test_more_requests_than_a_round_of_the_plan():
    """2,100 requests in interleaved groups: sections of the plan of several rounds."""
    rng = np.random.default_rng(6)
    B, G = 2100, 40
    groups = rng.integers(-1, G, B)
    ctx = np.where(rng.random(B) < 0.1, -1, 64 + rng.integers(0, 30, B))
    c = Case(groups, np.full(G, 64), ctx, rng.integers(0, 2, B), 1, 2, 1, 64, 32, seed=9)
    c.check(c.run())


@pytest.mark.parametrize("used,longest", [(1500, 3000), (150, 400)])
def test_own_tokens_of_many_requests_are_cut(used, longest):
    """1,500 requests under tables of more than 2,048 tokens: all in use, a few of them long (on a
    line), and a tenth in use, much alike (equal parts)."""
    rng = np.random.default_rng(used)
    B, G = 1500, 12
    ctx = np.full(B, -1)
    some = np.sort(rng.permutation(B)[:used])
    ctx[some] = 64 + rng.integers(0, 60 if used == B else longest, used)
    ctx[some[::200]] = 64 + longest
    c = Case(rng.integers(-1, G, B), np.full(G, 64), ctx, rng.integers(0, 2, B), 1, 2, 1, 64, 32, seed=4)
    c.table = np.pad(c.table, ((0, 0), (0, 80)), constant_values=-1)
    c.check(c.run())


def test_more_rows_than_a_row_of_the_joins_grid():
    rng = np.random.default_rng(3)
    B = 1024
    c = Case(np.zeros(B, int), [64], 64 + rng.integers(0, 20, B), np.full(B, 32), 32, 16, 2, 128, 32, seed=6)
    c.check(c.run())


def test_the_most_groups():
    B = 2 * sb.SV_MAX_GROUPS
    groups = np.arange(B) % sb.SV_MAX_GROUPS
    c = Case(groups, np.full(sb.SV_MAX_GROUPS, 96), 96 + np.arange(B) % 7, np.zeros(B, int), 0, 2, 1, 64, 32, seed=2)
    c.check(c.run())
    with pytest.raises(ValueError):
        c.cache.attend_shared(c.q, _i32(c.table), _i32(c.ctx), _i32(c.groups), _i32(np.zeros(sb.SV_MAX_GROUPS + 1)))


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_scales_and_sharp_softmax(scale):
    c = Case([0, 0, 0], [256], np.array([260, 300, 256]), np.array([4, 0, 2]), 4, 8, 2, 128, 64, seed=3)
    c.check(c.run(scale=scale), scale=scale)


def test_no_groups_is_the_attention_itself():
    c = Case([-1, 0, -3], [200], np.array([300, 260, 40]), np.array([4, 0, 2]), 4, 8, 2, 128, 64, seed=4)
    want = c.plain()
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    got = c.cache.attend_shared(c.q, _i32(c.table), _i32(c.ctx), _i32(c.groups), none, _i32(c.budgets))
    assert torch.equal(got, want)
    # A group of one shares nothing either.
    c.check(c.run())


def test_rows_behind_the_budget_and_empty_slots_keep_their_values():
    c = Case([0, 0, 0, 0], [128], np.array([140, -1, 129, -2**31]), np.array([2, 5, 0, 3]), 5, 4, 2, 64, 32, seed=2)
    out = torch.full((4, 6, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    got = c.run(out=out)
    assert got is out
    c.check(got, fill=3.0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_nan_token_reaches_the_rows_that_see_it_and_no_others(D):
    """In the prefix: all rows of its group; behind it: those rows of the one request."""
    def make():
        return Case([0, 1, 0, 1], [192, 64], np.array([200, 90, 230, 70]), np.array([3] * 4), 3, 4, 2, D, 32, seed=5)

    clean = make().run().double().cpu().numpy()
    assert not np.isnan(clean).any()
    _, _, ks, vs = lb.tile_addresses(D)
    g = D // 32 - 1
    for b, where in ((0, 0), (2, 191), (0, 195), (3, 71), (1, 33)):
        for side in ("value", "key"):
            c = make()
            c.cache.pool[int(c.table[b, where // 32]), 1, 0, int((vs if side == "value" else ks)[where % 32, g])] = 255
            got = c.run().double().cpu().numpy()
            want = clean.copy()
            for r in range(4):
                if c.table[r, where // 32] != c.table[b, where // 32]:
                    continue
                rows = [t for t in range(4) if c.ctx[r] + t >= where]
                for t in rows:
                    if side == "value":
                        want[r, t, 2:, 32 * g:] = np.nan
                    else:
                        want[r, t, 2:] = np.nan
            assert np.array_equal(np.isnan(got), np.isnan(want)), (D, b, where, side)
            assert np.array_equal(got, want, equal_nan=True)


def test_bad_pages_budgets_and_lengths_are_flagged():
    c = Case([0, 0, 1, 1], [128, 128], np.array([140, 150, 130, 129]), np.array([3, 1, 2, 0]), 3, 4, 2, 64, 32, seed=6)
    good = c.run()
    c.check(good)
    keep = c.table.copy()
    for bad in (-1, c.pages, 2**31 - 1):
        c.table = keep.copy()
        c.table[0, 1] = bad                   # the first group's prefix
        got = c.run()
        assert int(c.status) == sb.SV_FLAG_BAD_PAGE and torch.equal(got[2:], good[2:])
        c.table = keep.copy()
        c.table[1, 1] = bad                   # read through the first request's row only
        assert torch.equal(c.run(), good) and int(c.status) == 0
    c.table = keep
    c.ctx[0] = 32 * keep.shape[1] - 1
    got = c.run()
    assert int(c.status) == sb.SV_FLAG_BAD_LENGTH and not got[0].any()
    c.ctx[0], c.budgets[1] = 140, 99
    c.run()
    assert int(c.status) == sb.SV_FLAG_BAD_BUDGET


def test_queries_as_a_slice_of_a_fused_projection():
    c = Case([0, 0, 0], [64], np.array([70, 65, 129]), np.array([4, 1, 3]), 4, 8, 2, 128, 64, seed=4)
    want = c.run()
    fused = torch.full((3, 5, 12 * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    fused[..., :8 * 128] = c.q.flatten(2)
    for b in range(3):
        fused[b, c.budgets[b] + 1:] = float("nan")      # never read
    c.q = fused[..., :8 * 128].unflatten(-1, (8, 128))
    assert torch.equal(c.run(), want)


def test_a_pool_past_32_bit_offsets():
    Hkv, D, page = 8, 128, 128
    pages = (1 << 32) // (Hkv * (page // 32) * 34 * D) + 16
    big, small = BlockCache(DEV, pages, Hkv, D, page), BlockCache(DEV, 4, Hkv, D, page)
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v = (torch.randn(1, 300, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(2, 3, 16, D, generator=g, device=DEV).bfloat16()
    got = []
    for c, row in ((big, [pages - 1, 3, pages - 2]), (small, [0, 1, 2])):
        c.write(k, v, _i32([row]), _i32([0]))
        got.append(c.attend_shared(q, _i32([row, row]), _i32([297, 290]), _i32([0, 0]), _i32([290])))
    assert torch.equal(got[0], got[1]) and bool(got[0].any())


def test_replayed_on_another_stream_and_two_graphs():
    c = Case([0, 0, 1, 1, 0], [2048, 640], np.array([2100, 2600, 700, 640, -1]), np.array([4, 2, 0, 1, 3]), 4, 8, 2, 128,
             64, seed=8)
    want = c.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    args = c.q, _i32(c.table), _i32(c.ctx), _i32(c.groups), _i32(c.lens), _i32(c.budgets)
    outs, graphs = [torch.zeros_like(want) for _ in range(2)], []
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.cache.attend_shared(*args, out=out)
        graphs.append(graph)
    for _ in range(4):
        for graph, out in zip(graphs, outs):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert torch.equal(c.run(), want)


def test_bad_arguments_are_refused():
    c = Case([0, 0], [64], np.array([70, 65]), np.array([1, 1]), 1, 4, 2, 64, 32, seed=1)
    t, x, g, n, k = (_i32(v) for v in (c.table, c.ctx, c.groups, c.lens, c.budgets))
    good = dict(queries=c.q, page_table=t, ctx_lens=x, groups=g, shared_lens=n, budgets=k)
    for bad in (dict(queries=c.q.float()), dict(groups=g[:1]), dict(groups=g.long()), dict(shared_lens=n.cpu()),
                dict(shared_lens=n[None]), dict(ctx_lens=x.cpu()), dict(scale=float("nan")), dict(budgets=k[:1])):
        with pytest.raises((ValueError, RuntimeError)):      # the binding's checks, the library's
            c.cache.attend_shared(**{**good, **bad})
    empty = c.cache.attend_shared(c.q[:0], t[:0], x[:0], g[:0], n)
    assert empty.shape == (0, 2, 4, 64)
