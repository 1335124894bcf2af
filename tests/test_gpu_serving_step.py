"""The operators of a serving step in a run, as a program uses them: pages planned
from the lengths, projections normalised, rotated and written by slot, attention
behind the shared prefix or under a window with sinks, lengths moved on by what was
accepted. Every step's outputs against fp64 on the CPU over the keys and values
that the requests were given, in the cache's 4 bits.

Tolerance: the attention's own (see test_gpu_sinks.py)."""
import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, PageTables, schedule_budgets
from oracle import lowbit as lb, serving as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _bound(ref, mag, reach, D, n):
    rel = 2.0 ** -8 + 2 * (D + 2) * 2.0 ** -24 * reach[..., None] + 2.0 ** -20 * (1 + n / 4096)
    return rel * mag + 2.0 ** -8 * (1 + 2.0 ** -7) * np.abs(ref) + 1e-30


class Server:
    """A layer's cache over page tables, and what every request was given (on the CPU)."""

    def __init__(self, B, pages, page, width, Hq, Hkv, D, window, sinks, seed):
        self.__dict__.update(B=B, page=page, Hq=Hq, Hkv=Hkv, D=D, window=window, sinks=sinks)
        self.tables = PageTables(DEV, B, width, pages, page)
        self.cache = BlockCache(DEV, pages, Hkv, D, page)
        self.cache.pool.random_(0, 256, generator=torch.Generator(device=DEV).manual_seed(seed))
        self.rng = np.random.default_rng(seed)
        self.ctx = np.full(B, -1)
        self.given = [[] for _ in range(B)]             # (key, value) of every position, in 4 bits
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.freq = torch.tensor(1e4 ** (-np.arange(0, D, 2) / D), dtype=torch.float32, device=DEV)
        self.norm = torch.tensor(np.exp(0.3 * self.rng.normal(size=D)), dtype=torch.float32, device=DEV)

    def step(self, T, budgets, parents=None, prefix=None, groups=None, shared=None, check=True):
        B, Hq, Hkv, D = self.B, self.Hq, self.Hkv, self.D
        ctx, k = _i32(self.ctx), _i32(budgets)
        starts, slots, positions = self.tables.plan(
            ctx, k, T, self.window, self.sinks, None if parents is None else _i32(parents),
            None if prefix is None else _i32(prefix), status=self.status)
        fused = torch.tensor(self.rng.normal(size=(B, T, Hq + 2 * Hkv, D))).bfloat16().to(DEV)
        q, key, value = fused.split([Hq, Hkv, Hkv], 2)
        keys = torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=DEV)
        q = self.cache.write_rotated(q, key, value, slots, positions, self.freq, self.norm, self.norm, out_keys=keys,
                                     status=self.status)
        if groups is not None:
            out = self.cache.attend_shared(q, self.tables.table, starts, _i32(groups), _i32(shared), k, status=self.status)
        elif T <= 33:
            out = self.cache.attend(q, self.tables.table, starts, k, window=self.window, sinks=self.sinks, status=self.status)
        else:
            check = False                               # a prompt's chunk: its rows are not looked at here
        assert int(self.status) == 0
        assert np.array_equal(starts.cpu().numpy(), self.ctx)
        for b in range(B):
            if self.ctx[b] < 0:
                self.given[b] = []
                continue
            if parents is not None and parents[b] >= 0:
                self.given[b] = self.given[parents[b]][:prefix[b]]
            n = budgets[b] + 1
            rounded = [lb.cache_values(*lb.quantise_cache(x[b, :n].double().cpu().numpy())) for x in (keys, value)]
            self.given[b] = self.given[b][:self.ctx[b]] + list(zip(*rounded))
            assert len(self.given[b]) == self.ctx[b] + n
            if not check:
                continue
            all_k, all_v = (np.stack([p[i] for p in self.given[b]]) for i in (0, 1))
            ref, mag, reach = sv.attend(q[b, :n].double().cpu().numpy(), all_k, all_v, int(self.ctx[b]), D ** -0.5,
                                        self.window, self.sinks)
            err = np.abs(out[b, :n].double().cpu().numpy() - ref)
            tol = _bound(ref, mag, reach, D, len(self.given[b]))
            assert np.all(err <= tol), (b, float((err / tol).max()))
            assert not out[b, n:].any()


@pytest.mark.parametrize("D", [64, 128])
def test_requests_that_fork_from_a_prompt(D):
    s = Server(6, 60, 32, 16, 4, 2, D, 0, 0, seed=D)
    rng = np.random.default_rng(D)
    s.ctx[0] = 0
    s.step(170, [169, 0, 0, 0, 0, 0])
    # Four requests join behind the first 160 of its tokens, one starts by itself.
    s.ctx[:] = [170, 160, 160, 160, 160, 0]
    groups = [0, 0, 0, 0, 0, -1]
    parents, prefix = [-1, 0, 0, 0, 0, -1], [0, 160, 160, 167, 191, 0]
    budgets = rng.integers(0, 6, 6)
    s.step(6, budgets, parents, prefix, groups, [160])
    for i in range(4):
        s.ctx = np.where(s.ctx < 0, -1, s.ctx + np.minimum(budgets, rng.integers(0, 6, 6)) + 1)
        if i == 2:
            s.ctx[[0, 3]] = -1                          # the prompt's own request ends before the others
        budgets = schedule_budgets(torch.rand(6, 5, device=DEV), 14).cpu().numpy()
        s.step(6, budgets, groups=groups, shared=[160])
    s.ctx[:] = -1
    s.step(1, [0] * 6)
    assert not s.tables.refs.any() and bool((s.tables.table == -1).all())


def test_windows_with_sinks_give_their_pages_back():
    s = Server(4, 26, 32, 40, 4, 1, 64, 70, 33, seed=3)
    rng = np.random.default_rng(3)
    s.ctx[:] = [0, 0, -1, 0]
    s.step(100, [99, 40, 0, 80])
    s.ctx[:] = [100, 41, 0, 81]
    budgets = np.array([5, 0, 3, 2])
    for _ in range(40):
        s.step(8, budgets)
        s.ctx = s.ctx + np.minimum(budgets, rng.integers(0, 8, 4)) + 1
        budgets = rng.integers(0, 8, 4)
    # Two pages of sinks, and at most four of the window and the block each.
    assert s.ctx.max() > 200 and int((s.tables.refs > 0).sum()) <= 4 * 6


def test_a_step_in_a_graph():
    """Planned, written and attended in one captured graph, replayed as lengths grow."""
    B, T, D, Hq, Hkv, page = 3, 4, 128, 4, 2, 32
    g = torch.Generator(device=DEV).manual_seed(5)
    tables, cache = PageTables(DEV, B, 12, 30, page), BlockCache(DEV, 30, Hkv, D, page)
    ctx, budgets = _i32([0, 0, 0]), _i32([3, 1, 2])
    q, k, v = (torch.randn(B, T, h, D, generator=g, device=DEV).bfloat16() for h in (Hq, Hkv, Hkv))
    freq = torch.tensor(1e4 ** (-np.arange(0, D, 2) / D), dtype=torch.float32, device=DEV)
    groups, shared = _i32([0, 0, 0]), _i32([0])

    def step(tables, cache):
        starts, slots, positions = tables.plan(ctx, budgets, T)
        return cache.attend_shared(cache.write_rotated(q, k, v, slots, positions, freq), tables.table, starts, groups,
                                   shared, budgets)

    other = PageTables(DEV, B, 12, 30, page), BlockCache(DEV, 30, Hkv, D, page)
    step(tables, cache), step(*other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(tables, cache)
    for i in range(12):
        ctx += budgets + 1
        q.normal_(generator=g)
        k.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        want = step(*other)
        assert torch.equal(out, want) and torch.equal(tables.table, other[0].table)
        assert torch.equal(cache.pool, other[1].pool)
