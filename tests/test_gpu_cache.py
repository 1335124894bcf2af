"""The paged 4-bit cache on the GPU against the fp64 oracle. Codes are a
function of the input alone and every stored value is exact in both types, so
everything is compared for equality: written bytes with the oracle's, bytes
that no token covers with what was there before, values read back with the
oracle's values."""
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


def make_table(rng, counts, page, width, pages):
    """Distinct random pages for requests of counts[b] tokens; -1 elsewhere."""
    order = rng.permutation(pages)
    table, at = np.full((len(counts), width), -1, np.int64), 0
    for b, n in enumerate(counts):
        need = -(-max(int(n), 0) // page)
        table[b, :need] = order[at:at + need]
        at += need
    return table


def _values(rng, shape):
    """Gains over many octaves, so that many scales occur."""
    return rng.normal(size=shape) * np.exp2(rng.integers(-20, 20, shape[:-1] + (1,)).astype(float))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,heads,page,T", [(64, 3, 32, 1), (64, 1, 64, 37), (128, 2, 64, 6),
                                            (128, 1, 32, 70), (256, 2, 128, 9), (256, 1, 32, 33)])
def test_write_stores_the_oracles_bytes_and_no_others(D, heads, page, T, dtype):
    _log(f"[cache write] D={D} heads={heads} page={page} T={T} {dtype}")
    rng = np.random.default_rng(D + T)
    B = 5
    ctx = np.array([0, 31, 17, -1, 64])
    budgets = rng.integers(0, T, B)
    budgets[1] = T - 1
    pages, width = 40, -(-(64 + T) // page) + 1
    table = make_table(rng, np.where(ctx < 0, 0, ctx + budgets + 1), page, width, pages)
    before = rng.integers(0, 256, (pages, heads, page // 32, 34 * D)).astype(np.uint8)
    k, v = (torch.tensor(_values(rng, (B, T, heads, D))).to(dtype) for _ in range(2))
    cache = BlockCache(DEV, pages, heads, D, page, pool=torch.tensor(before).to(DEV))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache.write(k.to(DEV), v.to(DEV), _i32(table), _i32(ctx), _i32(budgets), status=status)
    want = before.copy()
    for b in range(B):
        n = budgets[b] + 1
        if ctx[b] >= 0:
            lb.write(want, table[b], int(ctx[b]), k[b, :n].double().numpy(),
                     v[b, :n].double().numpy(), page)
    got = cache.pool.cpu().numpy()
    assert np.array_equal(got, want)
    assert int(status) == 0
    # Read back: written tokens, and rows behind them left as they were.
    for out_type in (torch.float32, torch.bfloat16):
        out = tuple(torch.full((B, T, heads, D), 77.0, dtype=out_type, device=DEV) for _ in range(2))
        cache.read(_i32(table), _i32(ctx), _i32(budgets + 1), T, out=out, status=status)
        for b in range(B):
            n = 0 if ctx[b] < 0 else budgets[b] + 1
            ref = lb.read(want, table[b], int(ctx[b]), int(n), D, page) if n else (0, 0)
            for got_side, ref_side in zip(out, ref):
                g = got_side[b].double().cpu().numpy()
                assert np.array_equal(g[:n], ref_side) if n else True
                assert np.all(g[n:] == 77.0)
    assert int(status) == 0


def test_borders_specials_and_saturation():
    """Every rounding border of e2m1 at many scales, zeros of both signs,
    denormals, the largest magnitudes, and groups with a NaN or an infinity."""
    D, page = 128, 32
    rows = []
    borders = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -0.0])
    for e in (-120, -66, -64, -63, -1, 0, 5, 100, 125):
        g = np.concatenate([borders, -borders]) * np.exp2(float(e))
        up = np.nextafter(g.astype(np.float32), np.float32(np.inf)).astype(float)
        dn = np.nextafter(g.astype(np.float32), np.float32(-np.inf)).astype(float)
        rows.append(np.concatenate([g, up, dn, np.zeros(32)]))
    big = np.full(128, 3.4e38)
    big[::2] = -2.6e38
    rows.append(big)
    for bad in (np.nan, np.inf, -np.inf):
        r = np.linspace(-3, 3, 128)
        r[40] = bad
        rows.append(r)
    x = torch.tensor(np.array(rows), dtype=torch.float32)
    n = x.shape[0]
    k = x[None, :, None, :].contiguous().to(DEV)
    cache = BlockCache(DEV, 2, 1, D, page)
    table, zero = _i32([[1, 0]]), _i32([0])
    cache.write(k, -k, table, zero)
    gk, gv = cache.read(table, None, _i32([n]), n, dtype=torch.float32)
    codes, scale = lb.quantise_cache(x.double().numpy())
    ref = lb.cache_values(codes, scale)
    assert np.isnan(ref[-1, 32:64]).all() and np.isfinite(ref[:-3]).all()
    assert np.array_equal(gk[0, :, 0].double().cpu().numpy(), ref, equal_nan=True)
    assert np.array_equal(gv[0, :, 0].double().cpu().numpy(), -ref, equal_nan=True)
    gb, _ = cache.read(table, None, _i32([n]), n, dtype=torch.bfloat16)
    assert np.array_equal(gb[0, :, 0].double().cpu().numpy(), ref, equal_nan=True)


def test_slices_of_a_fused_projection():
    """Keys and values as slices of [B, T, (Hq + 2 Hkv) D] rows, on the next
    page of an existing context; the same bytes as contiguous copies give."""
    B, T, heads, D, page = 3, 6, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(4)
    fused = torch.randn(B, T, 8 * D, generator=g, device=DEV).bfloat16()
    k = fused[..., 4 * D:6 * D].unflatten(-1, (heads, D))
    v = fused[..., 6 * D:].unflatten(-1, (heads, D))
    table = torch.arange(B * 3, dtype=torch.int32, device=DEV).view(B, 3).contiguous()
    ctx = _i32([61, 0, 127])
    a, b = (BlockCache(DEV, 9, heads, D, page) for _ in range(2))
    a.write(k, v, table, ctx)
    b.write(k.contiguous(), v.contiguous(), table, ctx)
    assert torch.equal(a.pool, b.pool) and a.pool.any()
    one = BlockCache(DEV, 9, heads, D, page)            # a single token, odd batch stride
    one.write(k[:, 2:3], v[:, 2:3], table, ctx)
    two = BlockCache(DEV, 9, heads, D, page)
    two.write(k[:, 2:3].contiguous(), v[:, 2:3].contiguous(), table, ctx)
    assert torch.equal(one.pool, two.pool) and one.pool.any()


def test_rejected_tokens_are_undone_by_the_lengths():
    """A block of which the verify kept j tokens, then the next block over the
    rejected ones: the cache is what writing the kept tokens alone gives."""
    heads, D, page, T = 2, 64, 32, 6
    g = torch.Generator(device=DEV).manual_seed(9)
    k1, v1, k2, v2 = (torch.randn(1, T, heads, D, generator=g, device=DEV).bfloat16() for _ in range(4))
    table = _i32([[2, 0, 1]])
    for kept in range(T + 1):
        a, b = (BlockCache(DEV, 3, heads, D, page) for _ in range(2))
        for c in (a, b):
            first = (k1, v1) if c is a else (k1[:, :max(kept, 1)].contiguous(), v1[:, :max(kept, 1)].contiguous())
            if c is a or kept:
                c.write(*first, table, _i32([30]))
            c.write(k2, v2, table, _i32([30 + kept]))
        n = 30 + kept + T
        ra, rb = (c.read(table, None, _i32([n]), n) for c in (a, b))
        assert torch.equal(ra[0][:, 30:], rb[0][:, 30:]) and torch.equal(ra[1][:, 30:], rb[1][:, 30:])


def test_bad_budgets_lengths_and_pages_are_flagged_and_skipped():
    heads, D, page, T = 1, 64, 32, 4
    rng = np.random.default_rng(0)
    before = rng.integers(0, 256, (4, heads, 1, 34 * D)).astype(np.uint8)
    k = torch.tensor(rng.normal(size=(1, T, heads, D)), dtype=torch.float32)

    def call(row, ctx, budget):
        cache = BlockCache(DEV, 4, heads, D, page, pool=torch.tensor(before).to(DEV))
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        cache.write(k.to(DEV), k.to(DEV), _i32([row]), _i32([ctx]), _i32([budget]), status=status)
        return cache.pool.cpu().numpy(), int(status)

    def ref(row, ctx, lo, n):
        want = before.copy()
        x = k[0, lo:lo + n].double().numpy()
        lb.write(want, row, ctx + lo, x, x, page)
        return want

    for budget, n in ((99, 4), (-5, 1)):
        got, flags = call([2, 1], 3, budget)
        assert flags == sb.SV_FLAG_BAD_BUDGET and np.array_equal(got, ref([2, 1], 3, 0, n))
    got, flags = call([2, 1], 61, 3)                       # one token past the table's row
    assert flags == sb.SV_FLAG_BAD_LENGTH and np.array_equal(got, before)
    got, flags = call([2, 1], 2**31 - 2, 3)                # no wrap-around
    assert flags == sb.SV_FLAG_BAD_LENGTH and np.array_equal(got, before)
    for bad in (-1, 4, 2**31 - 1, -2**31):                 # second page outside the pool
        got, flags = call([2, bad], 30, 3)
        assert flags == sb.SV_FLAG_BAD_PAGE and np.array_equal(got, ref([2, -1], 30, 0, 2))
    # Reads: too many tokens, past the row, a bad page; what is skipped keeps its values.
    cache = BlockCache(DEV, 4, heads, D, page, pool=torch.tensor(before).to(DEV))
    for row, start, n, flag, good in (([2, 1], 0, 5, sb.SV_FLAG_BAD_LENGTH, 0),
                                      ([2, 1], 62, 4, sb.SV_FLAG_BAD_LENGTH, 0),
                                      ([2, 9], 30, 4, sb.SV_FLAG_BAD_PAGE, 2),
                                      ([2, 1], -1, 4, 0, 0), ([2, 1], 0, 0, 0, 0),
                                      ([2, 1], 0, -3, 0, 0)):
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = tuple(torch.full((1, 4, heads, D), 5.0, device=DEV) for _ in range(2))
        cache.read(_i32([row]), _i32([start]), _i32([n]), 4, out=out, status=status)
        assert int(status) == flag
        want = np.full((4, heads, D), 5.0)
        if good:
            want[:good] = lb.read(before, np.array(row), start, good, D, page)[0]
        assert np.array_equal(out[0][0].cpu().numpy(), want, equal_nan=True)


def test_a_pool_past_32_bit_offsets():
    """Pages near both ends of a pool of more than 4 GiB."""
    heads, D, page = 8, 256, 128
    per = heads * (page // 32) * 34 * D
    pages = (1 << 32) // per + 40
    pool = torch.empty((pages, heads, page // 32, 34 * D), dtype=torch.uint8, device=DEV)
    cache = BlockCache(DEV, pages, heads, D, page, pool=pool)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(2, 200, heads, D, generator=g, device=DEV) for _ in range(2))
    table = _i32([[pages - 1, 1], [0, pages - 2]])
    cache.write(k, v, table, _i32([0, 40]))
    got = cache.read(table, _i32([0, 40]), _i32([200, 200]), 200, dtype=torch.float32)
    for x, y in zip((k, v), got):
        ref = lb.cache_values(*lb.quantise_cache(x[:, ::37].double().cpu().numpy()))
        assert np.array_equal(y[:, ::37].double().cpu().numpy(), ref)


def test_python_refusals():
    cache = BlockCache(DEV, 4, 2, 64, 32)
    k = torch.zeros(1, 2, 2, 64, device=DEV)
    table, one = _i32([[0]]), _i32([0])
    for bad in (k.half(), k[..., :32], k.transpose(1, 2), k.cpu()):
        with pytest.raises(ValueError):
            cache.write(bad, bad, table, one)
    with pytest.raises(ValueError):
        cache.write(k, k.bfloat16(), table, one)
    for tab in (table.long(), table[0], _i32([[0], [0]])):
        with pytest.raises(ValueError):
            cache.write(k, k, tab, one)
    with pytest.raises(ValueError):
        cache.read(table, one, one, 2, dtype=torch.float16)
    for geometry in ((0, 2, 64, 32), (4, 2, 80, 32), (4, 2, 64, 48)):
        with pytest.raises(ValueError):
            BlockCache(DEV, *geometry)
    with pytest.raises(ValueError):
        BlockCache("cpu", 4, 2, 64, 32)


def test_two_streams_and_a_replayed_graph():
    """Writes of two halves of a batch on two streams at once, and a write and a
    read captured together and replayed with new tokens and lengths between
    eager calls of another cache."""
    B, T, heads, D, page = 6, 40, 2, 128, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    k, v = (torch.randn(B, T, heads, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(12, generator=g, device=DEV).int().view(B, 2)
    ctx, budgets = _i32([0, 31, 5, -1, 60, 88]), _i32([39, 0, 20, 3, 39, 39])
    a, b = (BlockCache(DEV, 12, heads, D, page) for _ in range(2))
    a.write(k, v, table, ctx, budgets)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        part = slice(3 * i, 3 * i + 3)
        b.write(k[part], v[part], table[part], ctx[part], budgets[part], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.pool, b.pool)
    out = tuple(torch.zeros_like(k) for _ in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.write(k, v, table, ctx, budgets)
        b.read(table, ctx, budgets, T, out=out)
    for i in range(4):
        k.mul_(-1.5)
        v.add_(0.25)
        budgets.copy_(_i32([30 + i, i, 39 - i, 3, 39, 7]))
        for x in out:
            x.zero_()
        a.write(k, v, table, ctx, budgets)
        want = a.read(table, ctx, budgets, T)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.pool, b.pool)
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_the_largest_batch():
    B = 16384
    g = torch.Generator(device=DEV).manual_seed(10)
    k, v = (torch.randn(B, 1, 1, 64, generator=g, device=DEV) for _ in range(2))
    table = torch.randperm(B, generator=g, device=DEV).int()[:, None]
    ctx = torch.randint(0, 32, (B,), generator=g, device=DEV, dtype=torch.int32)
    cache = BlockCache(DEV, B, 1, 64, 32)
    cache.write(k, v, table, ctx)
    got = cache.read(table, ctx, torch.ones_like(ctx), 1, dtype=torch.float32)
    for x, y in zip((k, v), got):
        ref = lb.cache_values(*lb.quantise_cache(x.double().cpu().numpy()))
        assert np.array_equal(y.double().cpu().numpy(), ref)
    # Batches, tokens and lists of none.
    before = cache.pool.clone()
    cache.write(k[:0], v[:0], table[:0], ctx[:0])
    cache.write(k[:, :0], v[:, :0], table, ctx)
    assert cache.read(table[:0], None, ctx[:0], 5)[0].shape == (0, 5, 1, 64)
    assert cache.read(table, None, ctx, 0)[0].shape == (B, 0, 1, 64)
    assert torch.equal(cache.pool, before)
