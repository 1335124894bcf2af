"""Edges of the low-bit operators on the GPU: bytes that no row sees, NaN
groups and bad pages in every way the attention's work is cut, three row tiles,
NaN blocks in the head's largest tiles, and the calls' limits."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, SpecVerify, binding as sb, head_logits
from draft_verify_sampling_spec_amd import head_quantize
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


# ---- three row tiles, and NaN groups and bad pages in every cut of the work -----------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("K,Hq,Hkv,ctx", [
    (8, 8, 2, [0, 1, 31, 32, 33, 95, -1, 300]),      # 36 rows
    (10, 8, 2, [5, 64, 511]),                        # 44 rows
    (15, 3, 1, [17, 800, 96]),                       # 48 rows
])
def test_three_row_tiles(D, K, Hq, Hkv, ctx):
    """Blocks of up to 48 rows a head, short contexts; ragged budgets leave one,
    two or three row tiles."""
    _log(f"[attend] three row tiles D={D} K={K} Hq={Hq} Hkv={Hkv}")
    rng = np.random.default_rng(K)
    budgets = rng.integers(0, K + 1, len(ctx))
    budgets[-1], budgets[0], budgets[1] = K, 0, K // 2
    c = ta.Case(len(ctx), K, Hq, Hkv, D, 32, np.array(ctx), budgets, seed=K)
    c.check(c.run())


@pytest.mark.parametrize("B,K,Hq,Hkv,D,lo,hi,window", [
    (64, 8, 32, 8, 128, 300, 9000, 0),         # shares of a line
    (24, 8, 16, 4, 64, 300, 12000, 0),
    (2, 8, 8, 2, 128, 30000, 60000, 0),        # few units, many parts each
    (1, 10, 8, 2, 64, 40000, 40000, 0),
    (16, 8, 32, 8, 128, 4000, 4100, 0),        # nearly equal units, few parts each
    (16, 8, 32, 8, 128, 5000, 9000, 3000),
])
def test_three_row_tiles_split_over_workgroups(B, K, Hq, Hkv, D, lo, hi, window):
    ta.test_every_way_the_work_is_cut(B, K, Hq, Hkv, D, lo, hi, window)


# Shapes of one to four row tiles: (B, K, Hq, Hkv, D, contexts from .. to, window).
CUTS = [
    (6, 8, 8, 2, 128, 40, 700, 0),             # direct, three row tiles
    (6, 8, 16, 2, 128, 40, 700, 0),            # direct, four, two row blocks
    (6, 4, 16, 2, 64, 40, 700, 90),            # direct, three, a window
    (5, 5, 8, 2, 256, 40, 700, 0),             # direct, two of 256 channels
    (2, 0, 8, 2, 128, 9000, 20000, 0),         # many parts, one row tile
    (2, 8, 8, 2, 128, 9000, 20000, 0),         # three
    (2, 7, 16, 2, 128, 9000, 20000, 0),        # four
    (2, 7, 16, 2, 64, 9000, 20000, 5000),
    (2, 5, 8, 2, 256, 9000, 20000, 0),
    (64, 8, 32, 8, 128, 300, 9000, 0),         # a line
    (24, 7, 64, 8, 64, 300, 9000, 0),
]


class Big:
    """A batch made on the GPU: random codes under sane scales."""

    def __init__(self, B, K, Hq, Hkv, D, lo, hi, window, page=64):
        g = torch.Generator(device=DEV).manual_seed(B + K + D)
        self.ctx = torch.randint(lo, hi + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        self.ctx[0], self.ctx[-1] = hi, lo
        self.budgets = torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
        self.budgets[0] = K
        need = (self.ctx + self.budgets + page) // page
        first = torch.cumsum(need, 0) - need
        width, pages = int(need.max()), int(need.sum())
        col = torch.arange(width, device=DEV)
        order = torch.randperm(pages, generator=g, device=DEV)
        self.table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp_max(pages - 1)], -1).int()
        self.cache = BlockCache(DEV, pages, Hkv, D, page)
        self.cache.pool.random_(0, 256, generator=g)
        self.cache.pool[..., 32 * D:].random_(122, 129, generator=g)
        self.q = torch.randn(B, K + 1, Hq, D, generator=g, device=DEV).bfloat16()
        self.K, self.Hq, self.Hkv, self.D, self.window, self.page = K, Hq, Hkv, D, window, page
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self):
        return self.cache.attend(self.q, self.table, self.ctx, self.budgets, window=self.window,
                                 status=self.status)

    def sees(self, b, pos):
        """Which rows t of request b see a position."""
        row = int(self.ctx[b]) + torch.arange(self.K + 1, device=DEV)
        seen = (pos <= row) & (torch.arange(self.K + 1, device=DEV) <= self.budgets[b])
        return seen & (pos > row - self.window) if self.window else seen


@pytest.mark.parametrize("cut", CUTS)
def test_nan_tokens_in_every_cut(cut):
    """NaN groups of values and of keys of one kv head: in a tile that every row
    sees whole, in the block itself (seen by its later rows only), at a window's
    edge and in front of every window. They reach exactly the rows that see the
    token; every other output keeps its bits."""
    _log(f"[attend] NaN tokens {cut}")
    x = Big(*cut)
    clean = x.run()
    assert not clean.isnan().any()
    b, h, group = 0, x.Hkv - 1, x.Hq // x.Hkv
    hi = int(x.ctx[b])
    kc, vc, ks, vs = lb.tile_addresses(x.D)
    where = [hi - 200 - 32 * (hi // 900), hi + x.K // 2, hi]
    if x.window:
        where = [hi - x.window // 2, hi + x.K // 2, hi - x.window + 1 + x.K // 2, hi - x.window]
    for pos in where:
        for side, at in (("value", vs), ("key", ks)):
            grp = 1
            i = int(x.table[b, pos // x.page]), h, pos % x.page // 32, int(at[pos % 32, grp])
            kept = x.cache.pool[i].item()
            x.cache.pool[i] = 255
            got = x.run()
            x.cache.pool[i] = kept
            want = torch.zeros_like(clean, dtype=torch.bool)
            ch = slice(32 * grp, 32 * grp + 32) if side == "value" else slice(None)
            want[b, x.sees(b, pos), h * group:(h + 1) * group, ch] = True
            assert torch.equal(got.isnan(), want), (pos, side)
            assert torch.equal(torch.where(want, 0, got), torch.where(want, 0, clean)), (pos, side)
    assert torch.equal(x.run(), clean) and int(x.status) == 0


@pytest.mark.parametrize("cut", CUTS)
def test_bad_pages_in_every_cut(cut):
    """A page outside the pool is flagged; every other request keeps its bits.
    Where rows have a window, the pages before it may be anything."""
    _log(f"[attend] bad pages {cut}")
    x = Big(*cut)
    hi = int(x.ctx[0])
    if x.window:
        x.table[0, :(hi - x.window + 1) // x.page] = -7
    clean = x.run()
    assert int(x.status) == 0
    for col in {max(0, hi - x.window // 2) // x.page if x.window else 0, hi // x.page}:
        kept = int(x.table[0, col])
        for bad in (-1, x.cache.num_pages, 2**31 - 1):
            x.table[0, col] = bad
            x.status.zero_()
            got = x.run()
            assert int(x.status) == sb.SV_FLAG_BAD_PAGE
            assert torch.equal(got[1:], clean[1:])
        x.table[0, col] = kept
    x.status.zero_()
    assert torch.equal(x.run(), clean) and int(x.status) == 0


def test_rows_of_a_prompts_chunk_in_blocks():
    """More rows than a call takes: a chunk of 80 tokens over a prefix is written
    at once and attended in blocks of 33 rows, each from its own position."""
    Hq, Hkv, D, page, n = 6, 2, 128, 64, 80
    g = torch.Generator(device=DEV).manual_seed(6)
    cache = BlockCache(DEV, 12, Hkv, D, page)
    table = torch.randperm(12, generator=g, device=DEV)[:10].int().view(2, 5)
    ctx, budgets = _i32([37, 200]), _i32([n - 1, 50])
    prefix = torch.randn(2, 2, 200, Hkv, D, generator=g, device=DEV).bfloat16()
    cache.write(prefix[0], prefix[1], table, _i32([0, 0]), ctx - 1)
    k, v = (torch.randn(2, n, Hkv, D, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(2, n, Hq, D, generator=g, device=DEV).bfloat16()
    cache.write(k, v, table, ctx, budgets)
    out = torch.zeros_like(q)
    most = sb.SV_MAX_K + 1
    for at in range(0, n, most):
        rows = q[:, at:at + most].contiguous()
        left = budgets - at                                # a request whose rows have ended is skipped
        start = torch.where(left < 0, -1, ctx + at)
        out[:, at:at + most] = cache.attend(rows, table, start, left.clamp(0, rows.shape[1] - 1))
    pool, tab = cache.pool.cpu().numpy(), table.cpu().numpy()
    for b, (c, last) in enumerate(((37, n - 1), (200, 50))):
        total = c + last + 1
        keys, values = lb.read(pool, tab[b], 0, total, D, page)
        ref, mag, reach = lb.attend(q[b, :last + 1].double().cpu().numpy(), keys, values, 0, c, D ** -0.5)
        err = np.abs(out[b, :last + 1].double().cpu().numpy() - ref)
        assert np.all(err <= ta._bound(ref, mag, reach, D, total))
        assert not out[b, last + 1:].any()


# ---- the 8-bit head --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,H,V", [(500, 256, 32000), (500, 384, 31999), (700, 264, 60008)])
def test_a_nan_block_in_the_largest_tiles(R, H, V, dtype):
    """256 x 256 tiles, from one workgroup to the next (bf16, V a multiple of 8)
    and one by one: a NaN block reaches its row or its 128 columns only; every
    other logit keeps its bits."""
    _log(f"[logits] NaN block R={R} H={H} V={V} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(R + V)
    hc, hs = head_quantize(torch.randn(R, H, generator=g, device=DEV), 1)
    wc, ws = head_quantize(torch.randn(V, H, generator=g, device=DEV), 128)
    clean = head_logits(hc, hs, wc, ws, dtype=dtype)
    assert bool(clean.isfinite().all())
    want = torch.zeros(R, V, dtype=torch.bool, device=DEV)
    for row, blk in ((1, 0), (R - 1, hs.shape[1] - 1)):
        hc.view(torch.uint8)[row, 128 * blk:128 * blk + 128] = 0x7f
        hs.view(torch.uint8)[row, blk] = 255
        want[row] = True
    for col, blk in ((3, 1), ((V - 1) // 128, 0)):
        wc.view(torch.uint8)[128 * col:128 * col + 128, 128 * blk:128 * blk + 128] = 0x7f
        ws.view(torch.uint8)[col, blk] = 255
        want[:, 128 * col:128 * col + 128] = True
    got = head_logits(hc, hs, wc, ws, dtype=dtype)
    assert torch.equal(got.isnan(), want)
    assert torch.equal(got.masked_fill(want, 0), clean.masked_fill(want, 0))


def test_states_of_more_than_one_launch():
    """More than 2^31 / 16 blocks of 128 channels: rows on both sides of the
    border between launches, the first and the last; all others are zeros."""
    rows, H = 1 << 20, 16512
    border = (1 << 27) // (H // 128)
    assert rows * (H // 128) > 1 << 27 and border < rows
    x = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    pick = torch.tensor([0, border - 1, border, border + 1, rows - 1], device=DEV)
    g = torch.Generator(device=DEV).manual_seed(8)
    x[pick] = torch.randn(pick.numel(), H, generator=g, device=DEV).bfloat16()
    codes, scales = head_quantize(x)
    rc, rs = lb.quantise_head(x[pick].double().cpu().numpy(), 1)
    assert np.array_equal(codes[pick].double().cpu().numpy(), rc)
    assert np.array_equal(np.exp2(scales.view(torch.uint8)[pick].double().cpu().numpy() - 127.0), rs)
    codes.view(torch.uint8)[pick] = 0
    scales.view(torch.uint8)[pick] = 63                    # 2^-64, the scale of zeros
    step = 1 << 16
    for at in range(0, rows, step):
        assert not codes.view(torch.uint8)[at:at + step].any()
        assert bool((scales.view(torch.uint8)[at:at + step] == 63).all())


@pytest.mark.parametrize("B,K,Hq,Hkv,D,long,short", [
    (128, 5, 24, 8, 256, 131000, 1000), (300, 2, 32, 16, 64, 70000, 30), (520, 1, 16, 8, 128, 50000, 200)])
def test_one_long_request_among_many_short_ones(B, K, Hq, Hkv, D, long, short):
    """More units than the chip holds, one request far longer than the others."""
    _log(f"[attend] skewed B={B} K={K} D={D} {long} among {short}")
    x = Big(B, K, Hq, Hkv, D, short // 2, short, 0)
    ctx = x.ctx.clone()
    ctx[B // 3] = long
    width = (long + K) // x.page + 1
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[:, :x.table.shape[1]] = x.table
    table[B // 3] = torch.arange(width, device=DEV) % x.cache.num_pages       # pages in turn
    got = x.cache.attend(x.q, table, ctx, x.budgets, status=x.status)
    assert int(x.status) == 0
    pick = [B // 3] + list(range(0, B, 7))                 # the long one first
    q, rows, lens, left = x.q[pick], table[pick].contiguous(), ctx[pick], x.budgets[pick]
    ta._check_on_gpu(x.cache, q, got[pick], rows, lens.tolist(), left.tolist())
    assert torch.equal(x.cache.attend(x.q, table, ctx, x.budgets), got)


def test_an_empty_slot_stays_empty_over_steps():
    """The loop of a serving step with a slot that holds no request: its page and
    its length stay as they are, and the other requests' outputs are those of a
    batch without it."""
    B, K, Hq, Hkv, D, V, page = 3, 3, 4, 2, 64, 500, 32
    g = torch.Generator(device=DEV).manual_seed(41)
    head = head_quantize(torch.randn(V, Hq * D, generator=g, device=DEV), 128)
    cache = BlockCache(DEV, 6, Hkv, D, page)
    cache.pool[4:] = 77                                    # the empty slot's pages
    table = _i32([[0, 1], [4, 5], [2, 3]])
    ctx_lens = _i32([9, -1, 0])
    qkv = torch.randn(4, B, K + 1, (Hq + 2 * Hkv) * D, generator=g, device=DEV).bfloat16()
    live = torch.tensor([0, 2], device=DEV)
    verify = SpecVerify(DEV, B, K, V, torch.float32)
    for step in range(4):
        q, k, v = (x.unflatten(-1, (-1, D)) for x in qkv[step].split([Hq * D, Hkv * D, Hkv * D], -1))
        budgets = _i32([K, 2, step])
        cache.write(k, v, table, ctx_lens, budgets)
        o = cache.attend(q, table, ctx_lens, budgets)
        logits = head_logits(*head_quantize(o.view(B * (K + 1), -1)), *head).view(B, K + 1, V)
        drafted = logits[:, :K].argmax(-1).int()
        drafted[:, 1] = 3
        _, n_accepted, _, _ = verify.run(logits, None, drafted, budgets, 0.0, 1, want_probs=False)
        assert torch.equal(o[live], cache.attend(q[live], table[live], ctx_lens[live], budgets[live]))
        before = ctx_lens
        ctx_lens = torch.where(ctx_lens < 0, ctx_lens, ctx_lens + n_accepted + 1)
        assert int(ctx_lens[1]) == -1 and bool((ctx_lens[live] > before[live]).all())
        assert ctx_lens.dtype == torch.int32
    assert bool((cache.pool[4:] == 77).all()) and cache.pool[:4].any()
    assert verify.status() == 0
    verify.close()


@pytest.mark.parametrize("B,K,Hq,Hkv,D,width", [(16384, 0, 4, 2, 64, 600), (2000, 32, 16, 2, 128, 1200),
                                                (3000, 5, 8, 4, 256, 800)])
def test_many_short_requests_under_a_wide_page_table(B, K, Hq, Hkv, D, width):
    """Tens of thousands of units that are cut on the device because the table
    would allow long ones: empty slots among them, every request like the one a
    period before it."""
    _log(f"[attend] {B} short requests, table of {width} pages, K={K} D={D}")
    period, page = 61, 64
    g = torch.Generator(device=DEV).manual_seed(B)
    cache = BlockCache(DEV, 4, Hkv, D, page)
    cache.pool.random_(0, 256, generator=g)
    cache.pool[..., 32 * D:].random_(122, 129, generator=g)
    at = torch.arange(B, device=DEV) % period
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[:, :4] = torch.stack([(at + i) % 4 for i in range(4)], 1).int()
    ctx = (at * 3 - 2).int()                               # -2 .. 178, in turn
    budgets = (at % (K + 1)).int()
    q = torch.randn(period, K + 1, Hq, D, generator=g, device=DEV).bfloat16()
    q = q.repeat(B // period + 1, 1, 1, 1)[:B].contiguous()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert sb.spec_verify_attention_workspace_bytes(B, K, Hq, Hkv, D, page, width, 0) > 256
    got = cache.attend(q, table, ctx, budgets, status=status)
    assert int(status) == 0
    for b0 in (0, B - period):
        part = slice(b0, b0 + period)
        ta._check_on_gpu(cache, q[part], got[part], table[part, :4].contiguous(), ctx[part].tolist(), budgets[part].tolist())
    # Every other request against the same one of the first period: two results
    # that are each off by test_gpu_attention's bound, in which the largest value
    # bounds the weights' sum of |v| and the output, and with the largest sum of
    # |q| every score's reach.
    top = 6.0 * 2.0 ** (128 - 127)
    reach = top * float(q[:period].float().abs().sum(-1).max()) * D ** -0.5
    each = (2.0 ** -8 * (2 + 2.0 ** -7) + 2 * (D + 2) * 2.0 ** -24 * reach + 2.0 ** -20 * (1 + 256 / 4096)) * top
    assert bool(((got.float() - got[:period][at].float()).abs() <= 2 * each).all())
    live = torch.arange(K + 1, device=DEV) <= torch.where(ctx < 0, -1, budgets)[:, None]
    assert bool((got.flatten(2).abs().amax(2) > 0).eq(live).all())
