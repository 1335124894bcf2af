"""Measured cases of the operators of a serving step in front of and inside the
target's attention: page tables and slot maps built from the requests' lengths,
queries and keys normalised and rotated with the keys and values quantised into
the paged 4-bit cache, attention under a sliding window with sink tokens, and
attention of requests that share a long prefix.

``own`` selects the library's entry points; otherwise every operator is
computed in its plain form (elementary torch operations in 32 bits, angles in
64).

The cache is uint8 [pages, kv heads, page_size / 32, 34 D]: tiles of 32 tokens
of one head, each [keys' codes 16 D | values' codes 16 D | keys' scales D |
values' scales D] in the orders that ``_tile_parts`` spells out; e2m1 codes
(sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6) with one power-of-two scale byte per
token, head and 32 channels. A slot is page * page_size + token in the page.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
TILE = 32                       # tokens of one cache tile
GROUP = 32                      # channels that share a 4-bit scale
MIN_EXP = -64                   # exponent of the smallest scale
NEW = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # Two steps of a small batch: 8 requests, 5 drafted tokens, contexts of up to 4,096 tokens.
        dict(name="pages-step", op="pages", B=8, T=6, page=64, ctx=3500, width=64, window=0, sinks=0,
             parents=False, tight=False),
        # Two steps of a full server: 512 requests of up to 65,536 tokens, new ones start from a shared prefix.
        dict(name="pages-serve", op="pages", B=512, T=9, page=64, ctx=60000, width=1024, window=0, sinks=0,
             parents=True, tight=False),
        # Prompts enter in chunks of 2,048 tokens under a window with sinks: pages behind it are given back.
        dict(name="pages-chunks", op="pages", B=64, T=2048, page=32, ctx=30000, width=1024, window=4096,
             sinks=64, parents=False, tight=False),
        # One verify step of the Qwen3-shaped batch: 8 requests, 5 drafted tokens each.
        dict(name="rotate-step", op="rotate", B=8, T=6, Hq=32, Hkv=8, D=128, page=64, ctx=1500, dtype="bf16",
             rot=128, interleaved=False, norm=True, ragged=False),
        # Sixteen prompts of up to 2,049 tokens, as slices of the fused projection's rows.
        dict(name="rotate-prompts", op="rotate", B=16, T=2049, Hq=32, Hkv=8, D=128, page=64, ctx=0, dtype="bf16",
             rot=128, interleaved=False, norm=True, ragged=True),
        # Heads of 256 channels of which 64 turn, in pairs, without norms, far out in long contexts, from fp32.
        dict(name="rotate-far", op="rotate", B=128, T=9, Hq=16, Hkv=8, D=256, page=32, ctx=1000000, dtype="f32",
             rot=64, interleaved=True, norm=False, ragged=True),
        # Single tokens, heads of 64 channels, a short window and 4 sinks.
        dict(name="sinks-token", op="sinks", B=32, K=0, Hq=64, Hkv=8, D=64, page=64, ctx=4000, window=128, sinks=4,
             ragged=True, empty=False),
        # The heavy batch's blocks under a window of 2,048 with 64 sinks.
        dict(name="sinks-heavy", op="sinks", B=128, K=8, Hq=32, Hkv=8, D=128, page=64, ctx=30000, window=2048,
             sinks=64, ragged=True, empty=True),
        # Few requests, a long window, sinks that end inside a tile and a page.
        dict(name="sinks-long", op="sinks", B=4, K=4, Hq=32, Hkv=8, D=128, page=128, ctx=131071, window=32768,
             sinks=1000, ragged=False, empty=False),
        # The Qwen3-shaped batch behind one system prompt of 2,000 tokens.
        dict(name="shared-step", op="shared", G=1, M=8, K=5, Hq=32, Hkv=8, D=128, page=64, prefix=2000, tail=300,
             empty=False),
        # The heavy batch (budgets 2..8) behind a prefix of 8,192 tokens.
        dict(name="shared-heavy", op="shared", G=1, M=128, K=8, Hq=32, Hkv=8, D=128, page=64, prefix=8192,
             tail=1000, empty=True),
        # Four prompts of 16,384 tokens, 64 samples of each, token by token.
        dict(name="shared-samples", op="shared", G=4, M=64, K=0, Hq=32, Hkv=8, D=128, page=64, prefix=16384,
             tail=500, empty=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rotate", "sinks", "shared", "shared"])
    page = rng.choice([32, 64, 128, 256])
    if op == "pages":
        B = _log_int(rng, 1, 512)
        T = _log_int(rng, 1, min(4096, (1 << 17) // B))
        ctx = _log_int(rng, 64, 60000)
        window = rng.choice([0, 0, _log_int(rng, 16, 8192)])
        return dict(op=op, B=B, T=T, page=page, ctx=ctx, width=-(-(ctx + 2 * T) // page) + rng.randint(0, 3),
                    window=window, sinks=_log_int(rng, 1, 300) if window else 0,
                    parents=rng.random() < 0.5, tight=rng.random() < 0.3)
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.randint(1, 8)
    Hq = rng.randint(1, 8) * Hkv
    if op == "rotate":
        B = _log_int(rng, 1, 128)
        most = (1 << 27) // (B * (Hq + 2 * Hkv) * D)          # at most 2^27 channel values
        return dict(op=op, B=B, T=_log_int(rng, 1, max(2, min(4096, most))), Hq=Hq, Hkv=Hkv, D=D, page=page,
                    ctx=_log_int(rng, 1, 100000), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    rot=rng.choice([D, D, D // 2, 32]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.7, ragged=rng.random() < 0.7)
    if op == "sinks":
        B = _log_int(rng, 1, 128)
        most = (1 << 28) // (B * Hkv * D)
        window = _log_int(rng, 16, max(32, min(16384, most)))
        return dict(op=op, B=B, K=rng.randint(0, 8), Hq=Hq, Hkv=Hkv, D=D, page=page,
                    ctx=_log_int(rng, 1, 60000), window=window, sinks=_log_int(rng, 1, 500),
                    ragged=rng.random() < 0.7, empty=rng.random() < 0.3)
    G = _log_int(rng, 1, 8)
    M = _log_int(rng, 1, 128 // G)
    K = rng.choice([0, 0, rng.randint(1, 8)])
    rows = G * M * (K + 1) * Hq
    prefix = _log_int(rng, 32, max(64, min(30000, (1 << 32) // (rows * D))))
    return dict(op=op, G=G, M=M, K=K, Hq=Hq, Hkv=Hkv, D=D, page=page, prefix=prefix,
                tail=_log_int(rng, 1, 1000), empty=rng.random() < 0.3)


# ---- the cache's format, plain ----------------------------------------------------

def _scale_exponent(amax):
    """Exponent of the smallest power of two s >= 2^MIN_EXP with amax <= 6 s."""
    m, e = torch.frexp(amax)                            # amax = m 2^e, 6 = 0.75 * 2^3
    e = e - 3 + (m > 0.75).to(e.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_min(MIN_EXP)


def _e2m1_encode(x):
    """e2m1 code (0..15) of values in [-6, 6]: nearest, ties to even."""
    y = x.abs()
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5)
         + (y >= 3.5) + (y > 5.0))
    return c + 8 * torch.signbit(x).to(torch.uint8)


def _e2m1_decode(code):
    """Value of e2m1 codes (uint8 0..15), fp32."""
    c = (code & 7).to(torch.float32)
    v = torch.where(c < 4, c * 0.5, torch.where(c < 6, c - 2.0, 2.0 * c - 8.0))
    return torch.where(code >= 8, -v, v)


def _power(e):
    """2^e, fp32, exactly (integers -126 <= e <= 127)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantize_cache(x):
    """x [..., D] (finite) -> (packed codes [..., D/2], scale bytes [..., D/32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    e = _scale_exponent(g.abs().amax(-1))
    code = _e2m1_encode(g * _power(-e).unsqueeze(-1)).flatten(-2)
    pair = code.unflatten(-1, (-1, 2))
    return pair[..., 0] | (pair[..., 1] << 4), (e + 127).to(torch.uint8)


def _dequantize_cache(packed, byte):
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    v = _e2m1_decode(code).unflatten(-1, (-1, GROUP)) * _power(byte.to(torch.int32) - 127).unsqueeze(-1)
    return v.flatten(-2)


def _tile_parts(tiles, D):
    """Views of tiles [..., 34 D] by token: keys' codes and values' codes
    [..., 32, D/2], keys' and values' scales [..., 32, D/32]."""
    lead = tiles.shape[:-1]
    n, g = len(lead), D // GROUP
    unit, planes, piece = min(16, D // 8), max(1, D // 128), min(4, D // 32)
    at = list(range(n))
    # Keys: [half of 16 tokens][unit of channels][token][bytes].
    k = tiles[..., :16 * D].view(*lead, 2, D // 2 // unit, 16, unit)
    k = k.permute(*at, n, n + 2, n + 1, n + 3).reshape(*lead, TILE, D // 2)
    # Values: [128 channels][half][4 tokens][piece of channels][token][bytes].
    v = tiles[..., 16 * D:32 * D].view(*lead, planes, 2, 4, 16, 4, piece)
    v = v.permute(*at, n + 1, n + 2, n + 4, n, n + 3, n + 5).reshape(*lead, TILE, D // 2)
    # Keys' scales: [group][token of the half][half].
    ks = tiles[..., 32 * D:33 * D].view(*lead, g, 16, 2)
    ks = ks.permute(*at, n + 2, n + 1, n).reshape(*lead, TILE, g)
    # Values' scales: [group][4 tokens][half][token].
    vs = tiles[..., 33 * D:].view(*lead, g, 4, 2, 4)
    vs = vs.permute(*at, n + 2, n + 1, n + 3, n).reshape(*lead, TILE, g)
    return k, v, ks, vs


def _tile_offsets(D, device):
    """Byte offsets inside a tile of what ``_tile_parts`` returns."""
    return _tile_parts(torch.arange(34 * D, device=device), D)


def _places(s, slots):
    """Flat byte positions [..., Hkv, n] in the pool of the four parts of the
    tokens in slots (int64, none negative)."""
    D, page = s["D"], s["page"]
    per_head = page // TILE
    head = torch.arange(s["Hkv"], device=DEVICE)
    tile = (slots // page).unsqueeze(-1) * (s["Hkv"] * per_head) + head * per_head + (slots % page // TILE).unsqueeze(-1)
    return [(tile * (34 * D)).unsqueeze(-1) + part[slots % TILE].unsqueeze(-2) for part in _tile_offsets(D, DEVICE)]


def _tokens(s, slots):
    """Keys and values [..., Hkv, D] (fp32) of the tokens in slots."""
    flat = s["pool"].view(-1)
    kc, vc, ks, vs = _places(s, slots)
    return _dequantize_cache(flat[kc], flat[ks]), _dequantize_cache(flat[vc], flat[vs])


def _slots_of(s, table, pos):
    """Slots of positions pos [B, n]; where the table holds no page, slot 0's page."""
    page = s["page"]
    pages = table.long().gather(1, (pos // page).clamp(0, table.shape[1] - 1)).clamp_min(0)
    return pages * page + pos % page


# ---- inputs ---------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _ints(lo, hi, n, g):
    """int32 [n], uniform over lo..hi."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEVICE, dtype=torch.int32)


def _table(need, g, spare=0):
    """A page table with pages in a random order where need [B, width] is true,
    -1 elsewhere. Returns (table, pages in all)."""
    total = int(need.sum()) + spare
    order = torch.randperm(max(total, 1), generator=g, device=DEVICE).to(torch.int32)
    at = (need.flatten().cumsum(0) - 1).clamp_min(0).view(need.shape)
    return torch.where(need, order[at], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), max(total, 1)


def _filled_pool(pages, case, g):
    """A cache whose every token was quantised from keys and values with
    channel gains between about 0.2 and 5, as projections have them."""
    D, Hkv, page = case["D"], case["Hkv"], case["page"]
    tiles = page // TILE
    pool = torch.empty(pages, Hkv, tiles, 34 * D, dtype=torch.uint8, device=DEVICE)
    gain = torch.exp(0.5 * torch.randn(2, Hkv, 1, 1, D, generator=g, device=DEVICE))
    ko, vo, kso, vso = _tile_offsets(D, DEVICE)
    step = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, step):
        part = pool[p:p + step]
        for side, (codes_at, scales_at) in enumerate(((ko, kso), (vo, vso))):
            x = torch.randn(part.shape[0], Hkv, tiles, TILE, D, generator=g, device=DEVICE)
            codes, byte = _quantize_cache(x * gain[side])
            part[..., codes_at.flatten()] = codes.flatten(-2)
            part[..., scales_at.flatten()] = byte.flatten(-2)
    return pool


def _columns(width):
    return torch.arange(width, device=DEVICE)


def _needed(ctx, count, page, width, window, sinks):
    """Which pages [B, width] hold a position that a row of the block may see."""
    first = _columns(width) * page
    end = (ctx + count)[:, None]
    need = first < end
    if window:
        seen = (first + page > (ctx[:, None] - window + 1)) | (first < sinks)
        need = need & seen
    return need & (ctx >= 0)[:, None]


def _prepare_pages(s, g):
    B, T, page, width = s["B"], s["T"], s["page"], s["width"]
    fits = width * page
    ctx = _ints(s["ctx"] // 8, s["ctx"], B, g).clamp_max(fits - 2 * T)
    ctx = ctx.clamp_min(0)
    budgets = _ints(0, T - 1, B, g)
    draw01 = torch.rand(B, generator=g, device=DEVICE)
    ends, starts = draw01 < 0.1, draw01 > 0.95
    none = torch.full_like(ctx, -1)
    # First step: some requests have ended, the others go on. Second: those slots
    # hold new requests, others have ended.
    later = ctx + torch.minimum(budgets, _ints(0, T - 1, B, g)) + 1
    s["ctx1"] = torch.where(ends, none, ctx)
    s["ctx2"] = torch.where(starts, none, torch.where(ends, ctx // 2, later))
    s["budgets"] = budgets
    s["parents1"], s["prefix1"] = none, torch.zeros_like(ctx)
    s["parents2"], s["prefix2"] = none, torch.zeros_like(ctx)
    if s["parents"]:
        # A request that lives in both steps, if the drawn one does.
        parent = _ints(0, B - 1, B, g)
        keeps = ~(ends | starts)[parent.long()]
        s["parents2"] = torch.where(ends & keeps, parent, none)
        s["prefix2"] = torch.minimum(s["ctx2"].clamp_min(0), ctx[parent.long()])
    count = budgets + 1
    held = _needed(ctx, count, page, width, s["window"], s["sinks"])
    # A pool for the most that the requests may need, or, tight, for what they need on average.
    longest = min(width, -(-(s["window"] + T) // page) + -(-s["sinks"] // page) + 1) if s["window"] else width
    mean = min((s["ctx"] * 9 / 16 + T) / page, longest)
    pages = max(1, int(B * mean)) if s["tight"] else B * longest
    held = held & (held.sum(1).cumsum(0) <= pages)[:, None]
    s["table"], _ = _table(held, g, pages - int(held.sum()))
    s["refs"] = torch.zeros(pages, dtype=torch.int32, device=DEVICE)
    s["refs"][s["table"][held].long()] = 1


def _rows_of(s, g):
    """Budgets 2 + Binomial(6, 1/3) where the block has 8, else up to K."""
    B, K = s["B"], s["K"]
    if K == 8:
        return (2 + (torch.rand(B, 6, generator=g, device=DEVICE) < 1 / 3).sum(1)).to(torch.int32)
    return _ints(K // 2, K, B, g)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    op, page = s["op"], s.get("page")
    if op == "pages":
        _prepare_pages(s, g)
    elif op == "rotate":
        B, T, Hq, Hkv, D = (s[n] for n in ("B", "T", "Hq", "Hkv", "D"))
        s["lens"] = _ints((T + 1) // 2, T, B, g) if s["ragged"] else torch.full((B,), T, dtype=torch.int32, device=DEVICE)
        ctx = _ints(s["ctx"] // 2, s["ctx"], B, g)
        # Tokens stand at ctx[b] onwards; of the pages before them only the last one is needed here.
        s["first"] = ctx % page
        s["table"], pages = _table(_needed(s["first"], s["lens"], page, -(-(page + T) // page), 0, 0), g)
        t = torch.arange(T, device=DEVICE)
        live = t < s["lens"][:, None]
        s["slots"] = torch.where(live, _slots_of(s, s["table"], s["first"][:, None] + t), -1).to(torch.int32)
        s["positions"] = torch.where(live, ctx[:, None] + t, -1).to(torch.int32)
        fused = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g, device=DEVICE)
        fused *= torch.exp(0.5 * torch.randn(D, generator=g, device=DEVICE))
        fused = fused.to(NEW[s["dtype"]])
        s["q"], s["k"], s["v"] = fused.split([Hq, Hkv, Hkv], 2)
        s["inv_freq"] = 1e6 ** (-torch.arange(0, s["rot"], 2, device=DEVICE, dtype=torch.float32) / s["rot"])
        s["wq"], s["wk"] = (torch.exp(0.3 * torch.randn(D, generator=g, device=DEVICE)) for _ in range(2)) if s["norm"] else (None, None)
        s["pool"] = torch.zeros(pages, Hkv, page // TILE, 34 * D, dtype=torch.uint8, device=DEVICE)
        s["out"] = torch.zeros(B, T, Hq, D, dtype=torch.bfloat16, device=DEVICE)
        s["out_k"], s["out_v"] = (torch.zeros(B, T, Hkv, D, dtype=torch.bfloat16, device=DEVICE) for _ in range(2))
    elif op == "sinks":
        B, K = s["B"], s["K"]
        s["ctx"] = _ints(case["ctx"] // 8, case["ctx"], B, g) if s["ragged"] else torch.full((B,), case["ctx"], dtype=torch.int32, device=DEVICE)
        s["budgets"] = _rows_of(s, g)
        if s["empty"] and B > 1:
            s["ctx"][B // 2] = -1                      # a slot that holds no request
        width = -(-(case["ctx"] + K + 1) // page)
        s["table"], pages = _table(_needed(s["ctx"], s["budgets"] + 1, page, width, s["window"], s["sinks"]), g)
        s["pool"] = _filled_pool(pages, case, g)
    else:
        G, M, K = s["G"], s["M"], s["K"]
        B = s["B"] = G * M
        # Prefixes of half to all of the length, in whole pages; tails behind them.
        common = _ints(case["prefix"] // 2, case["prefix"], G, g) // page * page if G > 1 else torch.full((1,), case["prefix"] // page * page, dtype=torch.int32, device=DEVICE)
        s["groups"] = torch.arange(G, device=DEVICE, dtype=torch.int32).repeat_interleave(M)
        s["shared_lens"] = common.to(torch.int32)
        s["ctx"] = (common[s["groups"].long()] + _ints(1, case["tail"], B, g)).to(torch.int32)
        s["budgets"] = _rows_of(s, g)
        if s["empty"] and B > 1:
            s["ctx"][B // 2] = -1
        width = -(-(case["prefix"] + case["tail"] + K + 1) // page)
        need = _needed(s["ctx"], s["budgets"] + 1, page, width, 0, 0)
        lead = need.view(G, M, width).any(1)           # the prefix's pages are the group's
        shared = (_columns(width) * page < common[:, None]) & lead
        own_pages = need & ~shared.repeat_interleave(M, 0)
        both, pages = _table(torch.cat([shared, own_pages]), g)
        s["table"] = torch.where(need, torch.where(own_pages, both[G:], both[:G].repeat_interleave(M, 0)), -1).to(torch.int32).contiguous()
        s["pool"] = _filled_pool(pages, case, g)
    if op in ("sinks", "shared"):
        shape = (s["B"], s["K"] + 1, s["Hq"], s["D"])
        s["q"] = torch.randn(shape, generator=g, device=DEVICE).to(torch.bfloat16)
        s["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEVICE)
    return s


# ---- the plain forms ------------------------------------------------------------

def _plain_plan(s, ctx, parents, prefix):
    """One step: table and refs in place; (starts, slots, positions)."""
    table, refs, page, T = s["table"], s["refs"], s["page"], s["T"]
    B, width = table.shape
    pages = refs.shape[0]
    count = s["budgets"].clamp(0, T - 1) + 1
    has = (table >= 0) & (table < pages)
    fits = ctx + count <= width * page
    need = torch.where(fits[:, None], _needed(ctx, count, page, width, s["window"], s["sinks"]), has)
    # From the parent's row as it stands before the step.
    of = table[parents.clamp_min(0).long()]
    take = need & ~has & (parents >= 0)[:, None] & (_columns(width) < (prefix // page)[:, None]) & (of >= 0) & (of < pages)
    one = torch.ones((), dtype=torch.int32, device=DEVICE)
    change = torch.zeros(pages + 1, dtype=torch.int32, device=DEVICE)
    change.index_add_(0, torch.where(take, of, pages).flatten().long(), one.expand(B * width))
    change.index_add_(0, torch.where(has & ~need, table, pages).flatten().long(), -one.expand(B * width))
    refs += change[:pages]
    # New pages: the lowest free ones, in the order of requests and positions.
    want = need & ~has & ~take
    news = want.sum(1)
    free = torch.argsort((refs > 0).to(torch.int8), stable=True).to(torch.int32)
    granted = (news == 0) | (news.cumsum(0) <= (refs <= 0).sum())
    rank = (want.flatten().cumsum(0) - 1).clamp(0, pages - 1).view(B, width)
    gets = want & granted[:, None]
    table.copy_(torch.where(gets, free[rank], torch.where(take, of, torch.where(has & need, table, -1))))
    change.zero_()
    change.index_add_(0, torch.where(gets, table, pages).flatten().long(), one.expand(B * width))
    refs.copy_(torch.where(change[:pages] > 0, change[:pages], refs))
    starts = torch.where((ctx >= 0) & fits & granted, ctx, -1).to(torch.int32)
    t = torch.arange(T, device=DEVICE)
    live = (starts >= 0)[:, None] & (t < count[:, None])
    pos = starts.long()[:, None] + t
    slots = torch.where(live, _slots_of(s, table, pos.clamp(0, width * page - 1)), -1).to(torch.int32)
    return starts, slots, torch.where(live, pos, -1).to(torch.int32)


def _plain_rotated(s, x, weight):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight
    angle = s["positions"].double()[..., None] * s["inv_freq"].double()
    c, d = angle.cos().float().unsqueeze(2), angle.sin().float().unsqueeze(2)
    rot = s["rot"]
    turn, rest = y[..., :rot], y[..., rot:]
    if s["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turn = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    else:
        a, b = turn[..., :rot // 2], turn[..., rot // 2:]
        turn = torch.cat([a * c - b * d, b * c + a * d], -1)
    return torch.cat([turn, rest], -1).to(torch.bfloat16)


def _plain_rotate(s):
    live = s["slots"] >= 0
    flat, slots = s["pool"].view(-1), s["slots"][live].long()
    kc, vc, ks, vs = _places(s, slots)
    for x, codes_at, scales_at in ((_plain_rotated(s, s["k"], s["wk"]), kc, ks), (s["v"], vc, vs)):
        codes, byte = _quantize_cache(x[live])
        flat[codes_at] = codes
        flat[scales_at] = byte
    keep = live[..., None, None]
    s["out"].copy_(torch.where(keep, _plain_rotated(s, s["q"], s["wq"]), s["out"]))
    s["out_k"][live], s["out_v"][live] = (x.to(torch.bfloat16) for x in _tokens(s, slots))
    return s["out"], s["out_k"], s["out_v"]


def _by_head(x, Hkv):
    """Rows [B, T, Hq, D] as [B, Hkv, T * group, D]."""
    B, T, Hq, D = x.shape
    return x.view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * (Hq // Hkv), D)


def _finish(s, o, live):
    """Outputs [B, Hkv, T * group, D] into out where a row is live."""
    B, T, Hq, D, Hkv = s["B"], s["K"] + 1, s["Hq"], s["D"], s["Hkv"]
    o = o.view(B, Hkv, T, Hq // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    s["out"].copy_(torch.where(live[..., None, None], o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _weights(z):
    """exp(z - max) and its sum; rows that see nothing: zeros."""
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    return p, p.sum(-1, keepdim=True).clamp_min(1e-30)


def _plain_sinks(s):
    T, D, group, Hkv = s["K"] + 1, s["D"], s["Hq"] // s["Hkv"], s["Hkv"]
    t = torch.arange(T, device=DEVICE)
    row = s["ctx"][:, None] + t                                   # position of every block row
    live = (s["ctx"][:, None] >= 0) & (t <= s["budgets"][:, None])
    # The sinks, then the window's positions behind them.
    low = (s["ctx"] - s["window"] + 1).clamp_min(s["sinks"])[:, None]
    pos = torch.cat([torch.arange(s["sinks"], device=DEVICE).expand(s["B"], -1),
                     low + torch.arange(s["window"] + T, device=DEVICE)], 1)
    k, v = (x.permute(0, 2, 1, 3) for x in _tokens(s, _slots_of(s, s["table"], pos)))
    sees = (pos[:, None] <= row[..., None]) & ((pos[:, None] > row[..., None] - s["window"]) | (pos[:, None] < s["sinks"]))
    sees = (sees & live[..., None]).repeat_interleave(group, 1)[:, None]
    z = _by_head(s["q"].float(), Hkv) @ k.transpose(-1, -2).contiguous() * D ** -0.5
    p, total = _weights(torch.where(sees, z, torch.full_like(z, -math.inf)))
    v = torch.where(sees.any(2)[..., None], v, torch.zeros_like(v))
    return _finish(s, (p @ v) / total, live)


def _plain_shared(s):
    G, M, T, D, Hkv = s["G"], s["M"], s["K"] + 1, s["D"], s["Hkv"]
    group, page = s["Hq"] // Hkv, s["page"]
    t = torch.arange(T, device=DEVICE)
    live = (s["ctx"][:, None] >= 0) & (t <= s["budgets"][:, None])
    q = _by_head(s["q"].float(), Hkv) * D ** -0.5                 # [B, Hkv, T group, D]
    # The prefix, once for all rows of the group, through its first live request's row.
    first = (s["ctx"].view(G, M) >= 0).to(torch.int8).argmax(1) + torch.arange(G, device=DEVICE) * M
    width = s["prefix"] // page * page
    pos = torch.arange(width, device=DEVICE).expand(G, -1)
    kp, vp = (x.permute(0, 2, 1, 3) for x in _tokens(s, _slots_of(s, s["table"][first], pos)))
    qg = q.view(G, M, Hkv, T * group, D).transpose(1, 2).reshape(G, Hkv, M * T * group, D)
    zp = qg @ kp.transpose(-1, -2).contiguous()
    zp = torch.where((pos < s["shared_lens"][:, None])[:, None, None], zp, torch.full_like(zp, -math.inf))
    zp = zp.view(G, Hkv, M, T * group, width).transpose(1, 2).reshape(G * M, Hkv, T * group, width)
    # Every request's own tokens.
    low = s["shared_lens"][s["groups"].long()][:, None]
    pos = low + torch.arange(s["tail"] + T, device=DEVICE)
    kt, vt = (x.permute(0, 2, 1, 3) for x in _tokens(s, _slots_of(s, s["table"], pos)))
    sees = pos[:, None] <= (s["ctx"][:, None] + t)[..., None]
    sees = (sees & live[..., None]).repeat_interleave(group, 1)[:, None]
    zt = q @ kt.transpose(-1, -2).contiguous()
    zt = torch.where(sees, zt, torch.full_like(zt, -math.inf))
    p, total = _weights(torch.cat([zp, zt], -1))
    pp = p[..., :width].reshape(G, M, Hkv, T * group, width).transpose(1, 2).reshape(G, Hkv, M * T * group, width)
    o = (pp @ vp).view(G, Hkv, M, T * group, D).transpose(1, 2).reshape(G * M, Hkv, T * group, D)
    vt = torch.where(sees.any(2)[..., None], vt, torch.zeros_like(vt))
    return _finish(s, (o + p[..., width:] @ vt) / total, live)


# ---- one pass -------------------------------------------------------------------

def _cache(s):
    """The cache object that a serving program holds over its pool."""
    if "cache" not in s:
        from draft_verify_sampling_spec_amd import BlockCache
        s["cache"] = BlockCache(s["pool"].device, s["pool"].shape[0], s["Hkv"], s["D"], s["page"], pool=s["pool"])
    return s["cache"]


def _pages(s):
    if "tables" not in s:
        from draft_verify_sampling_spec_amd import PageTables
        s["tables"] = PageTables(s["table"].device, s["B"], s["width"], s["refs"].shape[0], s["page"],
                                 table=s["table"], refs=s["refs"])
    return s["tables"]


def _plan(s, step):
    ctx, parents, prefix = s["ctx%d" % step], s["parents%d" % step], s["prefix%d" % step]
    if not own:
        return _plain_plan(s, ctx, parents, prefix)
    if not s["parents"]:
        parents = prefix = None
    return _pages(s).plan(ctx, s["budgets"], s["T"], window=s["window"], sinks=s["sinks"], parents=parents,
                          prefix_lens=prefix)


def run(s):
    op = s["op"]
    if op == "pages":
        # Two steps one after another, and what they leave behind.
        return _plan(s, 1), _plan(s, 2), s["table"], s["refs"]
    if own:
        if op == "rotate":
            q = _cache(s).write_rotated(s["q"], s["k"], s["v"], s["slots"], s["positions"], s["inv_freq"], s["wq"],
                                        s["wk"], interleaved=s["interleaved"], out=s["out"])
            # What was stored, as the values it stands for.
            return q, *_cache(s).read(s["table"], s["first"], s["lens"], s["T"], out=(s["out_k"], s["out_v"]))
        if op == "sinks":
            return _cache(s).attend(s["q"], s["table"], s["ctx"], s["budgets"], window=s["window"], sinks=s["sinks"],
                                    out=s["out"])
        return _cache(s).attend_shared(s["q"], s["table"], s["ctx"], s["groups"], s["shared_lens"], s["budgets"],
                                       out=s["out"])
    if op == "rotate":
        return _plain_rotate(s)
    if op == "sinks":
        return _plain_sinks(s)
    return _plain_shared(s)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    if op == "pages":
        B, T, width, page = case["B"], case["T"], case["width"], case["page"]
        seen = min(case["ctx"] * 9 / 16, case["window"] + case["sinks"]) if case["window"] else case["ctx"] * 9 / 16
        refs = B * (seen + T) / page                      # about as many pages as are held
        # Two steps: table and counts read once each, slots and positions written.
        return {"bytes": 2 * 4.0 * (B * width + refs + 2 * B * T + 3 * B), "flops": 2.0 * (B * width + refs)}
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    if op == "rotate":
        tokens = case["B"] * case["T"] * (0.75 if case["ragged"] else 1.0)
        size = 2 if case["dtype"] == "bf16" else 4
        cache = tokens * 2 * Hkv * D * 17 / 32
        # Written once and, for what is returned, read back.
        moved = tokens * (Hq + 2 * Hkv) * D * size + tokens * Hq * D * 2 + 2 * cache + tokens * 2 * Hkv * D * 2
        return {"bytes": moved, "flops": 8.0 * tokens * (Hq + Hkv) * D}
    K = case["K"]
    rows = 5.0 if K == 8 else 1 + 0.75 * K
    if op == "sinks":
        B = case["B"] - (1 if case["empty"] and case["B"] > 1 else 0)
        ctx = case["ctx"] * (9 / 16 if case["ragged"] else 1.0)
        tokens = min(ctx, case["window"] + case["sinks"]) + rows
        moved = B * (Hkv * tokens * D * 2 * 17 / 32 + 4 * rows * Hq * D)
        return {"bytes": moved, "flops": 4.0 * B * rows * Hq * D * tokens}
    B = case["G"] * case["M"] - (1 if case["empty"] and case["G"] * case["M"] > 1 else 0)
    prefix = case["prefix"] * (0.75 if case["G"] > 1 else 1.0)
    tail = case["tail"] / 2 + rows
    moved = (case["G"] * prefix + B * tail) * Hkv * D * 2 * 17 / 32 + B * 4 * rows * Hq * D
    return {"bytes": moved, "flops": 4.0 * B * rows * Hq * D * (prefix + tail)}


# ---- 64 bits, from the definitions ------------------------------------------------

def _two(e):
    """2^e, fp64, exactly (integers within the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_rounded(x):
    """Values of x [..., D] (fp64) in the cache's 4 bits, from the definition."""
    g = x.unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / 6.0))
    # The logarithm may be off by one at a border: settle it by comparison.
    e = torch.where(6.0 * _two(e - 1) >= amax, e - 1, e)
    e = torch.where(6.0 * _two(e) < amax, e + 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_min(MIN_EXP)
    scale = _two(e).unsqueeze(-1)
    y = g / scale
    octave = torch.floor(torch.log2(y.abs().clamp_min(1e-300)))
    octave = torch.where(_two(octave) > y.abs(), octave - 1, octave).clamp_min(0)
    step = _two(octave - 1)
    return (torch.round(y / step) * step * scale).flatten(-2)


def _exact_turned(s, x, weight):
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.double()
    half = s["rot"] // 2
    i = torch.arange(half, device=DEVICE)
    first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE), s["positions"].double()[..., None] * s["inv_freq"].double())
    z = torch.complex(y[..., first], y[..., second]) * turn.unsqueeze(2)
    out = y.clone()
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_tokens(s, b, pos):
    """Keys and values [n, Hkv, D] (fp64) of positions pos of request b, by address."""
    D, Hkv, page = s["D"], s["Hkv"], s["page"]
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEVICE)
    head = torch.arange(Hkv, device=DEVICE)
    ch = torch.arange(D, device=DEVICE)
    page_of = s["table"][b].long()[pos // page]
    tile = ((page_of[:, None] * Hkv + head) * (page // TILE) + (pos % page // TILE)[:, None]) * (34 * D)
    tok = pos % TILE
    half, low = tok // 16, tok % 16
    quad, i = low // 4, low % 4
    unit, piece = min(16, D // 8), min(4, D // 32)
    grp = torch.arange(D // GROUP, device=DEVICE)
    byte = ch // 2
    at_k = half[:, None] * (8 * D) + byte // unit * (16 * unit) + low[:, None] * unit + byte % unit
    per = 2 * piece                                        # channels of one piece
    plane, x = ch // (16 * per), ch % (16 * per) // per
    at_v = 16 * D + ((plane * 2 + half[:, None]) * 4 + quad[:, None]) * (64 * piece) + x * (4 * piece) + i[:, None] * piece + ch % per // 2
    at_ks = 32 * D + grp * 32 + low[:, None] * 2 + half[:, None]
    at_vs = 33 * D + grp * 32 + quad[:, None] * 8 + half[:, None] * 4 + i[:, None]
    flat = s["pool"].view(-1)
    got = []
    for at, at_s in ((at_k, at_ks), (at_v, at_vs)):
        raw = flat[tile[..., None] + at[:, None]]
        code = torch.where(ch % 2 == 1, raw >> 4, raw & 15)
        scale = _two(flat[tile[..., None] + at_s[:, None]].long() - 127)
        got.append(lut[code.long()] * scale.repeat_interleave(GROUP, -1))
    return got


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None                                        # whole numbers only
    s = prepare(case, seed)
    if op == "rotate":
        keep = (s["slots"] >= 0)[..., None, None]
        zero = torch.zeros((), dtype=torch.float64, device=DEVICE)
        # Keys enter the cache as the rotated keys rounded to bf16.
        k = _exact_turned(s, s["k"], s["wk"]).to(torch.bfloat16).double()
        return (torch.where(keep, _exact_turned(s, s["q"], s["wq"]), zero), torch.where(keep, _exact_rounded(k), zero),
                torch.where(keep, _exact_rounded(s["v"].double()), zero))
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
    group, D, Hkv = case["Hq"] // case["Hkv"], case["D"], case["Hkv"]
    for b, (ctx, budget) in enumerate(zip(s["ctx"].tolist(), s["budgets"].tolist())):
        if ctx < 0:
            continue
        row = torch.arange(ctx, ctx + budget + 1, device=DEVICE)[:, None]
        if op == "sinks":
            low = max(0, ctx - case["window"] + 1)
            pos = torch.cat([torch.arange(min(case["sinks"], low), device=DEVICE), torch.arange(low, ctx + budget + 1, device=DEVICE)])
            hidden = (pos > row) | ((row - pos >= case["window"]) & (pos >= case["sinks"]))
        else:
            pos = torch.arange(ctx + budget + 1, device=DEVICE)
            hidden = pos > row
        k, v = _exact_tokens(s, b, pos)
        q = s["q"][b, :budget + 1].double().unflatten(1, (Hkv, group))               # [t, h, g, D]
        z = torch.matmul(q.permute(1, 2, 0, 3), k.permute(1, 2, 0).unsqueeze(1)) / math.sqrt(D)
        w = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
        o = torch.matmul(w, v.permute(1, 0, 2).unsqueeze(1))                         # [h, g, t, D]
        out[b, :budget + 1] = o.permute(2, 0, 1, 3).flatten(1, 2)
    return out
