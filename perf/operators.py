"""Measured cases of the operators around a verify step that work on few bits.

Two groups. The paged 4-bit key/value cache of the target model: writing a
block's (or a prompt's) keys and values into it, reading tokens back, and the
attention of every row of a drafted block over it. And the output head in
8-bit floating point: quantising hidden states (a scale per row and 128
channels) or a head (a scale per 128 x 128 block), and the logits of quantised
states under a quantised head.

``own`` selects the library's entry points; otherwise every operator is
computed in its plain form (elementary torch operations in 32 bits).

Number formats. 4 bits: e2m1 codes (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6),
one power-of-two scale per token, head and 32 channels. 8 bits: e4m3, one
power-of-two scale per block of 128. A scale is one byte, 2^(byte - 127), 255
standing for NaN; it is the smallest power of two, at least 2^-64, under which
the block's largest magnitude does not exceed the format's largest value;
codes are rounded to nearest, ties to even.

The cache is uint8 [pages, kv heads, page_size / 32, 34 D]: tiles of 32 tokens
of one head, each [keys' codes 16 D | values' codes 16 D | keys' scales D |
values' scales D] in the orders that ``_tile_parts`` spells out.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
TILE = 32                       # tokens of one cache tile
GROUP = 32                      # channels that share a 4-bit scale
BLOCK = 128                     # channels (and head rows) that share an 8-bit scale
MIN_EXP = -64                   # exponent of the smallest scale
NEW = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # One verify step of the Qwen3-shaped batch: 8 requests, 5 drafted tokens each.
        dict(name="write-step", op="write", B=8, T=6, Hkv=8, D=128, page=64, ctx=1500, dtype="bf16",
             ragged=False),
        # Sixteen prompts of up to 2,049 tokens enter the cache from fp32 projections.
        dict(name="write-prompts", op="write", B=16, T=2049, Hkv=8, D=128, page=64, ctx=0,
             dtype="f32", ragged=True),
        # A short prefix read back, heads of 64 channels, fp32 for a check or a re-quantisation.
        dict(name="read-prefix", op="read", B=4, T=301, Hkv=4, D=64, page=32, ctx=17, dtype="f32",
             ragged=True),
        # Eight long contexts read back for another attention path.
        dict(name="read-contexts", op="read", B=8, T=16384, Hkv=8, D=128, page=128, ctx=0,
             dtype="bf16", ragged=True),
        # Single tokens over short contexts: the smallest serving call.
        dict(name="attend-token", op="attend", B=8, K=0, Hq=32, Hkv=8, D=128, page=64, ctx=577,
             window=0, ragged=True, empty=False),
        # The heavy batch's block shape (budgets 2..8) over ragged contexts of up to 8,192 tokens.
        dict(name="attend-heavy", op="attend", B=128, K=8, Hq=32, Hkv=8, D=128, page=64, ctx=8192,
             window=0, ragged=True, empty=True),
        # One request, a very long context: the work has to be split along it.
        dict(name="attend-long", op="attend", B=1, K=4, Hq=32, Hkv=8, D=128, page=64, ctx=131071,
             window=0, ragged=False, empty=False),
        # Heads of 256 channels with a sliding window, budget 5.
        dict(name="attend-window", op="attend", B=64, K=5, Hq=16, Hkv=8, D=256, page=32, ctx=5000,
             window=1024, ragged=True, empty=False),
        # Hidden states of the Qwen3-shaped step.
        dict(name="quantize-states", op="quantize", rows=48, H=2560, block_rows=1, dtype="bf16"),
        # The Qwen3-shaped head, once at load time.
        dict(name="quantize-head", op="quantize", rows=151936, H=2560, block_rows=128, dtype="bf16"),
        # Logits of the Qwen3-shaped step: 48 rows, the head's bytes are what counts.
        dict(name="logits-step", op="logits", R=48, H=2560, V=151936, dtype="f32"),
        # Logits of the heavy batch's target positions: a large product.
        dict(name="logits-heavy", op="logits", R=2560, H=2560, V=151936, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "quantize", "logits"])
    D = rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 128, 256])
    Hkv = rng.randint(1, 8)
    dtype = rng.choice(["bf16", "f32"])
    if op in ("write", "read"):
        B = _log_int(rng, 1, 64)
        most = (1 << 25) // (B * Hkv * D)                 # at most 2^25 channel values
        return dict(op=op, B=B, T=_log_int(rng, 1, max(2, min(8192, most))), Hkv=Hkv, D=D, page=page,
                    ctx=rng.randint(0, 500), dtype=dtype, ragged=rng.random() < 0.7)
    if op == "attend":
        B = _log_int(rng, 1, 128)
        group = rng.randint(1, 8)
        most = (1 << 28) // (B * Hkv * D)
        return dict(op=op, B=B, K=rng.randint(0, 8), Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                    ctx=_log_int(rng, 1, max(2, min(60000, most))),
                    window=rng.choice([0, 0, _log_int(rng, 16, 4096)]), ragged=rng.random() < 0.7,
                    empty=rng.random() < 0.3)
    H = 8 * _log_int(rng, 8, 640)
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, (1 << 27) // H), H=H,
                    block_rows=rng.choice([1, 128]), dtype=dtype)
    return dict(op=op, R=_log_int(rng, 1, 2048), H=H, V=_log_int(rng, 100, 60000), dtype=dtype)


# ---- number formats, plain ------------------------------------------------------

def _scale_exponent(amax, top_mantissa, top_exponent):
    """Exponent of the smallest power of two s >= 2^MIN_EXP with amax <= top * s,
    top = top_mantissa 2^top_exponent (top_mantissa in [0.5, 1))."""
    m, e = torch.frexp(amax)
    e = e - top_exponent + (m > top_mantissa).to(e.dtype)
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


def _scale_value(byte):
    """2^(byte - 127), fp32; NaN for 255."""
    v = _power(byte.to(torch.int32) - 127)
    return torch.where(byte == 255, torch.full_like(v, math.nan), v)


def _quantize_cache(x):
    """x [..., D] -> (packed codes [..., D/2], scale bytes [..., D/32])."""
    g = x.float().unflatten(-1, (-1, GROUP))
    amax = g.abs().amax(-1)
    bad = ~torch.isfinite(g).all(-1)
    e = _scale_exponent(torch.where(bad, torch.zeros_like(amax), amax), 0.75, 3)
    code = _e2m1_encode(g * _power(-e).unsqueeze(-1)).flatten(-2)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    pair = code.unflatten(-1, (-1, 2))
    return pair[..., 0] | (pair[..., 1] << 4), byte


def _dequantize_cache(packed, byte):
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2)
    v = _e2m1_decode(code).unflatten(-1, (-1, GROUP)) * _scale_value(byte).unsqueeze(-1)
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


def _quantize_head(x, block_rows):
    """x [N, H] -> (e4m3 codes [N, Hp], e8m0 scales [ceil(N / block_rows), Hp / 128])."""
    n, h = x.shape
    nb, hb = -(-n // block_rows), -(-h // BLOCK)
    f = torch.nn.functional.pad(x.float(), (0, hb * BLOCK - h, 0, nb * block_rows - n))
    f = f.view(nb, block_rows, hb, BLOCK)
    amax = f.abs().amax((1, 3))
    bad = ~torch.isfinite(f).all(3).all(1)
    e = _scale_exponent(torch.where(bad, torch.zeros_like(amax), amax), 0.875, 9)
    f = f * _power(-e)[:, None, :, None]
    f = torch.where(bad[:, None, :, None], torch.full_like(f, math.nan), f)
    codes = f.view(nb * block_rows, hb * BLOCK)[:n].to(torch.float8_e4m3fn)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return codes, byte.view(torch.float8_e8m0fnu)


def _dequantize_head(codes, scales, block_rows):
    n, hp = codes.shape
    s = _scale_value(scales.view(torch.uint8))
    s = s.repeat_interleave(block_rows, 0)[:n]
    return (codes.float().view(n, hp // BLOCK, BLOCK) * s.unsqueeze(-1)).view(n, hp)


# ---- inputs ---------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return g


def _ints(lo, hi, n, g):
    """int32 [n], uniform over lo..hi."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEVICE, dtype=torch.int32)


def _table(counts, page, width, g):
    """A page table for requests of counts[b] tokens: pages in a random order,
    -1 behind a request's last page. Returns (table, pages in all)."""
    need = (counts.clamp_min(0) + page - 1) // page
    total = int(need.sum())
    order = torch.randperm(max(total, 1), generator=g, device=DEVICE).to(torch.int32)
    first = torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEVICE, dtype=torch.int32)
    inside = col[None, :] < need[:, None]
    at = torch.where(inside, first[:, None] + col[None, :], torch.zeros_like(first)[:, None])
    return torch.where(inside, order[at.long()], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), max(total, 1)


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


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op in ("write", "read"):
        B, T, page = case["B"], case["T"], case["page"]
        count = _ints((T + 1) // 2, T, B, g) if case["ragged"] else torch.full((B,), T, dtype=torch.int32, device=DEVICE)
        s["ctx"] = _ints(0, case["ctx"], B, g)
        s["budgets"], s["lens"] = count - 1, count
        width = -(-(case["ctx"] + T) // page)
        s["table"], pages = _table(s["ctx"] + count, page, width, g)
        shape = (B, T, case["Hkv"], case["D"])
        s["out_k"], s["out_v"] = (torch.zeros(shape, dtype=NEW[case["dtype"]], device=DEVICE) for _ in range(2))
        if op == "write":
            s["pool"] = torch.zeros(pages, case["Hkv"], page // TILE, 34 * case["D"], dtype=torch.uint8, device=DEVICE)
            gain = torch.exp(0.5 * torch.randn(case["D"], generator=g, device=DEVICE))
            s["k"], s["v"] = ((torch.randn(shape, generator=g, device=DEVICE) * gain).to(NEW[case["dtype"]]) for _ in range(2))
        else:
            s["pool"] = _filled_pool(pages, case, g)
    elif op == "attend":
        B, K, page = case["B"], case["K"], case["page"]
        s["ctx"] = _ints(case["ctx"] // 8, case["ctx"], B, g) if case["ragged"] else torch.full((B,), case["ctx"], dtype=torch.int32, device=DEVICE)
        # Budgets 2 + Binomial(6, 1/3) where the block has 8, else up to K.
        s["budgets"] = (2 + (torch.rand(B, 6, generator=g, device=DEVICE) < 1 / 3).sum(1)).clamp_max(K).to(torch.int32) if K == 8 else _ints(K // 2, K, B, g) if case["ragged"] else torch.full((B,), K, dtype=torch.int32, device=DEVICE)
        if case["empty"] and B > 1:
            s["ctx"][B // 2] = -1                      # a slot that holds no request
        counts = torch.where(s["ctx"] < 0, 0, s["ctx"] + s["budgets"] + 1)
        width = -(-(case["ctx"] + K + 1) // page)
        s["table"], pages = _table(counts, page, width, g)
        s["pool"] = _filled_pool(pages, case, g)
        shape = (B, K + 1, case["Hq"], case["D"])
        s["q"] = torch.randn(shape, generator=g, device=DEVICE).to(torch.bfloat16)
        s["out"] = torch.zeros(shape, dtype=torch.bfloat16, device=DEVICE)
    elif op == "quantize":
        x = torch.randn(case["rows"], case["H"], generator=g, device=DEVICE)
        s["x"] = (x * torch.exp(0.5 * torch.randn(case["H"], generator=g, device=DEVICE))).to(NEW[case["dtype"]])
    else:
        R, H, V = case["R"], case["H"], case["V"]
        s["hq"], s["hs"] = _quantize_head(torch.randn(R, H, generator=g, device=DEVICE), 1)
        w = torch.randn(V, H, generator=g, device=DEVICE) * (3.0 / H ** 0.5)
        s["wq"], s["ws"] = _quantize_head(w, BLOCK)
    return s


# ---- the plain forms ------------------------------------------------------------

def _slots(s, start, count):
    """Where tokens start[b] .. start[b] + T - 1 of every request lie: tile
    index [B, T] (head 0), token in the tile, and which t < count[b]."""
    T, page, Hkv = s["T"], s["page"], s["Hkv"]
    t = torch.arange(T, device=DEVICE)
    pos = start.long()[:, None] + t
    valid = t < count[:, None]
    slot = torch.where(valid, pos // page, torch.zeros_like(pos))
    pages = s["table"].long().gather(1, slot).clamp_min(0)
    tile = pages * (Hkv * page // TILE) + pos % page // TILE
    return tile, pos % TILE, valid


def _head_bytes(s, tile, inside, part):
    """Flat byte positions [B, T, Hkv, n] of one part (offsets [32, n]) of the tokens."""
    D, per_head = s["D"], s["page"] // TILE
    heads = torch.arange(s["Hkv"], device=DEVICE) * per_head
    return (tile[..., None, None] + heads[:, None]) * (34 * D) + part[inside][:, :, None, :]


def _plain_read(s, start, count):
    flat = s["pool"].view(-1)
    tile, inside, valid = _slots(s, start, count)
    parts = _tile_offsets(s["D"], DEVICE)
    k, v = (_dequantize_cache(flat[_head_bytes(s, tile, inside, parts[i])], flat[_head_bytes(s, tile, inside, parts[i + 2])]) for i in (0, 1))
    keep = valid[..., None, None]
    s["out_k"].copy_(torch.where(keep, k.to(s["out_k"].dtype), s["out_k"]))
    s["out_v"].copy_(torch.where(keep, v.to(s["out_v"].dtype), s["out_v"]))
    return s["out_k"], s["out_v"]


def _plain_write(s):
    flat = s["pool"].view(-1)
    tile, inside, valid = _slots(s, s["ctx"], s["lens"])
    parts = _tile_offsets(s["D"], DEVICE)
    kc, ks = _quantize_cache(s["k"])
    vc, vs = _quantize_cache(s["v"])
    flat[_head_bytes(s, tile, inside, parts[0])[valid]] = kc[valid]
    flat[_head_bytes(s, tile, inside, parts[1])[valid]] = vc[valid]
    flat[_head_bytes(s, tile, inside, parts[2])[valid]] = ks[valid]
    flat[_head_bytes(s, tile, inside, parts[3])[valid]] = vs[valid]
    return _plain_read(s, s["ctx"], s["lens"])


def _plain_attend(s):
    B, T, D, Hq, Hkv, page = s["B"], s["K"] + 1, s["D"], s["Hq"], s["Hkv"], s["page"]
    group = Hq // Hkv
    pages = s["pool"][s["table"].clamp_min(0).long()]             # [B, n, Hkv, tiles, 34 D]
    tiles = pages.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, 34 * D)
    kc, vc, ks, vs = _tile_parts(tiles, D)
    L = kc.shape[2] * TILE
    k = _dequantize_cache(kc, ks).view(B, Hkv, L, D)
    v = _dequantize_cache(vc, vs).view(B, Hkv, L, D)
    pos = torch.arange(L, device=DEVICE)
    row = s["ctx"][:, None] + torch.arange(T, device=DEVICE)      # position of every block row
    live = (s["ctx"][:, None] >= 0) & (torch.arange(T, device=DEVICE) <= s["budgets"][:, None])
    sees = pos <= row[..., None]
    if s["window"] > 0:
        sees = sees & (pos > row[..., None] - s["window"])
    sees = sees & live[..., None]                                 # [B, T, L]
    q = s["q"].float().view(B, T, Hkv, group, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * group, D)
    z = q @ k.transpose(-1, -2) * D ** -0.5
    sees = sees.repeat_interleave(group, 1)[:, None]              # [B, 1, T group, L]
    z = torch.where(sees, z, torch.full_like(z, -math.inf))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    v = torch.where(sees.any(2)[..., None], v, torch.zeros_like(v))
    o = (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.view(B, Hkv, T, group, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    s["out"].copy_(torch.where(live[..., None, None], o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _plain_logits(s):
    h = _dequantize_head(s["hq"], s["hs"], 1)
    w = _dequantize_head(s["wq"], s["ws"], BLOCK)
    return (h @ w.T).to(NEW[s["dtype"]])


# ---- one pass -------------------------------------------------------------------

def _cache(s):
    """The cache object that a serving program holds over its pool."""
    if "cache" not in s:
        from draft_verify_sampling_spec_amd import BlockCache
        s["cache"] = BlockCache(s["pool"].device, s["pool"].shape[0], s["Hkv"], s["D"], s["page"], pool=s["pool"])
    return s["cache"]


def run(s):
    op = s["op"]
    if own:
        from draft_verify_sampling_spec_amd import head_logits, head_quantize
        if op == "write":
            # What was stored, as the values it stands for.
            _cache(s).write(s["k"], s["v"], s["table"], s["ctx"], s["budgets"])
            return _cache(s).read(s["table"], s["ctx"], s["lens"], s["T"], out=(s["out_k"], s["out_v"]))
        if op == "read":
            return _cache(s).read(s["table"], s["ctx"], s["lens"], s["T"], out=(s["out_k"], s["out_v"]))
        if op == "attend":
            return _cache(s).attend(s["q"], s["table"], s["ctx"], s["budgets"], window=s["window"], out=s["out"])
        if op == "quantize":
            return head_quantize(s["x"], s["block_rows"])
        return head_logits(s["hq"], s["hs"], s["wq"], s["ws"], dtype=NEW[s["dtype"]])
    if op == "write":
        return _plain_write(s)
    if op == "read":
        return _plain_read(s, s["ctx"], s["lens"])
    if op == "attend":
        return _plain_attend(s)
    if op == "quantize":
        return _quantize_head(s["x"], s["block_rows"])
    return _plain_logits(s)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("write", "read"):
        # Ragged counts are uniform over half to all of T.
        tokens = case["B"] * case["T"] * (0.75 if case["ragged"] else 1.0)
        values = tokens * case["Hkv"] * case["D"] * 2
        size = 2 if case["dtype"] == "bf16" else 4
        cache = values * 17 / 32                                   # codes and scales
        # A write stores its tokens and returns them: both directions.
        moved = (2 * size * values + 2 * cache) if op == "write" else (size * values + cache)
        return {"bytes": moved, "flops": 4 * values}
    if op == "attend":
        B, K, D = case["B"] - (1 if case["empty"] and case["B"] > 1 else 0), case["K"], case["D"]
        ctx = case["ctx"] * (9 / 16 if case["ragged"] else 1.0)
        rows = 5.0 if K == 8 else 1 + (0.75 * K if case["ragged"] else K)
        seen = min(ctx, case["window"]) if case["window"] else ctx
        tokens = seen + rows
        moved = B * (case["Hkv"] * tokens * D * 2 * 17 / 32 + 4 * rows * case["Hq"] * D)
        return {"bytes": moved, "flops": 4.0 * B * rows * case["Hq"] * D * tokens}
    if op == "quantize":
        n = case["rows"] * case["H"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + n, "flops": 3.0 * n}
    R, H, V = case["R"], case["H"], case["V"]
    return {"bytes": (R + V) * H + R * V * (2 if case["dtype"] == "bf16" else 4), "flops": 2.0 * R * H * V}


# ---- 64 bits, from the definitions ------------------------------------------------

def _two(e):
    """2^e, fp64, exactly (integers within the normal range)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_to(x, amax, mantissa_bits, least, top):
    """x [..., n] rounded to a floating format under the power-of-two scale that
    fits amax: (rounded x / scale, scale), everything in fp64."""
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / top))
    # The logarithm may be off by one at a border: settle it by comparison.
    e = torch.where(top * _two(e - 1) >= amax, e - 1, e)
    e = torch.where(top * _two(e) < amax, e + 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp_min(MIN_EXP)
    scale = _two(e)
    y = x / scale.unsqueeze(-1)
    octave = torch.floor(torch.log2(y.abs().clamp_min(1e-300)))
    octave = torch.where(_two(octave) > y.abs(), octave - 1, octave).clamp_min(least)
    step = _two(octave - mantissa_bits)
    return torch.round(y / step) * step, scale


def _exact_rounded(x):
    g = x.double().unflatten(-1, (-1, GROUP))
    y, scale = _round_to(g, g.abs().amax(-1), 1, 0, 6.0)
    return (y * scale.unsqueeze(-1)).flatten(-2)


def _exact_tokens(s, b, start, count):
    """Keys and values [count, Hkv, D] (fp64) of tokens start.. of request b, by address."""
    D, Hkv, page = s["D"], s["Hkv"], s["page"]
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEVICE)
    pos = torch.arange(start, start + count, device=DEVICE)
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
    s = prepare(case, seed)
    op = case["op"]
    if op == "write":
        keep = (torch.arange(case["T"], device=DEVICE) < s["lens"][:, None])[..., None, None]
        return tuple(torch.where(keep, _exact_rounded(s[n]), torch.zeros((), dtype=torch.float64, device=DEVICE)) for n in ("k", "v"))
    if op == "read":
        k, v = (torch.zeros(s["out_k"].shape, dtype=torch.float64, device=DEVICE) for _ in range(2))
        for b, (start, count) in enumerate(zip(s["ctx"].tolist(), s["lens"].tolist())):
            k[b, :count], v[b, :count] = _exact_tokens(s, b, start, count)
        return k, v
    if op == "attend":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEVICE)
        group, D = case["Hq"] // case["Hkv"], case["D"]
        for b, (ctx, budget) in enumerate(zip(s["ctx"].tolist(), s["budgets"].tolist())):
            if ctx < 0:
                continue
            first = max(0, ctx - case["window"] + 1) if case["window"] else 0
            k, v = _exact_tokens(s, b, first, ctx + budget + 1 - first)
            q = s["q"][b, :budget + 1].double().unflatten(1, (case["Hkv"], group))   # [t, h, g, D]
            z = torch.matmul(q.permute(1, 2, 0, 3), k.permute(1, 2, 0).unsqueeze(1)) / math.sqrt(D)
            pos = torch.arange(first, ctx + budget + 1, device=DEVICE)
            row = torch.arange(ctx, ctx + budget + 1, device=DEVICE)[:, None]
            hidden = pos > row
            if case["window"]:
                hidden = hidden | (row - pos >= case["window"])
            w = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
            o = torch.matmul(w, v.permute(1, 0, 2).unsqueeze(1))                     # [h, g, t, D]
            out[b, :budget + 1] = o.permute(2, 0, 1, 3).flatten(1, 2)
        return out
    if op == "quantize":
        n, h, block = case["rows"], case["H"], case["block_rows"]
        nb, hb = -(-n // block), -(-h // BLOCK)
        x = torch.zeros(nb * block, hb * BLOCK, dtype=torch.float64, device=DEVICE)
        x[:n, :h] = s["x"]
        x = x.view(nb, block, hb, BLOCK).transpose(1, 2).reshape(nb, hb, block * BLOCK)
        y, scale = _round_to(x, x.abs().amax(-1), 3, -6, 448.0)
        return y.view(nb, hb, block, BLOCK).transpose(1, 2).reshape(nb * block, hb * BLOCK)[:n], scale
    rows = _two(s["hs"].view(torch.uint8).long() - 127)
    cols = _two(s["ws"].view(torch.uint8).long() - 127).repeat_interleave(BLOCK, 0)[:case["V"]]
    h = s["hq"].double() * rows.repeat_interleave(BLOCK, 1)
    w = s["wq"].double() * cols.repeat_interleave(BLOCK, 1)
    return torch.matmul(h, w.T)
