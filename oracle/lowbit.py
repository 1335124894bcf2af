"""Plain CPU oracle of the 4-bit cache, the blocks' attention over it and the
8-bit output head.

TEST INFRASTRUCTURE. Only ``tests/`` may import this module. It shares no code
with the HIP library and the library never calls it.

Everything is fp64 on the exact values of the inputs.

Number formats (definitions, OCP's e2m1 and e4m3 element formats with a
power-of-two scale per block): a block with largest magnitude a has the scale
2^e, e the smallest integer >= -64 with a <= top * 2^e (top = 6 or 448), at
most the largest e whose top is finite in fp32; a value x becomes the
format's value nearest to x / 2^e, ties to the even code, saturating at top. A
block holding a NaN or an infinity is NaN as a whole (scale byte 255).

Attention: row t of a block at position p = ctx + t sees the positions j in
(p - window, p] (window 0: [0, p]); out = sum_j softmax_j(scale q . k_j) v_j,
taken over exactly those positions.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TILE, GROUP, BLOCK = 32, 32, 128
NAN_BYTE = 255


def scale_exponent(amax, top: float):
    """Exponents e of the blocks' scales, by comparison with every candidate."""
    amax = np.asarray(amax, dtype=np.float64)
    cap = {6.0: 125, 448.0: 119}[top]
    cand = np.arange(-64, cap + 1)
    fits = amax[..., None] <= top * np.exp2(cand.astype(np.float64))
    return np.where(fits.any(-1), cand[fits.argmax(-1)], cap)


def round_e2m1(y):
    """Codes (0..7, plus 8 for a set sign) of y = x / scale, |y| <= 6 or saturating."""
    y = np.asarray(y, dtype=np.float64)
    a = np.minimum(np.abs(y), 6.0)
    d = np.abs(a[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    near = d == best                                   # two codes at a tie: the even one
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return code + 8 * np.signbit(y)


def quantise_cache(x):
    """x [..., D] -> (codes [..., D] 0..15, scale bytes [..., D / 32])."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], 0.0, g)
    e = scale_exponent(np.abs(g).max(-1), 6.0)
    code = round_e2m1(g / np.exp2(e.astype(np.float64))[..., None])
    return code.reshape(x.shape), np.where(bad, NAN_BYTE, e + 127)


def cache_values(codes, bytes_):
    """Values of codes [..., D] under scale bytes [..., D / 32]."""
    v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    s = np.exp2(np.asarray(bytes_, dtype=np.float64) - 127.0)
    s = np.where(np.asarray(bytes_) == NAN_BYTE, np.nan, s)
    return v * np.repeat(s, GROUP, axis=-1)


def tile_addresses(D: int):
    """By the documented layout: byte of every (token, byte of D / 2) of keys and
    values, and of every (token, group)'s scale, inside a tile of 34 D bytes."""
    U, C = min(16, D // 8), min(4, D // 32)
    kc, vc = np.zeros((TILE, D // 2), int), np.zeros((TILE, D // 2), int)
    ks, vs = np.zeros((TILE, D // GROUP), int), np.zeros((TILE, D // GROUP), int)
    for tok in range(TILE):
        half, low = tok // 16, tok % 16
        quad = low // 4
        for y in range(D // 2):
            kc[tok, y] = half * 8 * D + (y // U) * 16 * U + low * U + y % U
            piece = y // C
            vc[tok, y] = (16 * D + ((piece // 16 * 2 + half) * 4 + quad) * 64 * C
                          + piece % 16 * 4 * C + low % 4 * C + y % C)
        for g in range(D // GROUP):
            ks[tok, g] = 32 * D + 32 * g + 2 * low + half
            vs[tok, g] = 33 * D + 32 * g + 8 * quad + 4 * half + low % 4
    return kc, vc, ks, vs


def write(pool, table_row, start: int, keys, values, page_size: int):
    """Store keys and values [n, heads, D] at positions start.. of one request."""
    n, heads, D = keys.shape
    kc, vc, ks, vs = tile_addresses(D)
    for side, (at, at_s) in ((keys, (kc, ks)), (values, (vc, vs))):
        codes, scale = quantise_cache(side)
        packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
        for t in range(n):
            pos = start + t
            page = int(table_row[pos // page_size])
            tile, tok = pos % page_size // TILE, pos % TILE
            for h in range(heads):
                pool[page, h, tile, at[tok]] = packed[t, h]
                pool[page, h, tile, at_s[tok]] = scale[t, h]


def read(pool, table_row, start: int, n: int, D: int, page_size: int):
    """Keys and values [n, heads, D] of positions start .. start + n - 1."""
    kc, vc, ks, vs = tile_addresses(D)
    pos = np.arange(start, start + n)
    page = np.asarray(table_row)[pos // page_size].astype(int)
    tiles = pool[page, :, pos % page_size // TILE]                # [n, heads, 34 D]
    tok = pos % TILE
    out = []
    for at, at_s in ((kc, ks), (vc, vs)):
        packed = np.take_along_axis(tiles, at[tok][:, None, :], axis=-1).astype(int)
        codes = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], D)
        scale = np.take_along_axis(tiles, at_s[tok][:, None, :], axis=-1)
        out.append(cache_values(codes, scale))
    return out


def attend(q, keys, values, first: int, ctx: int, scale: float, window: int = 0):
    """q [T, Hq, D] over keys and values [n, Hkv, D] of positions first..; also
    returns, per output, sum_j p_j |v_j| and, per row and head, the largest
    sum_i |scale q_i k_ji| of a seen position (for error bounds)."""
    T, Hq, D = q.shape
    group = Hq // keys.shape[1]
    out, mag, reach = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for t in range(T):
        p = ctx + t
        lo = max(0, p - window + 1) if window else 0
        sl = slice(lo - first, p + 1 - first)
        for h in range(Hq):
            k, v = keys[sl, h // group], values[sl, h // group]
            z = scale * (k @ q[t, h])
            w = np.exp(z - z.max())
            w /= w.sum()
            out[t, h], mag[t, h] = w @ v, w @ np.abs(v)
            reach[t, h] = (np.abs(scale) * (np.abs(k) @ np.abs(q[t, h]))).max()
    return out, mag, reach


def round_e4m3(y):
    """Values of e4m3 nearest to y, ties to even, saturating at 448."""
    y = np.asarray(y, dtype=np.float64)
    a = np.abs(y)
    _, ex = np.frexp(np.where(a > 0, a, 1.0))              # a = m 2^ex, m in [0.5, 1)
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), y)


def quantise_head(x, block_rows: int):
    """x [N, H] -> (values of the codes [N, Hp], scales [ceil(N / block_rows), Hp / 128])."""
    x = np.asarray(x, dtype=np.float64)
    n, h = x.shape
    nb, hb = -(-n // block_rows), -(-h // BLOCK)
    full = np.zeros((nb * block_rows, hb * BLOCK))
    full[:n, :h] = x
    f = full.reshape(nb, block_rows, hb, BLOCK)
    bad = ~np.isfinite(f).all(axis=(1, 3))
    f = np.where(bad[:, None, :, None], 0.0, f)
    s = np.exp2(scale_exponent(np.abs(f).max(axis=(1, 3)), 448.0).astype(np.float64))
    codes = round_e4m3(f / s[:, None, :, None])
    codes = np.where(bad[:, None, :, None], np.nan, codes)
    return codes.reshape(full.shape)[:n], np.where(bad, np.nan, s)


def head_values(codes, scales, block_rows: int):
    n = codes.shape[0]
    return codes * np.repeat(np.repeat(scales, block_rows, 0)[:n], BLOCK, 1)
