"""Plain CPU oracle of what a serving step does in front of and inside the
target's attention: page tables from lengths, normalised and rotated heads, the
positions that a row sees under a window with sinks.

TEST INFRASTRUCTURE. Only ``tests/`` may import this module. It shares no code
with the HIP library and the library never calls it. Whole numbers are exact,
everything else is fp64 on the exact values of the inputs.
"""
from __future__ import annotations

import numpy as np

BAD_BUDGET, BAD_LENGTH, BAD_PAGE, NO_PAGES, BAD_PARENT, NO_PREFIX = 0x1, 0x8, 0x10, 0x20, 0x40, 0x80


def visible(p: int, window: int = 0, sinks: int = 0):
    """The positions that a row at position p sees."""
    return [j for j in range(p + 1) if not window or j > p - window or j < sinks]


def needed_pages(ctx: int, n: int, page: int, window: int = 0, sinks: int = 0):
    """The pages that hold a position seen by a row at ctx or later, or a sink
    of the block's span, up to position ctx + n - 1."""
    if ctx < 0 or n <= 0:
        return set()
    low = max(0, ctx - window + 1) if window else 0
    need = set(range(low // page, (ctx + n - 1) // page + 1))
    if window:
        need |= set(range(0, min(-(-sinks // page), (ctx + n - 1) // page + 1)))
    return need


def plan(table, refs, ctx, budgets, T, page, window=0, sinks=0, parents=None, prefix=None):
    """(table, refs, starts, slots, positions, flags) after one step, request by request."""
    before, table, refs = np.array(table), np.array(table), np.array(refs)
    B, width = table.shape
    flags, new = 0, {}
    keep = set()
    for b in range(B):
        c = int(ctx[b])
        k = T - 1 if budgets is None else int(budgets[b])
        if c >= 0 and not 0 <= k < T:
            flags |= BAD_BUDGET
        n = min(max(k, 0), T - 1) + 1
        if c >= 0 and c + n > width * page:
            flags |= BAD_LENGTH
            keep.add(b)
            new[b] = []
            continue
        need = needed_pages(c, n, page, window, sinks)
        parent = -1 if parents is None else int(parents[b])
        if parent >= 0 and (parent >= B or parent == b or parents[parent] >= 0):
            flags |= BAD_PARENT
            parent = -1
        # Whole pages in front of the request's new tokens.
        common = min(max(int(prefix[b]), 0), max(c, 0)) // page if parent >= 0 else 0
        new[b] = []
        for i in range(width):
            held = int(before[b, i])
            if held >= len(refs):
                flags |= BAD_PAGE
            has = 0 <= held < len(refs)
            if has and i not in need:
                refs[held] -= 1
            if not (has and i in need):
                table[b, i] = -1
            if i in need and not has:
                other = int(before[parent, i]) if i < common else -1
                if 0 <= other < len(refs):
                    refs[other] += 1
                    table[b, i] = other
                else:
                    new[b].append(i)
                    if i < common:
                        flags |= NO_PREFIX
    free = [p for p in range(len(refs)) if refs[p] <= 0]
    starts, slots, positions = np.full(B, -1), np.full((B, T), -1), np.full((B, T), -1)
    used = 0
    for b in range(B):
        used += len(new[b])
        if new[b] and used > len(free):
            flags |= NO_PAGES
            continue
        for j, i in enumerate(new[b]):
            p = free[used - len(new[b]) + j]
            table[b, i] = p
            refs[p] = 1
        if b in keep or ctx[b] < 0:
            continue
        starts[b] = ctx[b]
        k = T - 1 if budgets is None else int(budgets[b])
        for t in range(min(max(k, 0), T - 1) + 1):
            pos = int(ctx[b]) + t
            positions[b, t] = pos
            slots[b, t] = table[b, pos // page] * page + pos % page
    return table, refs, starts, slots, positions, flags


def rotate(x, position, inv_freq=None, weight=None, eps=1e-6, interleaved=False, factor=1.0):
    """x [..., D] normalised and turned to its position (any shape that broadcasts
    against x without its channels); also, per channel, the sum of the magnitudes
    that went into it (for error bounds)."""
    y = np.asarray(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    out, mag = y.copy(), np.abs(y)
    half = 0 if inv_freq is None else len(inv_freq)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a = np.asarray(position, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(a) * factor, np.sin(a) * factor
        out[..., p] = y[..., p] * c - y[..., q] * s
        out[..., q] = y[..., q] * c + y[..., p] * s
        mag[..., p] = mag[..., q] = (np.abs(y[..., p]) + np.abs(y[..., q])) * abs(factor)
    return out, mag


def attend(q, keys, values, ctx: int, scale: float, window: int = 0, sinks: int = 0):
    """q [T, Hq, D] over keys and values [n, Hkv, D] of positions 0..n - 1; also
    returns, per output, sum_j p_j |v_j| and, per row and head, the largest
    sum_i |scale q_i k_ji| of a seen position (for error bounds)."""
    T, Hq, D = q.shape
    group = Hq // keys.shape[1]
    out, mag, reach = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for t in range(T):
        sees = visible(ctx + t, window, sinks)
        for h in range(Hq):
            k, v = keys[sees, h // group], values[sees, h // group]
            z = scale * (k @ q[t, h])
            w = np.exp(z - z.max())
            w /= w.sum()
            out[t, h], mag[t, h] = w @ v, w @ np.abs(v)
            reach[t, h] = (np.abs(scale) * (np.abs(k) @ np.abs(q[t, h]))).max()
    return out, mag, reach
