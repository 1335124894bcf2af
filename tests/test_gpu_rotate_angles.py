"""How exactly the rotated write forms its angles: pairs that the turn nearly
cancels, so that the rounding to bf16 hides nothing.

The arithmetic: the angle is formed in fp64, off by at most 2^-29 of a turn
(2 pi 2^-29 < 2^-26.3 radians), cosine and sine are rounded to fp32 (2^-24 of
themselves), so are the two products and their sum, the result goes to bf16
(2^-8 of itself). For x c - y s, and y c + x s likewise:
  2^-26.3 (|x s| + |y c|) + 2 (1 + 2^-20) 2^-24 (|x c| + |y s|) + (2^-24 + 2^-8) (1 + 2^-7) |result|."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache

# pi to 60 digits.
PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def _cases(n, half, seed):
    """Positions, frequencies (fp32, up to 1), and pairs near the angle's own (sine, cosine)."""
    rng = np.random.default_rng(seed)
    positions = rng.integers(-2**24, 2**24 + 1, n)
    positions[:4] = 2**24, -2**24, 1, 0
    freq = np.append(rng.random(half - 1), 1.0).astype(np.float32)
    a = positions[:, None].astype(float) * freq.astype(float)          # exact: 25 times 24 bits
    c, s = np.cos(a), np.sin(a)
    gain = np.exp2(rng.integers(-6, 7, a.shape).astype(float))
    return positions, freq, c, s, (s * gain).astype(np.float32), (c * gain).astype(np.float32)


def _bounds(c, s, x, y):
    x, y = x.astype(float), y.astype(float)
    out = []
    for r, near, far in ((x * c - y * s, abs(x * c) + abs(y * s), abs(x * s) + abs(y * c)),
                         (y * c + x * s, abs(y * c) + abs(x * s), abs(y * s) + abs(x * c))):
        out.append((r, 2 ** -26.3 * far + 2 * (1 + 2 ** -20) * 2 ** -24 * near
                    + (2 ** -24 + 2 ** -8) * (1 + 2 ** -7) * abs(r) + 1e-37))
    return out


def test_the_angle_in_turns_is_right_to_two_to_the_minus_29():
    """The formula itself, against exact arithmetic: position times (frequency times 1 / (2 pi)), all fp64."""
    rng = np.random.default_rng(0)
    worst = Fraction(0)
    for p, f in [(2**24, 1.0), (-2**24, 1.0), (2**24 - 1, float(np.float32(1 - 2**-24)))] + \
            [(int(p), float(np.float32(f))) for p, f in zip(rng.integers(-2**24, 2**24, 3000), rng.random(3000))]:
        x = float(p) * (f * 0.15915494309189533577)
        x -= np.rint(x)
        off = Fraction(float(x)) - Fraction(p) * Fraction(f) / (2 * PI)
        worst = max(worst, abs(off - round(off)))
    assert worst <= Fraction(1, 2**29)


def test_an_angle_rounded_to_fp32_would_be_seen():
    """The bounds below hold for the fp64 formula and not for an angle rounded to fp32 on the way."""
    positions, freq, c, s, x, y = _cases(2000, 64, 1)
    turns = positions[:, None] * (freq.astype(float) * 0.15915494309189533577)
    turns -= np.rint(turns)
    for rounded in (False, True):
        t = turns.astype(np.float32).astype(float) if rounded else turns
        cf, sf = np.cos(2 * np.pi * t).astype(np.float32), np.sin(2 * np.pi * t).astype(np.float32)
        got = torch.tensor(x * cf - y * sf).bfloat16().double().numpy(), torch.tensor(y * cf + x * sf).bfloat16().double().numpy()
        held = [bool((abs(g - r) <= tol).all()) for g, (r, tol) in zip(got, _bounds(c, s, x, y))]
        assert held == [not rounded, True]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_turned_pairs_that_cancel(D, interleaved):
    dev, n, half = torch.device("cuda:0"), 2000, D // 2
    positions, freq, c, s, x, y = _cases(n, half, D)
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    rows = np.zeros((1, n, 1, D), np.float32)
    rows[0, :, 0, first], rows[0, :, 0, second] = x.T, y.T
    q = torch.tensor(rows, device=dev)
    cache = BlockCache(dev, n // 32 + 1, 1, D, 32)
    slots = torch.arange(n, dtype=torch.int32, device=dev)[None]
    keys = torch.zeros(q.shape, dtype=torch.bfloat16, device=dev)
    out = cache.write_rotated(q, q, q, slots, torch.tensor(positions, dtype=torch.int32, device=dev)[None],
                              torch.tensor(freq, device=dev), interleaved=interleaved, out_keys=keys)
    for got in (out, keys):
        g = got[0, :, 0].double().cpu().numpy()
        for at, (r, tol) in zip((first, second), _bounds(c, s, x, y)):
            err = abs(g[:, at] - r)
            assert np.all(err <= tol), float((err / tol).max())
