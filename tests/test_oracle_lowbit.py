"""Pins of the low-bit oracle that do not come from it: torch's own float8
conversion, the formats' definitions, exact enumeration and invariants of the
softmax."""
import numpy as np
import pytest
import torch

from oracle import lowbit as lb


def test_e4m3_rounding_is_torchs():
    x = torch.cat([torch.linspace(-448, 448, 20001), torch.linspace(-0.05, 0.05, 5001)]).float()
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(lb.round_e4m3(x.double().numpy()), want)


def test_e2m1_codes_and_ties():
    for code, v in enumerate(lb.E2M1):
        assert lb.round_e2m1(v) == code and lb.round_e2m1(-v) == code + 8
    # A tie between two values goes to the one whose code is even.
    for y, code in ((0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)):
        assert lb.round_e2m1(y) == code
        assert lb.round_e2m1(np.nextafter(y, 9)) == max(code, lb.round_e2m1(y + 0.01))
    assert lb.round_e2m1(7.5) == 7


@pytest.mark.parametrize("top", [6.0, 448.0])
def test_scale_is_the_smallest_that_fits(top):
    rng = np.random.default_rng(3)
    amax = np.concatenate([top * 2.0 ** np.arange(-60, 100, 7), rng.uniform(0, 1e4, 500)])
    e = lb.scale_exponent(amax, top)
    assert np.all(amax <= top * 2.0 ** e)
    assert np.all((amax > top * 2.0 ** (e - 1.0)) | (e == -64))
    assert lb.scale_exponent(0.0, top) == -64


def test_every_byte_of_a_tile_has_one_place():
    for D in (64, 128, 256):
        seen = np.concatenate([a.ravel() for a in lb.tile_addresses(D)])
        assert np.array_equal(np.sort(seen), np.arange(34 * D))


def test_write_then_read_is_the_quantised_value():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (5, 2, 2, 34 * 64)).astype(np.uint8)
    k, v = rng.normal(size=(2, 70, 2, 64)) * 3
    row = np.array([4, 0, 3])
    lb.write(pool, row, 50, k, v, 64)
    got_k, got_v = lb.read(pool, row, 50, 70, 64, 64)
    for x, got in ((k, got_k), (v, got_v)):
        step = np.repeat(2.0 ** lb.scale_exponent(np.abs(x).reshape(70, 2, 2, 32).max(-1), 6.0), 32, -1)
        assert np.all(np.abs(got - x) <= step)         # half of the widest step, 2
        assert np.array_equal(got, lb.cache_values(*lb.quantise_cache(x)))


def test_attention_of_one_position_and_of_equal_keys():
    rng = np.random.default_rng(2)
    q = rng.normal(size=(2, 4, 64))
    k, v = rng.normal(size=(2, 9, 2, 64))
    out, _, _ = lb.attend(q[:1], k[:1], v[:1], 0, 0, 0.3)
    assert np.allclose(out[0], np.repeat(v[0], 2, 0), atol=1e-15)
    same = np.broadcast_to(k[:1], k.shape)
    out, _, _ = lb.attend(q, same, v, 0, 7, 0.3)
    assert np.allclose(out[1], np.repeat(v.mean(0), 2, 0), atol=1e-14)
    out, _, _ = lb.attend(q, same, v, 0, 7, 0.3, window=3)
    assert np.allclose(out[0], np.repeat(v[5:8].mean(0), 2, 0), atol=1e-14)
