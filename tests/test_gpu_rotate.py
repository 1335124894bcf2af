"""Normalised and rotated heads on their way into the 4-bit cache.

The cache's bytes are those of a plain write of the rotated keys (compared for
equality; the plain write is tested on its own). The rotated rows themselves are
compared with the fp64 oracle. Tolerance, from the arithmetic, with M the
magnitudes that go into a channel (|y_i| + |y_j|, times the factor):
  - the norm's sum of D squares, its root, quotient and two products are fp32:
    each lane's 8 squares and the tree over lanes, at most 16 roundings of the
    sum, halved by the root, and 5 more: (8 + 5) 2^-24 M; weights are exact;
  - sine and cosine: the angle's fraction of a turn, rounded to fp32, is off by
    2^-26 + 2^-28 turns, so 2^-23.1 radians; the functions by 2 roundings of
    values up to 1, their factor and the two products by one each: 2^-21.5 M;
  - the result is rounded to bf16: half a step, 2^-8 of itself."""
import sys

import numpy as np
import pytest
import torch

from draft_verify_sampling_spec_amd import BlockCache, binding as sb
from oracle import serving as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _log(*a):
    print(*a, file=sys.stderr, flush=True)


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def _check(got, x, positions, live, **kw):
    """got bf16 [B, T, H, D] against the oracle on x of the same shape."""
    ref, mag = sv.rotate(x.double().numpy(), positions[..., None], **kw)
    g = got.double().cpu().numpy()
    tol = (13 * 2.0 ** -24 + 2.0 ** -21.5) * mag * (1 + 2.0 ** -8) + 2.0 ** -8 * (1 + 2.0 ** -10) * np.abs(ref) + 1e-37
    err = np.abs(g - ref)
    assert np.all(err[live] <= tol[live]), float((err[live] / tol[live]).max())


class Case:
    def __init__(self, B, T, Hq, Hkv, D, page, dtype, seed=0, spread=4):
        rng = np.random.default_rng(seed)
        self.__dict__.update(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, page=page)
        gain = np.exp2(rng.integers(-spread, spread + 1, (B, T, 1, 1)).astype(float)) * np.exp(0.5 * rng.normal(size=D))
        self.q, self.k, self.v = (torch.tensor(rng.normal(size=(B, T, h, D)) * gain).to(dtype) for h in (Hq, Hkv, Hkv))
        self.pages = -(-B * T // page) + 3
        # Distinct slots anywhere in the pool; some tokens have none.
        last = self.pages * page - 1
        self.slots = np.append(last, rng.permutation(last)[:B * T - 1]).reshape(B, T)
        self.slots[rng.random((B, T)) < 0.2] = -1
        self.live = self.slots >= 0
        self.rng = rng

    def cache(self, fill=None):
        c = BlockCache(DEV, self.pages, self.Hkv, self.D, self.page)
        c.pool.copy_(torch.tensor(np.random.default_rng(9).integers(0, 256, c.pool.shape).astype(np.uint8)))
        return c

    def run(self, positions, inv_freq=None, wq=None, wk=None, tensors=None, **kw):
        c = self.cache()
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        q, k, v = (t.to(DEV) for t in (self.q, self.k, self.v)) if tensors is None else tensors
        out = torch.full((self.B, self.T, self.Hq, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        keys = torch.full((self.B, self.T, self.Hkv, self.D), 77.0, dtype=torch.bfloat16, device=DEV)
        f = None if inv_freq is None else torch.tensor(inv_freq, dtype=torch.float32, device=DEV)
        w = [None if x is None else x.to(DEV) for x in (wq, wk)]
        got = c.write_rotated(q, k, v, _i32(self.slots), _i32(positions), f, *w, out=out, out_keys=keys,
                              status=status, **kw)
        assert got is out and int(status) == 0
        return c, out, keys

    def check(self, positions, inv_freq=None, wq=None, wk=None, **kw):
        c, out, keys = self.run(positions, inv_freq, wq, wk, **kw)
        opt = {n: x for n, x in kw.items() if n in ("eps", "interleaved", "factor")}
        f = None if inv_freq is None else np.asarray(inv_freq, dtype=np.float32).astype(float)
        for got, x, w in ((out, self.q, wq), (keys, self.k, wk)):
            _check(got, x, positions, self.live, inv_freq=f, weight=None if w is None else w.double().numpy(), **opt)
            assert bool((got[~torch.tensor(self.live)] == 77.0).all())
        # The pool's bytes: a plain write of the rotated keys, token by token.
        plain = self.cache()
        v = self.v.to(DEV)
        kw = keys.to(v.dtype)
        n = self.B * self.T
        ctx = _i32(np.where(self.live, self.slots, -1).reshape(-1))
        table = _i32(np.arange(self.pages)[None].repeat(n, 0))
        plain.write(kw.view(n, 1, self.Hkv, self.D), v.reshape(n, 1, self.Hkv, self.D), table, ctx)
        assert torch.equal(c.pool, plain.pool)


def _freq(rot, base=1e4):
    return base ** (-np.arange(0, rot, 2) / rot)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot,interleaved,norm", [
    (1, 1, 1, 1, 64, 64, False, True),
    (3, 6, 8, 2, 128, 128, False, True),
    (2, 37, 6, 3, 64, 16, True, True),
    (5, 9, 4, 4, 256, 64, False, False),
    (2, 5, 24, 1, 256, 256, True, True),
    (1, 70, 5, 1, 128, 96, False, True),
    (4, 3, 7, 7, 64, 32, True, False),
    (2, 4, 8, 8, 128, 0, False, True),
])
def test_shapes(B, T, Hq, Hkv, D, rot, interleaved, norm, dtype):
    _log(f"[rotate] B={B} T={T} Hq={Hq} Hkv={Hkv} D={D} rot={rot} interleaved={interleaved} norm={norm} {dtype}")
    c = Case(B, T, Hq, Hkv, D, 32, dtype, seed=D + T)
    positions = c.rng.integers(0, 5000, (B, T))
    w = [torch.tensor(np.exp(0.3 * c.rng.normal(size=D))).to(t) for t in (torch.float32,) * 2] if norm else [None, None]
    c.check(positions, _freq(rot) if rot else None, *w, interleaved=interleaved)


def test_bf16_weights_on_one_side_only_eps_and_factor():
    c = Case(2, 5, 4, 2, 128, 64, torch.bfloat16, seed=1)
    w = torch.tensor(np.exp(c.rng.normal(size=128))).bfloat16()
    positions = c.rng.integers(0, 900, (2, 5))
    c.check(positions, _freq(128), w, None, eps=0.5, factor=1.25)
    c.check(positions, _freq(64), None, w, eps=1e-5, factor=-0.5)


def test_positions_far_out_and_before_zero():
    c = Case(2, 6, 4, 2, 128, 64, torch.float32, seed=2)
    positions = np.array([[2**24, 2**24 - 1, 10**7 + 1, 2**20 + 3, 0, 1], [-1, -5, 16777215, 999999, 131071, 2]])
    c.check(positions, _freq(128, 1e6))
    c.check(positions, np.linspace(0.3, 1.0, 32), interleaved=True)


def test_rows_of_zeros_and_of_what_is_not_finite():
    """A zero row stays zero under the norm; a NaN or an infinity stays in its token and head."""
    c = Case(1, 4, 2, 2, 64, 32, torch.float32, seed=3)
    c.slots[:] = [[3, 40, 5, 70]]
    c.q[0, 0], c.k[0, 0] = 0, 0
    c.q[0, 1, 0, 5], c.k[0, 2, 1, 60], c.v[0, 3, 0, 1] = float("nan"), float("inf"), float("nan")
    w = torch.ones(64)
    cache, out, keys = c.run(np.arange(4)[None], _freq(64), w, w)
    assert not out[0, 0].any() and not keys[0, 0].any()
    bad = torch.isnan(out)
    assert bool(bad[0, 1, 0].all()) and int(bad.sum()) == 64
    bad = ~torch.isfinite(keys)
    assert int(bad[0, 2, 1].sum()) >= 1 and not bad[0, [0, 1, 3]].any() and not bad[0, 2, 0].any()
    table = _i32(np.arange(c.pages)[None])
    k, v = cache.read(table, None, _i32([96]), 96)
    assert bool(torch.isnan(v[0, 70, 0, :32]).all()) and not torch.isnan(v[0, 70, 0, 32:]).any()
    assert not torch.isnan(v[0, 70, 1]).any()
    assert bool(torch.isnan(k[0, 5, 1]).any()) and not torch.isnan(k[0, [3, 40, 70]]).any()


def test_slices_of_a_fused_projection():
    c = Case(3, 5, 8, 2, 128, 64, torch.bfloat16, seed=4)
    fused = torch.full((3, 5, 20 * 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    parts, at = [], 0
    for t in (c.q, c.k, c.v):
        n = t.shape[2] * 128
        fused[..., at:at + n] = t.to(DEV).flatten(2)
        parts.append(fused[..., at:at + n].unflatten(-1, (-1, 128)))
        at += n + 512
    positions = c.rng.integers(0, 900, (3, 5))
    want = c.run(positions, _freq(128))
    got = c.run(positions, _freq(128), tensors=parts)
    assert torch.equal(got[0].pool, want[0].pool) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_slots_outside_the_pool_are_flagged_and_skipped():
    c = Case(1, 3, 2, 1, 64, 32, torch.bfloat16, seed=5)
    c.slots[:] = [[c.pages * 32, 7, 2**31 - 1]]
    cache = c.cache()
    before = cache.pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = cache.write_rotated(c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), _i32(c.slots), _i32([[0, 1, 2]]), status=status)
    assert int(status) == sb.SV_FLAG_BAD_PAGE
    assert not out[0, 0].any() and not out[0, 2].any() and torch.equal(out[0, 1], c.q[0, 1].to(DEV))
    changed = (cache.pool != before).flatten(2).any(-1)
    assert int(changed.sum()) == 1 and bool(changed[0, 0])


def test_a_pool_past_32_bit_offsets():
    Hkv, D, page = 8, 128, 128
    pages = (1 << 32) // (Hkv * (page // 32) * 34 * D) + 16
    big = BlockCache(DEV, pages, Hkv, D, page)
    c = Case(1, 4, 8, Hkv, D, page, torch.bfloat16, seed=6)
    q, k, v = (t.to(DEV) for t in (c.q, c.k, c.v))
    last = pages * page
    big.write_rotated(q, k, v, _i32([[last - 1, last - 2, 0, last - 200]]), _i32([[3, 4, 5, 6]]))
    small = BlockCache(DEV, 3, Hkv, D, page)
    small.write_rotated(q, k, v, _i32([[383, 382, 0, 384 - 200]]), _i32([[3, 4, 5, 6]]))
    assert torch.equal(big.pool[-2:], small.pool[-2:]) and torch.equal(big.pool[0], small.pool[0])
    assert not big.pool[1:-2].any()


def test_more_tokens_than_a_row_of_the_grid():
    """300,000 tokens, against two calls of 150,000."""
    n, D = 300_000, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (torch.randn(1, n, 1, D, generator=g, device=DEV).bfloat16() for _ in range(3))
    slots = torch.randperm(n, generator=g, device=DEV).int()[None]
    pos = torch.arange(n, dtype=torch.int32, device=DEV)[None]
    f = torch.tensor(_freq(D), dtype=torch.float32, device=DEV)
    one, two = (BlockCache(DEV, n // 64 + 1, 1, D, 64) for _ in range(2))
    for c in (one, two):
        c.pool.zero_()
    got = one.write_rotated(q, k, v, slots, pos, f)
    parts = [two.write_rotated(*(x[:, i:i + n // 2].contiguous() for x in (q, k, v, slots, pos)), f)
             for i in (0, n // 2)]
    assert torch.equal(got, torch.cat(parts, 1)) and torch.equal(one.pool, two.pool)


def test_bad_arguments_are_refused():
    c = Case(1, 3, 2, 1, 64, 32, torch.bfloat16, seed=5)
    cache = c.cache()
    q, k, v, s = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV), _i32(c.slots)
    good = dict(queries=q, keys=k, values=v, slots=s, positions=s)
    f = torch.ones(32, device=DEV)
    for bad in (dict(queries=q.half()), dict(keys=k.float()), dict(values=v[:, :2]), dict(slots=s.long()),
                dict(positions=s[:, :2]), dict(inv_freq=f[:5]), dict(inv_freq=torch.ones(40, device=DEV)),
                dict(inv_freq=f.double()), dict(q_norm=f), dict(q_norm=torch.ones(64, device=DEV).half()),
                dict(q_norm=torch.ones(64, device=DEV), k_norm=torch.ones(64, device=DEV).bfloat16()),
                dict(out=torch.zeros_like(q).float()), dict(eps=-1.0), dict(factor=float("nan")),
                dict(queries=q.cpu()), dict(queries=q.expand(1, 3, 2, 64).transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((ValueError, RuntimeError)):      # the binding's checks, the library's
            cache.write_rotated(**{**good, **bad})
    empty = cache.write_rotated(q[:, :0], k[:, :0], v[:, :0], s[:, :0].contiguous(), s[:, :0].contiguous())
    assert empty.shape == (1, 0, 2, 64)


def test_a_captured_call_and_another_stream():
    c = Case(2, 6, 4, 2, 128, 64, torch.bfloat16, seed=7)
    positions = c.rng.integers(0, 900, (2, 6))
    cache, want, _ = c.run(positions, _freq(128))
    args = [t.to(DEV) for t in (c.q, c.k, c.v)] + [_i32(c.slots), _i32(positions), torch.tensor(_freq(128), dtype=torch.float32, device=DEV)]
    again, out = c.cache(), torch.full_like(want, 77.0)
    again.write_rotated(*args, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again.write_rotated(*args, out=out)
    for _ in range(3):
        again.pool.copy_(c.cache().pool)
        out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again.pool, cache.pool)
    side = torch.cuda.Stream()
    other = c.cache()
    torch.cuda.synchronize()
    got = other.write_rotated(*args, stream=side)
    side.synchronize()
    assert torch.equal(other.pool, cache.pool)
    assert torch.equal(got[torch.tensor(c.live)], want[torch.tensor(c.live)])
