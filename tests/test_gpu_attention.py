"""Rotary positions, the paged MX cache and attention over it on the GPU,
against the 64-bit restatement in attention_reference.

Tolerances, derived:
  * rope: cos and sin within 2·2^-24 of 1, a product and a fused product and
    sum, each within 2^-24 of its terms: 4·2^-24·m·(|u| + |v|), with half a step of
    the output's type.
  * cache: without a rotation codes and scale bytes are equal; with one, the
    code and byte must be ones that a value within that bound has.  Read
    values are equal.
  * attention: a score's products are exact and its D/16 partial sums each
    within 2^-23 of scale·Σ|q k| =: A, three factors' roundings beside them
    (fp32 queries: 2^-22 more); in units of log2 its exponent u and the
    difference from the maximum round to 2^-24 of at most 1.45 A + 160.  So a
    probability is off by e <= (D/16 + 8)·2^-23·A·ln 2 + 2^-23·(1.45 A + 160)·ln 2 +
    2^-21 (ex2) relative, the numerator and the denominator by that each, and
    their sums by (keys/16 + 30)·2^-23.  Rounded to fp16 it is off by
    finfo.eps / 2 = 2^-11 (two terms for fp32: 2^-22), or 2^-30 of the largest
    P·max|v| a key below fp16's normal numbers.
"""
import numpy as np
import pytest

import attention_reference as ref
import mx_reference as mx

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")


def _torch():
    import torch
    return torch


@pytest.fixture(autouse=True)
def kernel(request):
    """The attention kernel that a test's calls take: as planned, or the one that `KERNELS` says."""
    which = getattr(request, "param", None)
    if which:
        _q().force_attention_kernel(which)
    yield which
    if which:
        _q().force_attention_kernel(None)


KERNELS = pytest.mark.parametrize("kernel", ["few", "many"], indirect=True)


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def _dev(a, name="float32"):
    t = _torch().from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(getattr(_torch(), name))
    return t, t.double().cpu().numpy()


def _half(name):
    return _torch().finfo(getattr(_torch(), name)).eps / 2


def _least(name):
    """Half the spacing of a type's numbers below its smallest normal one (float16: 2^-24 / 2), where a rounding is
    off by that instead of a share of the value."""
    f = _torch().finfo(getattr(_torch(), name))
    return f.smallest_normal * f.eps / 2


def _i32(a):
    return _torch().tensor(np.asarray(a), dtype=_torch().int32, device="cuda")


# Rotary positions.

ROPE = [(1, 1, 32, 32, False), (1, 32, 128, 128, False), (5, 3, 96, 48, False), (3, 2, 64, 64, True),
        (7, 5, 128, 2, True), (9, 1, 80, 24, False), (4, 3, 33, 10, True), (6, 2, 250, 250, False), (2, 1, 1, 0, False),
        (2500, 2, 64, 32, True), (2500, 3, 128, 128, False), (700, 3, 128, 128, False), (1301, 2, 96, 96, False), (40, 7, 256, 256, True), (1, 700, 128, 128, False)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,D,R,interleaved", ROPE)
def test_rope(T, H, D, R, interleaved, dtype):
    q, torch = _q(), _torch()
    r = np.random.default_rng(T * 1000 + D + R)
    x, xv = _dev(r.normal(size=(T, H, D)), dtype)
    pos = r.integers(0, 200000, T)
    f = np.array([10000.0 ** (-2 * i / max(R, 1)) for i in range(R // 2)])
    y = q.rope_rotate(x, torch.tensor(pos, device="cuda", dtype=torch.int32 if T % 2 else torch.int64),
                      q.Rope(torch.tensor(f, device="cuda", dtype=torch.float64), interleaved, 1.25))
    want = ref.turned(xv, pos, f, interleaved, 1.25)
    pairs = np.abs(ref.turned(np.abs(xv), np.zeros(T), f, interleaved)) + np.abs(
        ref.turned(np.abs(xv), np.full(T, 1), np.full(R // 2, np.pi / 2), interleaved)) if R else 0 * xv
    bound = 4 * 2.0 ** -24 * 1.25 * pairs + _half(dtype) * (np.abs(want) + 2.0 ** -20 * pairs) + _least(dtype)
    bound[..., R:] = 0
    got = y.double().cpu().numpy()
    assert y.dtype == x.dtype and (np.abs(got - want) <= bound).all()
    q.device_status()


@pytest.mark.parametrize("far", [2 ** 31 - 1, -2 ** 31, 2 ** 44 + 12345, -(2 ** 50)])
def test_rope_far_positions(far):
    """Angles of far positions keep their precision: the frequency is a multiple of 2^-64 turns, 2π·2^-64 < 2^-61
    radians, from a product good to 2^-62 of its value, so an angle is off by at most |p|·(2^-61 + |f|·2^-60)."""
    q, torch = _q(), _torch()
    from fractions import Fraction
    f = np.array([1.0, 0.37, 1e-3, 1e-8, 5.0, 0.0, -0.25, 1e-300, 3e4])
    pos = [far, far + 1, far - 1 if far > -2 ** 31 else far, 0]
    x = torch.zeros(4, 1, 18, device="cuda")
    x[..., :9] = 1
    wide = max(abs(p) for p in pos) > 2 ** 31 or max(pos) >= 2 ** 31
    y = q.rope_rotate(x, torch.tensor(pos, device="cuda", dtype=torch.int64 if wide else torch.int32),
                      q.Rope(torch.tensor(f, device="cuda"))).cpu().numpy().astype(np.float64)
    two_pi = Fraction(628318530717958647692528676655900576839433879875021, 10 ** 50)   # 2 pi to 50 digits
    for t, p in enumerate(pos):
        for i, fi in enumerate(f):
            a = Fraction(float(fi)) * p
            a -= two_pi * (a // two_pi)
            slack = 4 * 2.0 ** -24 + abs(p) * (2.0 ** -61 + abs(fi) * 2.0 ** -60)
            assert abs(y[t, 0, i] - np.cos(float(a))) <= slack and abs(y[t, 0, 9 + i] - np.sin(float(a))) <= slack


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_and_strided(dtype, interleaved):
    """A part of a fused projection's rows turned where it lies, unaligned; what lies beside it stays."""
    q, torch = _q(), _torch()
    for T, offset, pitch in ((5, 0, 704), (300, 3, 709), (3000, 8, 712)):
        r = np.random.default_rng(T)
        whole, wv = _dev(r.normal(size=(T, pitch)), dtype)
        x = whole[:, offset:offset + 640].view(T, 5, 128)
        pos = torch.arange(T, device="cuda", dtype=torch.int32)
        rope = q.Rope(q.rope_frequencies(128), interleaved)
        apart = q.rope_rotate(x.clone(), pos, rope)
        assert q.rope_rotate(x, pos, rope, out=x) is x
        assert torch.equal(x, apart)
        after = whole.double().cpu().numpy()
        assert np.array_equal(after[:, :offset], wv[:, :offset]) and np.array_equal(after[:, offset + 640:], wv[:, offset + 640:])


def test_rope_specials():
    """NaN and infinite values stay in their pair; frequencies that are not finite give NaN in theirs."""
    q, torch = _q(), _torch()
    x = torch.ones(2, 1, 64, device="cuda")
    x[0, 0, 3], x[1, 0, 40] = float("nan"), float("inf")
    f = q.rope_frequencies(64)
    f[5] = float("inf")
    y = q.rope_rotate(x, torch.tensor([3, 4], device="cuda", dtype=torch.int32), q.Rope(f))
    bad = ~torch.isfinite(y[:, 0])
    assert bad[0].nonzero().flatten().tolist() == [3, 5, 35, 37] and bad[1].nonzero().flatten().tolist() == [5, 8, 37, 40]


def test_rope_frequencies():
    q = _q()
    f = q.rope_frequencies(128, 10000.0).cpu().numpy()
    assert f.shape == (64,) and f[0] == 1 and abs(f[63] - 10000.0 ** (-126 / 128)) < 1e-18
    assert np.allclose(q.rope_frequencies(128, scaling="linear", factor=4).cpu().numpy(), f / 4, rtol=1e-15)
    ntk = q.rope_frequencies(128, scaling="ntk", factor=8).cpu().numpy()
    assert ntk[0] == 1 and abs(ntk[63] * 8 / f[63] - 1) < 1e-12
    parts = q.rope_frequencies(128, scaling="parts", factor=8, original=4096).cpu().numpy()
    turns = 4096 * f / (2 * np.pi)
    assert np.array_equal(parts[turns > 32], f[turns > 32]) and np.array_equal(parts[turns < 1], f[turns < 1] / 8)
    assert ((parts <= f) & (parts >= f / 8)).all()


# The cache.

class Case:
    """A batch in a cache whose pages are dealt at random; every other byte of the cache is noise."""

    def __init__(self, seed, news, lengths, heads, D, page, bits, spare=3, width=None, offset=0):
        r = self.rng = np.random.default_rng(seed)
        used = [-(-max(n, 0) // page) for n in lengths]
        total = sum(used) + spare
        order = r.permutation(total)
        width = max(used + [1]) if width is None else width
        self.table = np.full((len(lengths), width), -7, np.int32)    # entries past a sequence's pages are not read
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.starts = (offset + np.concatenate([[0], np.cumsum(news)])).astype(np.int32)
        self.lengths = np.asarray(lengths, np.int32)
        self.T, self.heads, self.D, self.page, self.bits = int(self.starts[-1]), heads, D, page, bits
        self.cache = {}
        for w in "kv":
            self.cache[w + "_codes"] = r.integers(0, 256, (total, heads, page, D * bits // 8)).astype(np.uint8)
            self.cache[w + "_scales"] = r.integers(0, 256, (total, heads, page, 4)).astype(np.uint8)

    @property
    def batch(self):
        return self.starts, self.lengths, self.table

    def device_batch(self):
        return tuple(_i32(a) for a in self.batch)

    def device_cache(self):
        t = {k: _torch().from_numpy(v.copy()).cuda() for k, v in self.cache.items()}
        return _q().MxCache(t["k_codes"], t["k_scales"], t["v_codes"], t["v_scales"], self.D, self.bits)

    def fill(self, size=1.0, spread=0.4):
        """The sequences' tokens get values quantised from normal ones with channels of different size."""
        for w in "kv":
            c = np.exp(spread * self.rng.normal(size=(self.heads, self.D))) * size
            for i, n in enumerate(self.lengths):
                for p in range(n):
                    pg, at = self.table[i, p // self.page], p % self.page
                    v = self.rng.normal(size=(self.heads, self.D)) * c
                    for h in range(self.heads):
                        codes, byte = ref.head_codes(v[h], self.bits)
                        self.cache[w + "_codes"][pg, h, at], self.cache[w + "_scales"][pg, h, at] = codes, byte
        return self


CACHE = [([1], [1], 1, 32, 16), ([1, 1, 1], [5, 17, 64], 3, 128, 16), ([3, 0, 40], [3, 9, 100], 2, 64, 48),
         ([70], [200], 5, 96, 32), ([2, 5], [1, 33], 1, 128, 64), ([2600, 31], [2700, 31], 2, 64, 128),
         ([800], [850], 3, 128, 16), ([1400, 9], [1500, 40], 2, 64, 32)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,lengths,heads,D,page", CACHE)
def test_cache_write_and_read(news, lengths, heads, D, page, dtype, bits):
    q, torch = _q(), _torch()
    c = Case(len(news) + D, news, lengths, heads, D, page, bits)
    cache, batch = c.device_cache(), c.device_batch()
    scale = np.exp(2 * c.rng.normal(size=(c.T + 2, heads, 1)))
    k, kv = _dev(c.rng.normal(size=(c.T + 2, heads, D)) * scale, dtype)   # two rows behind the last sequence
    v, vv = _dev(c.rng.normal(size=(c.T + 2, heads, D)) * scale, dtype)
    assert q.mx_cache_write(cache, k, v, *batch) is cache
    want = {n: a.copy() for n, a in c.cache.items()}
    rows = {}
    for t, _, _, pg, at in ref.places(c.batch, page):
        for w, x in (("k", kv), ("v", vv)):
            for h in range(heads) if c.T < 500 or t % 97 == 0 else ():
                want[w + "_codes"][pg, h, at], want[w + "_scales"][pg, h, at] = ref.head_codes(x[t, h], bits)
        if c.T < 500 or t % 97 == 0:
            rows[t] = (pg, at)
        else:
            for n in want:
                want[n][pg, :, at] = getattr(cache, n)[pg, :, at].cpu().numpy()
    for n in want:
        assert np.array_equal(getattr(cache, n).cpu().numpy(), want[n]), n
    out = [torch.full((c.T + 2, heads, D), -3.0, device="cuda", dtype=getattr(torch, dtype)) for _ in "kv"]
    got = q.mx_cache_read(cache, *batch, out=out)
    for w, o in zip("kv", got):
        o = o.cpu()
        assert (o[c.T:] == -3).all()
        for t, (pg, at) in rows.items():
            val = torch.from_numpy(ref.head_values(want[w + "_codes"][pg, :, at], want[w + "_scales"][pg, :, at], bits))
            assert torch.equal(o[t], val.to(o.dtype)), (w, t)
    again = q.mx_cache_read(cache, *batch, tokens=c.T, dtype=torch.float32)
    for w, o in zip("kv", again):
        for t, (pg, at) in rows.items():
            val = ref.head_values(want[w + "_codes"][pg, :, at], want[w + "_scales"][pg, :, at], bits)
            assert np.array_equal(o[t].double().cpu().numpy(), val)
    q.device_status()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("R,interleaved,D", [(128, False, 128), (64, True, 128), (36, False, 96), (64, False, 64), (6, True, 32)])
def test_cache_write_turns_keys(R, interleaved, D, dtype, bits):
    q, torch = _q(), _torch()
    c = Case(R, [9, 30], [4000, 30], 2, D, 16, bits)
    cache, batch = c.device_cache(), c.device_batch()
    k, kv = _dev(c.rng.normal(size=(c.T, 2, D)), dtype)
    v, vv = _dev(c.rng.normal(size=(c.T, 2, D)), dtype)
    f = q.rope_frequencies(R)
    q.mx_cache_write(cache, k, v, *batch, rope=q.Rope(f, interleaved, 1.1))
    pos = np.zeros(c.T)
    for t, _, p, _, _ in ref.places(c.batch, 16):
        pos[t] = p
    fn = f.cpu().numpy()
    want = ref.turned(kv, pos, fn, interleaved, 1.1)
    pairs = np.abs(ref.turned(np.abs(kv), 0 * pos, fn, interleaved)) + np.abs(
        ref.turned(np.abs(kv), 0 * pos + 1, np.full(R // 2, np.pi / 2), interleaved))
    off = 4 * 2.0 ** -24 * 1.1 * pairs
    off[..., R:] = 0
    codes, scales = cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy()
    for t, _, _, pg, at in ref.places(c.batch, 16):
        assert np.array_equal(cache.v_codes[pg, 1, at].cpu().numpy(), ref.head_codes(vv[t, 1], bits)[0])
        for h in range(2):
            w, o = want[t, h], off[t, h]
            byte = scales[pg, h, at]
            lo = ref.head_codes(np.maximum(np.abs(w) - o, 0), bits)[1]
            hi = ref.head_codes(np.abs(w) + o, bits)[1]
            assert ((lo <= byte) & (byte <= hi)).all()
            got = mx.code_values(bits)[mx.unpack(codes[pg, h, at][None], bits)][0]
            unit = np.repeat(np.exp2(byte[:D // 32].astype(float) - 127), 32)
            below = mx.code_values(bits)[mx.nearest_code((w - o) / unit, bits)]
            above = mx.code_values(bits)[mx.nearest_code((w + o) / unit, bits)]
            assert ((below <= got) & (got <= above)).all()
    q.device_status()


@pytest.mark.parametrize("T", [700, 1301, 2600, 5003])
def test_rows_in_pieces_and_at_once(T):
    """Rotated and written rows have the same bits whatever the number of rows that a call has."""
    q, torch = _q(), _torch()
    c = Case(T, [T], [T + 11], 3, 128, 16, 8)
    k, _ = _dev(c.rng.normal(size=(T, 3, 128)), "bfloat16")
    rope = q.Rope(q.rope_frequencies(128))
    _, lengths, pages = c.device_batch()
    at_once, pieces = c.device_cache(), c.device_cache()
    q.mx_cache_write(at_once, k, k, *c.device_batch(), rope=rope)
    turned = q.rope_rotate(k, torch.arange(11, T + 11, device="cuda"), rope)
    for i in range(0, T, 100):
        n = min(100, T - i)
        q.mx_cache_write(pieces, k[i:i + n], k[i:i + n], _i32([0, n]), _i32([11 + i + n]), pages, rope=rope)
        assert torch.equal(turned[i:i + n], q.rope_rotate(k[i:i + n], torch.arange(11 + i, 11 + i + n, device="cuda"), rope))
    assert all(torch.equal(a, b) for a, b in zip(at_once[:4], pieces[:4]))
    back = q.mx_cache_read(at_once, *c.device_batch(), tokens=T)
    for i in range(0, T, 100):
        n = min(100, T - i)
        some = q.mx_cache_read(at_once, _i32([0, n]), _i32([11 + i + n]), pages, tokens=n)
        assert torch.equal(back[0][i:i + n], some[0]) and torch.equal(back[1][i:i + n], some[1])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,interleaved,D", [(128, False, 128), (64, True, 128), (36, False, 96), (64, False, 64)])
def test_turned_keys_beside_borders_of_codes(R, interleaved, D, bits):
    """Keys that the rotation takes to within a unit or two of the border between two codes get the code of the exact
    value, where that is 2^-25 of it or more away from the border (the angles and what is made of them are good to 2^-26)."""
    q, torch = _q(), _torch()
    T = 200
    c = Case(R + bits, [T], [T + 3000], 1, D, 16, bits)
    pos = np.arange(3000, 3000 + T)
    f = q.rope_frequencies(R)
    a = pos[:, None] * f.cpu().numpy()
    steps = 16 if bits == 8 else 4          # the significand's borders: odd multiples of 1 / steps
    border = (1 + (2 * c.rng.integers(0, steps // 2, a.shape) + 1) / steps) * 2.0 ** c.rng.integers(0, 2, a.shape)
    near = np.abs(np.cos(a)) >= 0.7         # which of the two parts comes to lie beside it
    part = border / np.where(near, np.cos(a), np.sin(a))
    swap = c.rng.random(a.shape) < 0.5      # from u or from v
    u, v = np.where(swap, 0, part), np.where(swap, part, 0)
    x = np.ones((T, 1, D))
    if interleaved:
        x[:, 0, 0:R:2], x[:, 0, 1:R:2] = u, v
    else:
        x[:, 0, :R // 2], x[:, 0, R // 2:R] = u, v
    k, kv = _dev(x, "float32")
    cache, batch = c.device_cache(), c.device_batch()
    q.mx_cache_write(cache, k, k, *batch, rope=q.Rope(f, interleaved))
    want = ref.turned(kv, pos, f.cpu().numpy(), interleaved)
    codes, scales = cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy()
    beside = 0
    for t, _, _, pg, at in ref.places(c.batch, 16):
        w, unit = want[t, 0], np.repeat(np.exp2(scales[pg, 0, at][:D // 32].astype(float) - 127), 32)
        got = mx.unpack(codes[pg, 0, at][None], bits)[0]
        lo, hi = (mx.nearest_code(w * (1 + e) / unit, bits) for e in (-2.0 ** -25, 2.0 ** -25))
        sure = lo == hi
        assert np.array_equal(got[sure], lo[sure]), (t, np.flatnonzero(sure & (got != lo)))
        wide = [mx.nearest_code(w * (1 + e) / unit, bits) for e in (-2.0 ** -22, 2.0 ** -22)]
        beside += int((sure & (wide[0] != wide[1])).sum())
    # It is these that are tested: an input m · 2^e is off by up to 2^-24 / m of itself, hence by more than 2^-25
    # with probability 1 - m / 2: a quarter of the T R / 2, on average.
    assert beside > T * R // 16


def test_cache_write_specials():
    """A block with an infinity or a NaN reads back as NaN, its neighbours as they are."""
    q, torch = _q(), _torch()
    c = Case(1, [2], [2], 1, 96, 16, 8)
    cache, batch = c.device_cache(), c.device_batch()
    k = torch.ones(2, 1, 96, device="cuda")
    k[0, 0, 40], k[1, 0, 95] = float("inf"), float("nan")
    q.mx_cache_write(cache, k, torch.zeros_like(k), *batch)
    back, zero = q.mx_cache_read(cache, *batch, tokens=2)
    bad = torch.isnan(back[:, 0])
    assert bad[0].nonzero().flatten().tolist() == list(range(32, 64))
    assert bad[1].nonzero().flatten().tolist() == list(range(64, 96))
    assert (back[~torch.isnan(back)] == 1).all() and (zero == 0).all()


# Attention.

def _check(c, x, y, qv, dtype, causal=True, scale=None, heads=None):
    scale = c.D ** -0.5 if scale is None else scale
    want, spread, A, most, keys = ref.attention(qv, c.cache, c.batch, c.bits, scale, causal)
    e = ((c.D / 16 + 8) * A + 1.45 * A + 160) * 2.0 ** -23 * np.log(2) + 2.0 ** -21
    e = 2 * e + (keys / 16 + 30) * 2.0 ** -23 + (2.0 ** -22 + 2.0 ** -21 * A if dtype == "float32" else 2.0 ** -11)
    bound = e * spread + keys * 2.0 ** -30 * most + _half(dtype) * np.abs(want) * 1.01 + _least(dtype) + 1e-37
    got = y.double().cpu().numpy()[:c.T][c.starts[0]:]
    want, bound = want[:c.T][c.starts[0]:], bound[:c.T][c.starts[0]:]
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    worst = (np.abs(got - want) - bound)[ok].max(initial=-1)
    assert worst <= 0, (worst, np.abs(got - want)[ok].max())


ATT = [  # new tokens, lengths, kv heads, group, D, page, bits
    ([1], [1], 1, 1, 32, 16, 8), ([1], [1000], 4, 1, 128, 16, 8), ([1] * 5, [1, 16, 17, 333, 64], 2, 1, 128, 16, 4),
    ([1], [3000], 1, 7, 128, 64, 4), ([2, 1, 3], [40, 129, 3], 2, 3, 64, 48, 8), ([5], [5], 1, 8, 96, 32, 8),
    ([0, 4, 0, 9], [50, 90, 0, 9], 2, 2, 128, 128, 8), ([17], [517], 1, 1, 64, 16, 4), ([40, 3], [40, 200], 2, 4, 128, 64, 8),
    ([150], [150], 2, 1, 128, 32, 8), ([130], [390], 1, 2, 96, 48, 4), ([64, 1, 65], [300, 257, 65], 1, 3, 64, 64, 8),
    ([300], [300], 1, 1, 128, 16, 4), ([129], [700], 1, 4, 128, 64, 8)]


@KERNELS
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,lengths,heads,group,D,page,bits", ATT)
def test_attention(news, lengths, heads, group, D, page, bits, dtype):
    q = _q()
    c = Case(sum(lengths) + D, news, lengths, heads, D, page, bits).fill()
    x, xv = _dev(1.5 * c.rng.normal(size=(c.T, heads * group, D)), dtype)
    y = q.mx_attention(x, c.device_cache(), *c.device_batch())
    q.device_status()
    _check(c, x, y, xv, dtype)


@KERNELS
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("news,lengths", [([1, 1], [70, 33]), ([20, 7], [100, 7]), ([140], [200])])
def test_attention_without_causal_mask(news, lengths, dtype):
    q = _q()
    c = Case(4, news, lengths, 2, 64, 16, 8).fill()
    x, xv = _dev(1.5 * c.rng.normal(size=(c.T, 4, 64)), dtype)
    y = q.mx_attention(x, c.device_cache(), *c.device_batch(), causal=False, scale=0.3)
    _check(c, x, y, xv, dtype, causal=False, scale=0.3)


@KERNELS
@pytest.mark.parametrize("news", [[3, 2], [60, 150]])
def test_attention_rows_that_see_nothing(news):
    """More new rows than tokens, and sequences of no tokens: zeros; rows of no sequence stay."""
    q, torch = _q(), _torch()
    c = Case(9, news, [1, 0], 1, 64, 16, 8, offset=2).fill()
    x, xv = _dev(c.rng.normal(size=(c.T + 3, 2, 64)), "float32")
    out = torch.full_like(x, 7.0)
    assert q.mx_attention(x, c.device_cache(), *c.device_batch(), out=out) is out
    assert (out[:2] == 7).all() and (out[c.T:] == 7).all()
    assert (out[2:2 + news[0] - 1] == 0).all() and (out[2 + news[0]:c.T] == 0).all()
    _check(c, x, out, xv, "float32")
    y = q.mx_attention(x, c.device_cache(), *c.device_batch(), causal=False)
    assert (y[2 + news[0]:c.T] == 0).all()


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [4, 100])
def test_attention_strided(n, dtype):
    """Queries as a part of a fused projection, outputs with heads outermost, neither aligned."""
    q, torch = _q(), _torch()
    c = Case(21, [n], [n + 77], 2, 96, 32, 8).fill()
    fused, _ = _dev(c.rng.normal(size=(n, 1001)), dtype)
    x = fused[:, 5:5 + 4 * 96].view(n, 4, 96)
    buf = torch.full((4, n, 101), 9.0, device="cuda", dtype=x.dtype)
    out = buf[:, :, 3:99].transpose(0, 1)
    q.mx_attention(x, c.device_cache(), *c.device_batch(), out=out)
    _check(c, x, out, x.double().cpu().numpy(), dtype)
    assert (buf[:, :, :3] == 9).all() and (buf[:, :, 99:] == 9).all()


@KERNELS
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 150])
@pytest.mark.parametrize("spread", ["tokens", "blocks", "queries"])
def test_attention_of_wide_ranges(spread, n, dtype):
    """Keys and values whose tokens, or blocks, differ by many powers of two, and queries of any size."""
    q, torch = _q(), _torch()
    c = Case(33, [n], [n + 200], 1, 128, 16, 8).fill(size=0.3)
    size = np.ones((n, 1, 1))
    if spread == "queries":
        size = np.exp2(c.rng.integers(-12, 8, (n, 1, 1)))
    else:
        for w, most in (("k", 6), ("v", 40)):
            s = c.cache[w + "_scales"][..., :4].astype(int)
            by = c.rng.integers(-most, 3, s.shape[:3] + (1,) if spread == "tokens" else s.shape)
            c.cache[w + "_scales"] = np.clip(s + by, 0, 250).astype(np.uint8)
    x, xv = _dev(size * c.rng.normal(size=(n, 2, 128)), dtype)
    y = q.mx_attention(x, c.device_cache(), *c.device_batch())
    _check(c, x, y, xv, dtype)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("n", [7, 150])
def test_attention_hidden_keys_have_no_part(n, dtype):
    """Huge, tiny and infinite-scale keys and values at positions that a row does not see, in the same group of tokens
    as those that it sees, leave its output as it is, to the rounding of other powers of two."""
    q, torch = _q(), _torch()
    c = Case(7, [n], [n + 20], 1, 128, 16, 8).fill()
    x, xv = _dev(c.rng.normal(size=(n, 2, 128)), dtype)
    for w in "kv":
        for p in range(22, n + 20):         # all but the first rows' last keys
            s = c.cache[w + "_scales"][c.table[0, p // 16], 0, p % 16]
            s[:] = np.clip(s.astype(int) + int(c.rng.choice([-60, 0, 40, 100])), 0, 254)
    y = q.mx_attention(x, c.device_cache(), *c.device_batch())
    d = Case(7, [2], [22], 1, 128, 16, 8)
    d.cache, d.table = c.cache, c.table
    few, _ = _dev(xv[:2], dtype)
    _check(d, few, y[:2], xv[:2], dtype)


@KERNELS
@pytest.mark.parametrize("n", [1, 3, 140])
def test_attention_nan_stays_where_it_is_seen(n):
    """NaN blocks of k and v behind a row's last key, in other sequences' pages and in free ones do not reach it; seen
    ones do, those of v only its block's values.  NaN and infinite queries make their own rows NaN."""
    q, torch = _q(), _torch()
    c = Case(5, [n, n], [n + 60, n + 40], 1, 128, 16, 8).fill()
    for i, (where, block) in enumerate((("k", 1), ("v", 2))):
        p = c.lengths[i] - 1                        # the last key: the last row's alone
        c.cache[where + "_scales"][c.table[i, p // 16], 0, p % 16, block] = 255
        c.cache[where + "_codes"][c.table[i, p // 16], 0, p % 16, 32 * block:32 * block + 32] = 0
    used = set(int(t) for i in range(2) for t in c.table[i, :-(-int(c.lengths[i]) // 16)])
    for pg in set(range(c.cache["k_codes"].shape[0])) - used:
        for w in "kv":
            c.cache[w + "_scales"][pg] = 255
    for i in range(2):                              # places behind the last token, in its page
        p = int(c.lengths[i])
        if p % 16:
            for w in "kv":
                c.cache[w + "_scales"][c.table[i, p // 16], :, p % 16:] = 255
                c.cache[w + "_codes"][c.table[i, p // 16], :, p % 16:] = 0x7F
    for dtype in ("bfloat16", "float32"):
        x, xv = _dev(c.rng.normal(size=(c.T, 2, 128)), dtype)
        y = q.mx_attention(x, c.device_cache(), *c.device_batch())
        _check(c, x, y, xv, dtype)
        bad = torch.isnan(y)
        assert bad[n - 1].all() and not bad[:n - 1].any() and not bad[n:2 * n - 1].any()
        assert bad[-1, :, 64:96].all() and not bad[-1, :, :64].any() and not bad[-1, :, 96:].any()
    if n > 1:
        x[0, 0, 5], x[1, 1, 7] = float("nan"), float("inf")
        bad = torch.isnan(q.mx_attention(x, c.device_cache(), *c.device_batch()))
        assert bad[0, 0].all() and not bad[0, 1].any() and bad[1, 1].all() and not bad[1, 0].any()


@KERNELS
def test_attention_repeats_bit_by_bit():
    q, torch = _q(), _torch()
    for news, lengths, heads in (([1, 1], [3000, 777], 2), ([200], [1500], 1)):
        c = Case(2, news, lengths, heads, 64, 16, 8)
        for w in "kv":
            c.cache[w + "_scales"] = (c.cache[w + "_scales"] % 8 + 115).astype(np.uint8)
            c.cache[w + "_codes"] = np.where(c.cache[w + "_codes"] % 128 == 127, 0, c.cache[w + "_codes"])
        x, _ = _dev(c.rng.normal(size=(c.T, 4 * heads, 64)), "bfloat16")
        cache, batch = c.device_cache(), c.device_batch()
        first = q.mx_attention(x, cache, *batch)
        assert torch.isfinite(first).all()
        for _ in range(5):
            assert torch.equal(q.mx_attention(x, cache, *batch), first)


def _bad_batches():
    yield "page above the cache", 5, lambda c: c.table.__setitem__((0, 1), 10 ** 6)
    yield "negative page", 5, lambda c: c.table.__setitem__((0, 0), -1)
    yield "positions beyond the table", 5, lambda c: c.lengths.__setitem__(0, 10 ** 6)


@KERNELS
@pytest.mark.parametrize("n", [5, 150])
@pytest.mark.parametrize("what", range(3))
def test_bad_pages_are_reported_and_not_accessed(what, n):
    q, torch = _q(), _torch()
    c = Case(3, [n, 4], [n + 30, 20], 1, 64, 16, 8).fill()
    list(_bad_batches())[what][2](c)
    cache, batch = c.device_cache(), c.device_batch()
    before = [t.clone() for t in cache[:4]]
    x, xv = _dev(c.rng.normal(size=(c.T, 2, 64)), "float32")
    q.device_status()
    calls = [lambda: q.mx_attention(x, cache, *batch)]
    if what == 2:   # (a bad page that a small write does not touch is no error of its)
        calls += [lambda: q.mx_cache_read(cache, *batch, tokens=c.T), lambda: q.mx_cache_write(cache, x[:, :1], x[:, :1], *batch)]
    for call in calls:
        y = call()
        with pytest.raises(q.Q4mmError) as e:
            q.device_status()
        assert e.value.code == -7
        q.device_status()
        if torch.is_tensor(y):      # the other sequence is as it should be
            d = Case(3, [n, 4], [n + 30, 20], 1, 64, 16, 8).fill()
            ok = q.mx_attention(x, d.device_cache(), *d.device_batch())
            assert torch.equal(y[n:], ok[n:])
            q.device_status()
    if what == 2:
        pages = [int(p) for p in c.table[1, :2]]
        for t, b in zip(cache[:4], before):
            rest = [p for p in range(t.shape[0]) if p not in pages]
            assert torch.equal(t[rest], b[rest])


def test_no_tokens_and_no_sequences():
    q, torch = _q(), _torch()
    cache = q.mx_cache(4, 2, 64, page=16)
    none = (_i32([0, 0]), _i32([5]), _i32([[1]]))
    assert q.mx_attention(torch.zeros(0, 4, 64, device="cuda"), cache, *none).shape == (0, 4, 64)
    k = torch.zeros(0, 2, 64, device="cuda")
    q.mx_cache_write(cache, k, k, *none)
    assert q.mx_cache_read(cache, *none, tokens=0)[0].shape == (0, 2, 64)
    assert q.rope_rotate(k, _i32([]), q.Rope(q.rope_frequencies(64))).shape == (0, 2, 64)
    out = torch.full((3, 4, 64), 5.0, device="cuda")
    q.mx_attention(torch.zeros(3, 4, 64, device="cuda"), cache, _i32([0]), _i32([]), _i32(np.zeros((0, 0))), out=out)
    assert (out == 5).all()
    q.device_status()


def test_steps_in_a_graph_and_on_another_stream():
    """Decoding steps captured once and replayed on new tokens, lengths and pages, against plain calls."""
    q, torch = _q(), _torch()
    c = Case(8, [1, 1], [30, 77], 2, 64, 16, 8, spare=4, width=8).fill()
    for i, n in ((0, 2), (1, 5)):       # free pages to grow into
        c.table[i, n] = min(set(range(len(c.cache["k_codes"]))) - set(c.table[c.table >= 0].tolist()))
    cache, (starts, lengths, pages) = c.device_cache(), c.device_batch()
    plain = c.device_cache()
    rope = q.Rope(q.rope_frequencies(64))
    x, k, v = (torch.zeros(2, h, 64, device="cuda", dtype=torch.bfloat16) for h in (4, 2, 2))
    pos = lengths - 1

    def step(on, **kw):
        r = q.rope_rotate(x, pos, rope, **kw)
        q.mx_cache_write(on, k, v, starts, lengths, pages, rope=rope, **kw)
        return q.mx_attention(r, on, starts, lengths, pages, **kw)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(c.device_cache())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(cache)
    g = torch.Generator(device="cuda").manual_seed(0)
    for i in range(4):
        for t in (x, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        graph.replay()
        assert torch.equal(out, step(plain))
        lengths += 1
        pos.copy_(lengths - 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        y = step(plain, stream=side)
    torch.cuda.synchronize()
    graph.replay()
    assert torch.equal(out, y)
    q.device_status()


def test_captured_without_a_call_before():
    """A process whose first calls are captured: nothing of them needs a call outside a capture."""
    import os
    import subprocess
    import sys
    code = """
import torch, quantized_matmul_q4_gb300 as q
cache = q.mx_cache(64, 1, 64, page=16)
rope = q.Rope(q.rope_frequencies(64))
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
x, v = torch.randn(2, 200, 1, 64, device="cuda")
many = (i32(0, 200), i32(200), torch.arange(64, dtype=torch.int32, device="cuda")[None])
few = (i32(0, 1), i32(200), many[2])
pos = torch.arange(200, device="cuda")
def calls():
    q.mx_cache_write(cache, x, v, *many, rope=rope)
    out = [q.rope_rotate(x, pos, rope), *q.mx_cache_read(cache, *many, tokens=200)]
    for which in ("few", "many"):
        q.force_attention_kernel(which)
        out.append(q.mx_attention(x, cache, *many))
    q.force_attention_kernel(None)
    return out + [q.mx_attention(x[:1], cache, *few)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
q.device_status()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


@KERNELS
def test_broadcast_inputs():
    """Rows, heads, keys and values of stride zero."""
    q, torch = _q(), _torch()
    c = Case(12, [40], [50], 2, 64, 16, 8).fill()
    one, _ = _dev(c.rng.normal(size=(1, 1, 64)), "float32")
    row, _ = _dev(c.rng.normal(size=(1, 6, 64)), "float32")
    for x in (one.expand(40, 6, 64), row.expand(40, 6, 64)):
        y = q.mx_attention(x, c.device_cache(), *c.device_batch())
        assert torch.equal(y, q.mx_attention(x.contiguous(), c.device_cache(), *c.device_batch()))
    got, want = c.device_cache(), c.device_cache()
    rope = q.Rope(q.rope_frequencies(64))
    k = one.expand(40, 2, 64)
    q.mx_cache_write(got, k, k, *c.device_batch(), rope=rope)
    q.mx_cache_write(want, k.contiguous(), k.contiguous(), *c.device_batch(), rope=rope)
    assert all(torch.equal(a, b) for a, b in zip(got[:4], want[:4]))
    pos = torch.arange(40, device="cuda")
    assert torch.equal(q.rope_rotate(k, pos, rope, out=torch.empty(40, 2, 64, device="cuda")), q.rope_rotate(k.contiguous(), pos, rope))


@KERNELS
def test_long_cache_offsets_pass_32_bits():
    """Pages whose bytes lie beyond 2^32 of the base."""
    q, torch = _q(), _torch()
    pages = 5 * 2 ** 30 // (16 * 64) // 1
    codes = [torch.empty(pages, 1, 16, 64, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full((pages, 1, 16, 4), 120, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache = q.MxCache(codes[0], scales[0], codes[1], scales[1], 64, 8)
    for n in (3, 150):
        small = Case(6, [n], [n + 21], 1, 64, 16, 8).fill()
        moved = [pages - 1 - int(p) for p in small.table[0]]
        for name in small.cache:
            for old, new in zip(small.table[0], moved):
                getattr(cache, name)[new] = torch.from_numpy(small.cache[name][old]).cuda()
        x, xv = _dev(small.rng.normal(size=(n, 2, 64)), "bfloat16")
        batch = small.device_batch()
        y = q.mx_attention(x, cache, batch[0], batch[1], _i32([moved]))
        assert torch.equal(y, q.mx_attention(x, small.device_cache(), *batch))
        k, v = _dev(small.rng.normal(size=(n, 1, 64)))[0], _dev(small.rng.normal(size=(n, 1, 64)))[0]
        near = small.device_cache()
        q.mx_cache_write(near, k, v, *batch)
        q.mx_cache_write(cache, k, v, batch[0], batch[1], _i32([moved]))
        for a, b in zip(q.mx_cache_read(near, *batch, tokens=n), q.mx_cache_read(cache, batch[0], batch[1], _i32([moved]), tokens=n)):
            assert torch.equal(a, b)
    q.device_status()
