"""MX operators on the GPU against the 64-bit restatement in mx_reference.

Tolerances, derived:
  * quantisation and dequantisation are exact (v / scale is a multiplication by
    a power of two; the conversion rounds once): codes, scale bytes and values
    are equal.
  * rmsnorm: v takes one rounding for h, one for the product with the norm and
    one for the weight, and the norm's relative error, half that of the sum of
    squares (a tree of at most 32 + 10 + 10 additions of positive terms, and
    the squares' own rounding: 53 · 2^-24) plus rsqrtf's 2 ulp and the
    addition of eps: below 40 · 2^-24 < 3e-6 in all.  A code must then be one
    that some value within that of the exact one has, under the scale byte
    found, which must be that of some such block maximum.
  * swiglu: the exponential and its correction (5 · 2^-24), one addition, the
    reciprocal (2 · 2^-24), two multiplications: 10 · 2^-24 < 1e-6 relative
    (test_gpu_mx_swiglu_range holds it to that over the whole range of gates).
  * matmul: products are exact; at most Kp / 32 sums are chained per output,
    each within one unit in the last place of a partial sum, 2^-23 of
    sum |x w| (the tensor cores may cut instead of rounding); then the
    rounding to the output's type (2^-11 for float16, 2^-8 for bfloat16).
"""
import numpy as np
import pytest

import mx_reference as ref
from mx_cases import ANY, PAIRS, SPLIT

pytestmark = pytest.mark.gpu

GUARD = 4096
TYPES = ("float32", "float16", "bfloat16")


def _torch():
    import torch
    return torch


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def _dtype(name):
    return getattr(_torch(), name)


def _dev(a, name="float32"):
    """numpy values on the GPU in a type, and the float64 values they have there."""
    t = _torch().from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_dtype(name))
    return t, t.double().cpu().numpy()


def _guarded(n, dtype, fill):
    buf = _torch().full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
    return buf, buf[GUARD:GUARD + n]


def _guards_ok(buf, n, fill):
    b = buf.cpu()
    return bool((b[:GUARD] == fill).all()) and bool((b[GUARD + n:] == fill).all())


def _mx_out(rows, K, bits):
    """A guarded MxTensor and a check that nothing outside it was written."""
    q, torch = _q(), _torch()
    Kp = ref.padded(K)
    nc, ns = rows * Kp * bits // 8, -(-rows // 128) * (Kp // 128) * 512
    cb, c = _guarded(nc, torch.uint8, 0xA5)
    sb, s = _guarded(ns, torch.uint8, 0xA5)
    out = q.MxTensor(c.view(rows, -1), s.view(-1, Kp // 128, 512), K, bits)
    return out, lambda: _guards_ok(cb, nc, 0xA5) and _guards_ok(sb, ns, 0xA5)


def _host(mx):
    """Unpacked codes [rows, Kp], scale bytes [rows, Kp/32], and the raw tiles."""
    t = mx.scales.cpu().numpy()
    return ref.unpack(mx.codes.cpu().numpy(), mx.bits), ref.untile(t, mx.rows), t


def _assert_padding(mx):
    """Codes past K and scale bytes of padding rows and blocks are zero."""
    codes, byte, tiles = _host(mx)
    assert not codes[:, mx.K:].any()
    assert not byte[:, -(-mx.K // 32):].any()
    assert np.array_equal(tiles, ref.tile(byte))


def _rng(*seed):
    return np.random.default_rng([7, *seed])


def _values(g, rows, K):
    """Rows of mixed sizes, with zeros, ties and one far larger value."""
    v = g.standard_normal((rows, K)) * np.exp(2 * g.standard_normal((rows, 1)))
    v[:, ::7] = 0
    v[:, 1::11] = np.round(v[:, 1::11] * 4) / 4
    v.reshape(-1)[g.integers(0, v.size)] = 3000
    return v


SHAPES = [(1, 1), (1, 31), (1, 32), (2, 33), (3, 100), (5, 128), (1, 129), (7, 1000), (33, 256), (127, 384),
          (128, 40), (129, 520), (260, 72)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,K", SHAPES + [(2, 65536)])
def test_quantize_and_back(rows, K, bits, name):
    q, torch = _q(), _torch()
    x, v = _dev(_values(_rng(rows, K), rows, K), name)
    out, untouched = _mx_out(rows, K, bits)
    assert q.mx_quantize(x, bits=bits, out=out) is out
    codes, byte = ref.quantize(v, bits)
    got, got_byte, _ = _host(out)
    assert np.array_equal(got_byte, byte)
    assert np.array_equal(got, codes)
    _assert_padding(out)
    assert untouched()
    want = ref.values(codes, byte, bits)[:, :K]
    assert np.array_equal(q.mx_dequantize(out).cpu().numpy().astype(np.float64), want)
    y = q.mx_dequantize(out, dtype=x.dtype)
    assert y.dtype == x.dtype
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(torch.float32).to(x.dtype))


@pytest.mark.parametrize("bits", [4, 8])
def test_quantize_extremes(bits):
    q, torch = _q(), _torch()
    v = np.zeros((8, 160), np.float32)
    v[0, :40] = np.linspace(-1, 1, 40) * np.float32(3.4028235e38)   # the largest floats
    v[1, :40] = np.linspace(1, 2, 40) * np.float32(2.0 ** -126)     # the smallest normal ones
    v[2, :40] = np.arange(40) * np.float32(2.0 ** -149)             # subnormals
    v[3, 5], v[3, 40], v[3, 70] = np.inf, -np.inf, np.nan           # three bad blocks, two good ones
    v[3, 100], v[3, 130] = 1, -2
    v[4, :] = -0.0
    v[5, ::2], v[5, 1::2] = 7.99, 2.0 ** -20                        # cut at the largest code, and lost to zero
    v[6, 0], v[6, 1:32] = 448, 464                                  # the largest E4M3 code and its tie
    out = q.mx_quantize(torch.from_numpy(v).cuda(), bits=bits)
    codes, byte = ref.quantize(v.astype(np.float64), bits)
    got, got_byte, _ = _host(out)
    assert np.array_equal(got_byte, byte) and np.array_equal(got, codes)
    assert got_byte[3, 0] == got_byte[3, 1] == got_byte[3, 2] == 255
    back = q.mx_dequantize(out).cpu().numpy()
    assert np.isnan(back[3, :96]).all() and np.isfinite(back[3, 96:]).all()


def test_every_code_dequantizes():
    q, torch = _q(), _torch()
    for bits in (4, 8):
        codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
        if bits == 4:
            codes = codes & 15
        byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)   # every scale byte
        mx = q.MxTensor(torch.from_numpy(ref.pack(codes, bits)).cuda(), torch.from_numpy(ref.tile(byte)).cuda(), 256,
                        bits)
        with np.errstate(over="ignore", invalid="ignore"):
            want = ref.values(codes, byte, bits).astype(np.float32)
        assert np.array_equal(q.mx_dequantize(mx).cpu().numpy(), want, equal_nan=True)


def _strided(a, name, how):
    """The same rows inside a wider tensor: (view, float64 values)."""
    torch = _torch()
    rows, K = a.shape
    if how == "aligned":        # 16-byte rows inside wider ones
        wide = torch.full((rows, K + 64), 7.0, dtype=_dtype(name), device="cuda")
        view = wide[:, 32:32 + K]
    elif how == "odd":          # nothing aligned but the elements
        wide = torch.full((rows, K + 13), 7.0, dtype=_dtype(name), device="cuda")
        view = wide[:, 5:5 + K]
    else:                       # every other row
        wide = torch.full((2 * rows, K), 7.0, dtype=_dtype(name), device="cuda")
        view = wide[::2]
    view.copy_(torch.from_numpy(a.astype(np.float32)).cuda())
    return view, view.double().cpu().numpy()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("how", ["aligned", "odd", "skipped"])
def test_quantize_strided_rows(how, name):
    q = _q()
    x, v = _strided(_values(_rng(3), 37, 168), name, how)
    got, got_byte, _ = _host(q.mx_quantize(x, bits=8))
    codes, byte = ref.quantize(v, 8)
    assert np.array_equal(got, codes) and np.array_equal(got_byte, byte)


@pytest.mark.parametrize("how", ["aligned", "odd", "skipped"])
def test_dequantize_into_strided_rows(how):
    q, torch = _q(), _torch()
    x, v = _dev(_values(_rng(4), 37, 168))
    mx = q.mx_quantize(x, bits=4)
    view, _ = _strided(np.zeros((37, 168)), "float32", how)
    q.mx_dequantize(mx, out=view)
    codes, byte = ref.quantize(v, 4)
    assert np.array_equal(view.double().cpu().numpy(), ref.values(codes, byte, 4)[:, :168])
    base = view._base.cpu()
    if how != "skipped":
        left = view.storage_offset()
        assert bool((base[:, :left] == 7).all()) and bool((base[:, left + 168:] == 7).all())
    else:
        assert bool((base[1::2] == 7).all())


def test_leading_dimensions():
    q, torch = _q(), _torch()
    x = torch.randn(2, 3, 64, device="cuda")
    a, b = q.mx_quantize(x), q.mx_quantize(x.view(6, 64))
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    one = q.mx_quantize(x[0, 0])
    assert one.rows == 1 and torch.equal(one.codes, a.codes[:1])
    with pytest.raises(ValueError):
        q.mx_quantize(x.transpose(0, 1))     # rows that are not evenly spaced are not copied silently
    with pytest.raises(ValueError):
        q.mx_quantize(x[0].t())


def _assert_rounds(mx, v, slack):
    """mx is a quantisation of values within `slack` of v."""
    bits = mx.bits
    codes, byte, _ = _host(mx)
    lo, hi = np.abs(v) - slack, np.abs(v) + slack
    least, most = ref.scale_bytes(np.maximum(lo, 0), bits), ref.scale_bytes(hi, bits)
    assert ((least <= byte) & (byte <= most)).all()
    val = ref.code_values(bits)
    got = val[codes][:, :v.shape[1]]
    a = val[ref.codes_under(v - slack, byte, bits)][:, :v.shape[1]]
    b = val[ref.codes_under(v + slack, byte, bits)][:, :v.shape[1]]
    assert ((a <= got) & (got <= b)).all()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,K", SHAPES + [(3, 8192), (2, 11008), (2, 32769), (1, 65536), (2, 16384)])
def test_rmsnorm(rows, K, bits, name):
    q, torch = _q(), _torch()
    g = _rng(rows, K, 1)
    x, xv = _dev(_values(g, rows, K), name)
    r, rv = _dev(4 * g.standard_normal((rows, K)), name)
    w, wv = _dev(1 + 0.3 * g.standard_normal(K), name)
    out, untouched = _mx_out(rows, K, bits)
    hb, h = _guarded(rows * K, x.dtype, 3.0)
    got, gh = q.mx_rmsnorm(x, w, eps=1e-5, residual=r, bits=bits, out=out, h_out=h.view(rows, K))
    v, hv = ref.rmsnorm(xv, wv, float(np.float32(1e-5)), rv)
    _assert_rounds(got, v, 3e-6 * np.abs(v))
    _assert_padding(got)
    # h is the fp32 sum rounded once more to its type (float32: once in all).
    want = (x.float() + r.float()).to(x.dtype)
    assert torch.equal(gh, want)
    assert untouched() and _guards_ok(hb, rows * K, 3.0)


@pytest.mark.parametrize("name,wname", [("bfloat16", "float32"), ("float16", "float32"), ("float32", "float32")])
def test_rmsnorm_without_residual_and_with_float32_weight(name, wname):
    q = _q()
    g = _rng(9)
    x, xv = _strided(_values(g, 70, 488), name, "odd")
    w, wv = _dev(g.standard_normal(488), wname)
    got = q.mx_rmsnorm(x, w, eps=1e-3)
    v, _ = ref.rmsnorm(xv, wv, float(np.float32(1e-3)))
    _assert_rounds(got, v, 3e-6 * np.abs(v))


@pytest.mark.parametrize("K", [1000, 40000])     # kept in registers, and read twice
@pytest.mark.parametrize("which", ["x", "residual"])
def test_rmsnorm_in_place(which, K):
    q, torch = _q(), _torch()
    x, r, w = (torch.randn(9, K, device="cuda") for _ in range(3))
    want, wh = q.mx_rmsnorm(x, w[0], residual=r)
    target = x if which == "x" else r
    got, gh = q.mx_rmsnorm(x, w[0], residual=r, h_out=target)
    assert gh is target and torch.equal(gh, wh)
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)


def test_rmsnorm_of_zeros_and_bad_rows():
    q, torch = _q(), _torch()
    x = torch.randn(5, 256, device="cuda")
    x[1] = 0
    x[2, 40], x[3, 3] = float("nan"), float("inf")
    w = torch.ones(256, device="cuda")
    clean = q.mx_rmsnorm(torch.nan_to_num(x, 0.0, 0.0), w)
    codes, byte, _ = _host(q.mx_rmsnorm(x, w))
    cc, cb, _ = _host(clean)
    assert not codes[1].any() and not byte[1].any()
    assert (byte[2] == 255).all()                   # the sum is NaN: every value of the row is
    assert byte[3, 0] == 255 and not (codes[3, 32:] & 0x7F).any()   # inf · 0, and the others over infinity
    for i in (0, 4):
        assert np.array_equal(codes[i], cc[i]) and np.array_equal(byte[i], cb[i])


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("rows,K", SHAPES)
def test_swiglu(rows, K, bits, name):
    q, torch = _q(), _torch()
    g = _rng(rows, K, 2)
    both = np.concatenate([3 * g.standard_normal((rows, K)), _values(g, rows, K)], axis=1)
    both[0, 0] = -100.0
    t, v = _dev(both, name)
    out, untouched = _mx_out(rows, K, bits)
    got = q.mx_swiglu(t[:, :K], t[:, K:], bits=bits, out=out)      # two halves of one tensor's rows
    want = ref.swiglu(v[:, :K], v[:, K:])
    _assert_rounds(got, want, 1e-6 * np.abs(want) + 1e-36 * np.abs(v[:, K:]))
    _assert_padding(got)
    assert untouched()


def _rows_at(a, name, offset, gap):
    """Rows that start `offset` elements past a 512-byte boundary, `gap` elements between them, NaN all around."""
    torch = _torch()
    rows, K = a.shape
    n = rows * (K + gap) - gap
    buf = torch.full((GUARD + n + GUARD,), float("nan"), dtype=_dtype(name), device="cuda")
    view = buf[GUARD + offset:][:n + gap].as_strided((rows, K), (K + gap, 1))
    view.copy_(torch.from_numpy(a.astype(np.float32)).cuda())

    def surroundings_ok():
        b = buf.clone()
        b[GUARD + offset:][:n + gap].as_strided((rows, K), (K + gap, 1)).fill_(float("nan"))
        return bool(b.isnan().all())

    return view, view.double().cpu().numpy(), surroundings_ok


# Rows that end before, on and past a granule of 16 bytes, a scale block, a warp's 256 values; one, two and three rows
# (no neighbours, one, two) and enough for several 128-row blocks.
PLACES = [(3, 1, 0), (3, 5, 0), (1, 9, 0), (2, 17, 1), (140, 23, 0), (70, 31, 2), (131, 33, 5), (3, 255, 0), (3, 257, 0),
          (257, 260, 0), (5, 516, 3), (6, 1119, 0)]


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("offset", range(8))
@pytest.mark.parametrize("rows,K,gap", PLACES)
def test_rows_that_start_anywhere(rows, K, gap, offset, name):
    q, torch = _q(), _torch()
    g = _rng(rows, K, offset, 5)
    a, b = _values(g, rows, K), 4 * g.standard_normal((rows, K))
    x, xv, _ = _rows_at(a, name, offset, gap)
    r, rv, _ = _rows_at(b, name, (3 * offset + 1) % 8, gap + 1)
    bits = 4 if offset & 1 else 8

    mx = q.mx_quantize(x, bits=bits)
    codes, byte = ref.quantize(xv, bits)
    got, got_byte, _ = _host(mx)
    assert np.array_equal(got_byte, byte) and np.array_equal(got, codes)
    _assert_padding(mx)

    y, _, clean = _rows_at(np.zeros((rows, K)), name, offset, gap)
    q.mx_dequantize(mx, out=y)
    want = torch.from_numpy(ref.values(codes, byte, bits)[:, :K]).to(torch.float32).to(x.dtype)
    assert torch.equal(y.cpu(), want) and clean()

    v = ref.swiglu(rv, xv)
    mx = q.mx_swiglu(r, x, bits=bits)
    _assert_rounds(mx, v, 1e-6 * np.abs(v) + 1e-36 * np.abs(xv))
    _assert_padding(mx)

    w, wv, _ = _rows_at(1 + 0.3 * g.standard_normal((1, K)), "float32" if offset & 2 else name, (5 * offset) % 8, 0)
    h, _, clean = _rows_at(np.zeros((rows, K)), name, (offset + 3) % 8, gap)
    mx, _ = q.mx_rmsnorm(x, w[0], eps=1e-5, residual=r, bits=bits, h_out=h)
    v, _ = ref.rmsnorm(xv, wv[0], float(np.float32(1e-5)), rv)
    _assert_rounds(mx, v, 3e-6 * np.abs(v))
    _assert_padding(mx)
    assert torch.equal(h, (x.float() + r.float()).to(x.dtype)) and clean()


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("K", [1001, 4095, 9001, 40001])     # one, two and four groups a thread, and read twice
def test_rmsnorm_of_many_unaligned_rows(K, name):
    q, torch = _q(), _torch()
    g = _rng(K, 6)
    rows = 180
    x, xv = _dev(_values(g, rows, K), name)
    r, rv = _dev(4 * g.standard_normal((rows, K)), name)
    w, wv = _dev(1 + 0.3 * g.standard_normal(K), name)
    mx, h = q.mx_rmsnorm(x, w, eps=1e-5, residual=r, h_out=torch.empty_like(x))
    v, _ = ref.rmsnorm(xv, wv, float(np.float32(1e-5)), rv)
    _assert_rounds(mx, v, 3e-6 * np.abs(v))
    _assert_padding(mx)
    assert torch.equal(h, (x.float() + r.float()).to(x.dtype))


# Products.

def _random_mx(g, rows, K, bits, spread=6):
    """Random codes (no NaN) and scale bytes; returns the MxTensor and its values."""
    q, torch = _q(), _torch()
    Kp = ref.padded(K)
    codes = g.integers(0, 16 if bits == 4 else 256, (rows, Kp)).astype(np.uint8)
    if bits == 8:
        codes[(codes & 0x7F) == 0x7F] = 0
    codes[:, K:] = 0
    byte = g.integers(127 - spread, 127 + spread, (rows, Kp // 32)).astype(np.uint8)
    byte[:, -(-K // 32):] = 0
    mx = q.MxTensor(torch.from_numpy(ref.pack(codes, bits)).cuda(), torch.from_numpy(ref.tile(byte)).cuda(), K, bits)
    return mx, ref.values(codes, byte, bits)


ROUND = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def _assert_product(y, xv, wv, name):
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = (xv.shape[1] // 32 + 1) * 2.0 ** -23 * size + ROUND[name] * np.abs(want) + (
        2.0 ** -24 if name == "float16" else 0)
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", ANY + SPLIT + PAIRS)
def test_matmul(T, K, N, bits):
    q, torch = _q(), _torch()
    g = _rng(T, K, N, bits)
    x, xv = _random_mx(g, T, K, bits)
    w, wv = _random_mx(g, N, K, 4)
    buf, out = _guarded(T * N, torch.float32, -5.0)
    out.fill_(float("nan"))
    y = q.mx_matmul(x, w, out=out.view(T, N))
    torch.cuda.synchronize()
    q.device_status()
    _assert_product(y, xv, wv, "float32")
    assert _guards_ok(buf, T * N, -5.0)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(20, 2560, 700), (64, 4096, 601), (250, 4224, 520), (60, 1000, 7100), (420, 640, 4901),
                                   (1200, 300, 2050)])
def test_matmul_rounds_its_sums_to_16_bits(T, K, N, bits):
    q, torch = _q(), _torch()
    g = _rng(T, K, N, bits, 2)
    x, _ = _random_mx(g, T, K, bits, spread=2)
    w, _ = _random_mx(g, N, K, 4, spread=2)
    y = q.mx_matmul(x, w)
    for name in ("float16", "bfloat16"):
        buf, out = _guarded(T * N, _dtype(name), -5.0)
        assert torch.equal(q.mx_matmul(x, w, out=out.view(T, N)), y.to(_dtype(name)))
        assert _guards_ok(buf, T * N, -5.0)


@pytest.mark.parametrize("name", ["float16", "bfloat16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(1, 512, 300), (5, 1000, 129), (40, 256, 255), (130, 384, 131), (300, 640, 260)])
def test_matmul_16_bit_outputs(T, K, N, bits, name):
    q, torch = _q(), _torch()
    g = _rng(T, K, N, bits, 1)
    x, xv = _random_mx(g, T, K, bits, spread=2)
    w, wv = _random_mx(g, N, K, 4, spread=2)
    if bits == 8:      # keep float16 in range
        x = q.MxTensor(x.codes, x.scales - (x.scales > 0).byte() * 8, K, bits)
        xv = xv / 256
    buf, out = _guarded(T * N, _dtype(name), -5.0)
    y = q.mx_matmul(x, w, out=out.view(T, N))
    _assert_product(y, xv, wv, name)
    assert _guards_ok(buf, T * N, -5.0)


def test_matmul_wide_rows_and_many_outputs():
    q = _q()
    g = _rng(21)
    for T, K, N, bits in ((2, 65536, 130, 8), (2, 65536, 130, 4), (1, 256, 20000, 8), (4, 384, 30000, 4)):
        x, xv = _random_mx(g, T, K, bits)
        w, wv = _random_mx(g, N, K, 4)
        _assert_product(q.mx_matmul(x, w), xv, wv, "float32")
    q.device_status()


@pytest.mark.parametrize("bits", [4, 8])
def test_matmul_extreme_scales(bits):
    # Scales up to 2^60 against 2^-60, and a row whose blocks differ by 2^40.
    q, torch = _q(), _torch()
    g = _rng(22, bits)
    x, xv = _random_mx(g, 3, 512, bits, spread=20)
    w, wv = _random_mx(g, 200, 512, 4, spread=20)
    up = q.MxTensor(x.codes, x.scales + (x.scales > 0).byte() * 60, 512, bits)
    down = q.MxTensor(w.codes, w.scales - (w.scales > 0).byte() * 60, 512, 4)
    _assert_product(q.mx_matmul(up, down), xv, wv, "float32")


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T", [1, 20, 140])
def test_matmul_nan_scale_stays_in_its_row(T, bits):
    q, torch = _q(), _torch()
    g = _rng(23, T, bits)
    x, xv = _random_mx(g, T, 640, bits)
    w, wv = _random_mx(g, 300, 640, 4)
    clean = q.mx_matmul(x, w)
    xs, ws = ref.untile(x.scales.cpu().numpy(), T), ref.untile(w.scales.cpu().numpy(), 300)
    xs[T // 2, 3], ws[130, 19] = 255, 255
    x2 = q.MxTensor(x.codes, torch.from_numpy(ref.tile(xs)).cuda(), 640, bits)
    w2 = q.MxTensor(w.codes, torch.from_numpy(ref.tile(ws)).cuda(), 640, 4)
    y = q.mx_matmul(x2, w2)
    assert bool(torch.isnan(y[T // 2]).all()) and bool(torch.isnan(y[:, 130]).all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[T // 2], keep[:, 130] = False, False
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(1, 4096, 520), (40, 2048, 300), (600, 1024, 700), (1500, 1024, 5000)])
def test_matmul_gives_the_same_bits_again(T, K, N, bits):
    q, torch = _q(), _torch()
    g = _rng(24, T)
    x, _ = _random_mx(g, T, K, bits)
    w, _ = _random_mx(g, N, K, 4)
    first = q.mx_matmul(x, w)
    for _ in range(20):
        assert torch.equal(q.mx_matmul(x, w), first)


def test_a_token_does_not_depend_on_its_batch():
    # Each row of a batch has the sum of its own call up to the order of the
    # additions, so a row's error bound holds whatever rows go with it.
    q, torch = _q(), _torch()
    g = _rng(25)
    x, xv = _random_mx(g, 300, 1024, 8)
    w, wv = _random_mx(g, 256, 1024, 4)
    _assert_product(q.mx_matmul(x, w), xv, wv, "float32")
    byte = ref.untile(x.scales.cpu().numpy(), 300)
    for t in (0, 137, 299):
        one = q.MxTensor(x.codes[t:t + 1], torch.from_numpy(ref.tile(byte[t:t + 1])).cuda(), 1024, 8)
        _assert_product(q.mx_matmul(one, w), xv[t:t + 1], wv, "float32")


def test_no_rows():
    q, torch = _q(), _torch()
    x = torch.empty(0, 96, device="cuda")
    mx = q.mx_quantize(x)
    assert mx.rows == 0 and mx.codes.shape == (0, 128) and mx.scales.numel() == 0
    assert q.mx_dequantize(mx).shape == (0, 96)
    assert q.mx_swiglu(x, x).rows == 0
    n, h = q.mx_rmsnorm(x, torch.ones(96, device="cuda"), residual=x)
    assert n.rows == 0 and h.shape == (0, 96)
    w = q.mx_quantize(torch.randn(40, 96, device="cuda"), bits=4)
    assert q.mx_matmul(mx, w).shape == (0, 40)


def test_chain_on_a_stream_of_its_own():
    # Quantised weights and activations come from kernels just before the
    # product on the same stream; nothing synchronises in between.
    q, torch = _q(), _torch()
    s = torch.cuda.Stream()
    g = _rng(26)
    a, b = (torch.from_numpy(g.standard_normal((n, 2048)).astype(np.float32)).cuda() for n in (24, 640))
    want = None
    torch.cuda.synchronize()
    for i in range(10):
        with torch.cuda.stream(s):
            x, w = q.mx_quantize(a * (i + 1)), q.mx_quantize(b, bits=4)
            y = q.mx_matmul(x, w)
            z = q.mx_matmul(q.mx_quantize(y, bits=4), q.mx_quantize(y, bits=4))
        s.synchronize()
        if i == 0:
            xv, wv = (q.mx_dequantize(t).double().cpu().numpy() for t in (x, w))
            _assert_product(y, xv, wv, "float32")
            v = q.mx_dequantize(q.mx_quantize(y, bits=4)).double().cpu().numpy()
            _assert_product(z, v, v, "float32")
            want = y.clone()
        if i == 1:
            assert torch.equal(y, 2 * want)
    # A stream given by hand, with the tensors of another.
    y2 = q.mx_matmul(q.mx_quantize(a, stream=s), q.mx_quantize(b, bits=4, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(y2, want)


def test_in_a_cuda_graph():
    q, torch = _q(), _torch()
    x = torch.randn(33, 1024, device="cuda")
    w = q.mx_quantize(torch.randn(500, 1024, device="cuda"), bits=4)
    g = torch.randn(1024, device="cuda")

    def step():
        n, h = q.mx_rmsnorm(x, g, residual=x)
        y = q.mx_matmul(n, w)
        return q.mx_swiglu(y, y, bits=4), h
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, h = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(33, 1024, device="cuda"))
        graph.replay()
        want, wh = step()
        assert torch.equal(out.codes, want.codes) and torch.equal(out.scales, want.scales) and torch.equal(h, wh)


# Refusals of the Python calls on GPU tensors.

def test_refusals():
    q, torch = _q(), _torch()
    x = torch.zeros(4, 128, device="cuda")
    m8, m4 = q.mx_quantize(x), q.mx_quantize(x, bits=4)
    w = torch.ones(128, device="cuda")
    bad = [lambda: q.mx_quantize(x.int()), lambda: q.mx_quantize(x.double()), lambda: q.mx_quantize(x, bits=6),
           lambda: q.mx_quantize(x, out=m4), lambda: q.mx_quantize(x[:2], out=m8), lambda: q.mx_quantize(x.t()[::2]),
           lambda: q.mx_quantize(torch.tensor(1.0, device="cuda")), lambda: q.mx_swiglu(x, x[:3]),
           lambda: q.mx_swiglu(x, x.half()), lambda: q.mx_rmsnorm(x, w[:64]), lambda: q.mx_rmsnorm(x, w, residual=x[:2]),
           lambda: q.mx_rmsnorm(x, w, residual=x.half()), lambda: q.mx_rmsnorm(x, w, h_out=x),
           lambda: q.mx_rmsnorm(x, w.cpu()), lambda: q.mx_matmul(m8, m8), lambda: q.mx_matmul(m4, q.mx_quantize(x[:, :64], 4)),
           lambda: q.mx_matmul(m8, m4, out=torch.empty(4, 5, device="cuda")),
           lambda: q.mx_matmul(m8, m4, dtype=torch.float64),
           lambda: q.mx_matmul(m8._replace(scales=m8.scales[:, :0]), m4),
           lambda: q.mx_matmul(m8._replace(codes=m8.codes[:, :64]), m4),
           lambda: q.mx_dequantize(m8._replace(bits=4)), lambda: q.mx_dequantize(m8, dtype=torch.int32)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    with pytest.raises(q.Q4mmError):       # float16 input, bfloat16 weight
        q.mx_rmsnorm(x.half(), w.bfloat16())
    with pytest.raises(q.Q4mmError):
        q.mx_rmsnorm(x, w, eps=-1.0)
    with pytest.raises(q.Q4mmError):       # y over x's codes
        big = torch.zeros(4 * 128, dtype=torch.uint8, device="cuda")
        q.mx_matmul(m8._replace(codes=big.view(4, 128)), m4, out=big[:64].view(torch.float32).view(4, 4))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,N", [(1, 4096, 512), (24, 4096, 300), (100, 4096, 300), (300, 4096, 300),
                                   (200, 4096, 10000)])
def test_wait_runs_out_then_next_call_is_right(T, K, N, bits):
    # One stage of weights never arrives and waits last a millisecond: the
    # kernel reports it and leaves the context usable.
    q, torch = _q(), _torch()
    g = _rng(27, T, bits)
    x, xv = _random_mx(g, T, K, bits)
    w, wv = _random_mx(g, N, K, 4)
    torch.cuda.synchronize()
    q.device_status()
    q.arm_wait_failure(0, 2_000_000)
    q.mx_matmul(x, w)
    torch.cuda.synchronize()
    with pytest.raises(q.Q4mmError) as e:
        q.device_status()
    assert e.value.code == -5
    q.device_status()
    _assert_product(q.mx_matmul(x, w), xv, wv, "float32")
    q.device_status()


@pytest.mark.parametrize("tokens", [1, 30, 260])
def test_feed_forward_example(tokens):
    """The example's block against the same block on the values that its codes
    stand for: each product is within its own bound of those, and the whole
    differs from float32 on unquantised values by the formats' error only."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "llama_ffn_mx.py")
    spec = importlib.util.spec_from_file_location("llama_ffn_mx", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    torch = _torch()
    weights, x, residual = ex.make(768, 1100, tokens, seed=tokens)
    block = ex.MxFeedForward(**weights)
    y, h = block(x, residual)
    ref = ex.reference(x, residual, **weights)
    assert torch.equal(h, x + residual)
    # A 4-bit weight is off by up to a quarter of its value and by about a
    # ninth on the mean, in three matrices one after the other.
    off = float((y.float() - ref).norm() / ref.norm())
    assert 0.02 < off < 0.35
    _q().device_status()
