"""mx_swiglu over the whole range of gates: far below zero, where e^-gate
passes the largest float32, with infinities and NaN, and to the last units
of float32 everywhere.

Tolerance, derived (u = 2^-24, half a unit in the last place).  Down to
gate = -87: e^-gate takes 4 u (the exponential's 2 units) and 1 u (its
correction), 1 + e^-gate one more, the reciprocal 2 u (1 unit), the products
with gate and up 1 u each: 10 u.  Below, gate·e^(gate + 100)·(up·c)·c with
c = e^-50: 4 u for the exponential, 1 u for each of four products and of two
c's: 10 u.  Results below float32's normal range are off by another half of
2^-149, and those past the largest float32 are infinities.
"""
import numpy as np
import pytest

import mx_reference as ref
from test_gpu_mx import TYPES, _assert_padding, _assert_rounds, _dev, _host, _q, _rng, _torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
LARGEST = {"float32": 3.0e38, "float16": 6.0e4, "bfloat16": 3.0e38}


def _slack(v):
    return np.where(np.isinf(v), 0, 10 * U * np.abs(np.where(np.isinf(v), 0, v)) + 2.0 ** -149)


def _float32_range(v):
    return np.where(np.abs(v) > np.finfo(np.float32).max, np.copysign(np.inf, v), v)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lo,hi", [(-91, -86), (-88.8, -87.2), (-130, -87), (-190, -100), (-1000, -86), (-95, 5)])
def test_gates_far_below_zero(lo, hi, bits, name):
    # Every value of a block lies there, so that its scale is that of such results.
    q = _q()
    g = _rng(41, bits, int(-lo))
    rows, K = 9, 200
    gate, gv = _dev(g.uniform(lo, hi, (rows, K)), name)
    size = LARGEST[name] * np.exp2(-g.uniform(0, 1, (rows, K)) * np.linspace(0, 40, rows)[:, None])
    up, uv = _dev(np.copysign(size, g.standard_normal((rows, K))), name)
    mx = q.mx_swiglu(gate, up, bits=bits)
    v = _float32_range(ref.swiglu(gv, uv))
    _assert_rounds(mx, v, _slack(v))
    _assert_padding(mx)


def test_a_block_of_far_gates_keeps_its_values():
    q, torch = _q(), _torch()
    gate = torch.full((1, 32), -88.0, device="cuda")
    back = q.mx_dequantize(q.mx_swiglu(gate, torch.full_like(gate, 1e30)))
    want = -88.0 / (1.0 + np.exp(88.0)) * 1e30      # -5.3e-7
    assert np.abs(back.cpu().numpy() / want - 1).max() < 1 / 16


# Ranges of the gate, and the power of two that the block's largest value is
# 300 times of: such that up stays below the largest float32.
RANGES = [(-170, -150, -119), (-150, -100, -90), (-100, -87, -18), (-88, -86, -18), (-87, -60, 0), (-60, -20, 0),
          (-20, -1, 0), (-1, -0.01, 0), (0.01, 1, 0), (1, 20, 0), (20, 120, 0)]


@pytest.mark.parametrize("lo,hi,power", RANGES)
def test_products_close_to_a_tie_fall_on_their_side(lo, hi, power):
    # up puts the product 11 to 14 u above or below the middle of two codes.
    q = _q()
    g = _rng(42, int(lo + 200))
    rows, K = 64, 1024
    grid = ref.code_values(8)[8:118]                   # normal codes up to 224
    tie = ((grid[1:] + grid[:-1]) / 2)[g.integers(0, len(grid) - 1, (rows, K))]
    gate = g.uniform(lo, hi, (rows, K)).astype(np.float32)
    off = np.where(g.random((rows, K)) < 0.5, -1, 1) * g.uniform(12, 13, (rows, K)) * U
    one = ref.swiglu(gate.astype(np.float64), np.ones((rows, K)))
    up = (tie * (1 + off) * 2.0 ** power / one).astype(np.float32)
    gate[:, ::32], up[:, ::32] = 100, 3 * 2.0 ** power
    assert np.isfinite(up).all() and (np.abs(up) >= 2.0 ** -126).all()
    v = ref.swiglu(gate.astype(np.float64), up.astype(np.float64))
    beside = np.delete(v / tie / 2.0 ** power - 1, np.s_[::32], axis=1)
    assert (np.abs(beside) > 10.5 * U).all()
    mx = q.mx_swiglu(_dev(gate)[0], _dev(up)[0], bits=8)
    codes, byte = ref.quantize(v, 8)
    got, got_byte, _ = _host(mx)
    assert np.array_equal(got_byte, byte) and (byte == 127 + power).all()
    assert np.array_equal(got, codes)


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("bits", [4, 8])
def test_infinities_and_nan(bits, name):
    q, torch = _q(), _torch()
    inf, nan = float("inf"), float("nan")
    low = torch.finfo(getattr(torch, name)).min
    g = _rng(43)
    gate, up = g.standard_normal((12, 96)), g.standard_normal((12, 96))
    bad = [(inf, 1), (-inf, 1), (nan, 1), (1, inf), (1, -inf), (1, nan), (-100, inf), (inf, 0), (-1e4, nan)]
    for i, (a, b) in enumerate(bad):
        gate[i, 40], up[i, 40] = a, b
    gate[9, 40], up[9, 40] = low, -low       # a mask's value: e^gate is zero whatever up is
    gate[10, 32:64], up[10, 32:64] = low, low
    gate[11, 32:64], up[11, 32:64] = -1e4, 1e4
    gt, gv = _dev(gate, name)
    ut, uv = _dev(up, name)
    codes, byte, _ = _host(q.mx_swiglu(gt, ut, bits=bits))
    assert (byte[:9, 1] == 255).all() and not codes[:9, 32:64].any()
    half = (1 << (bits - 1)) - 1
    assert (byte[10:, 1] == 0).all() and not (codes[10:, 32:64] & half).any()
    assert (codes[9, 40] & half) == 0
    with np.errstate(all="ignore"):
        v = ref.swiglu(gv, uv)
    v[:9, 32:64] = 0
    mx = q.mx_swiglu(torch.where(torch.from_numpy(v == 0).cuda(), 0.0, gt.float()).to(gt.dtype), ut.nan_to_num(1, 1, 1),
                     bits=bits)
    clean, clean_byte, _ = _host(mx)
    keep = np.ones(codes.shape, bool)
    keep[:9, 32:64] = keep[10:, 32:64] = keep[:, 96:] = False
    keep[9, 40] = False
    assert np.array_equal(codes[keep], clean[keep]) and np.array_equal(byte[:, [0, 2]], clean_byte[:, [0, 2]])
    v[9, 40] = 0
    _assert_rounds(mx, v, _slack(v))
