"""MX operators without a GPU: the tests' 64-bit restatement against values
worked out by hand, and the refusals of the C ABI and of the Python calls."""
import ctypes

import numpy as np
import pytest

import mx_reference as ref

DIM, NULL, ALIGN, ALIAS = -1, -2, -3, -6
A, B, C, D, E, F = (0x10000000 * i for i in range(1, 7))   # fake device addresses, far apart


@pytest.fixture(scope="module")
def q4mm():
    import quantized_matmul_q4_gb300 as m
    return m


# The restatement.

def test_code_values():
    assert ref.code_values(4)[:8].tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    e4m3 = ref.code_values(8)
    assert e4m3[1] == 2.0 ** -9 and e4m3[8] == 2.0 ** -6 and e4m3[0x38] == 1.0 and e4m3[0x7E] == 448.0
    assert np.isnan(e4m3[0x7F]) and e4m3[0xB8] == -1.0


@pytest.mark.parametrize("u,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6),
                                    (5.0, 6), (5.01, 7), (7.9, 7), (-0.75, 10), (-0.0, 8)])
def test_e2m1_rounds_to_nearest_even(u, code):
    assert ref.nearest_code(np.array([u]), 4)[0] == code


@pytest.mark.parametrize("u,code", [(448.0, 0x7E), (511.0, 0x7E), (2.0 ** -10, 0), (3 * 2.0 ** -10, 2), (17.0, 0x58),
                                    (19.0, 0x5A), (-1.0, 0xB8)])
def test_e4m3_rounds_to_nearest_even(u, code):
    assert ref.nearest_code(np.array([u]), 8)[0] == code


def test_scale_of_a_block():
    v = np.zeros((1, 160))
    v[0, 0], v[0, 40], v[0, 64], v[0, 100] = 7.99, 2.0 ** -140, np.inf, 8.0
    assert ref.scale_bytes(v, 4)[0].tolist() == [127, 0, 255, 128, 0, 0, 0, 0]
    assert ref.scale_bytes(v, 8)[0].tolist() == [121, 0, 255, 122, 0, 0, 0, 0]


def test_tile_places():
    byte = np.arange(130 * 8, dtype=np.int64).reshape(130, 8).astype(np.uint8)
    t = ref.tile(byte)
    assert t.shape == (2, 2, 512)
    assert t[0, 0, 0] == byte[0, 0] and t[0, 1, 3] == byte[0, 7] and t[0, 0, 4] == byte[32, 0]
    assert t[0, 0, 16] == byte[1, 0] and t[0, 0, 511] == byte[127, 3] and t[1, 0, 16] == byte[129, 0]
    assert np.array_equal(ref.untile(t, 130), byte)


# Refusals of the C ABI, before any CUDA call.

def _refused(q4mm, code, fn, *args, word=None):
    with pytest.raises(q4mm.Q4mmError) as e:
        fn(*args)
    assert e.value.code == code, q4mm.last_error()
    if word:
        assert word in q4mm.last_error()


def test_sizes_are_checked(q4mm):
    for K in (0, -32, 65537):
        _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 128, 0, B, C, K, 4, 8, word="inputDim")
        _refused(q4mm, DIM, q4mm.mx_dequantize_ptr, A, B, C, 128, 0, K, 4, 8, word="inputDim")
        _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, 0, K, 16, 1, word="inputDim")
    for bits in (0, 3, 5, 16, -4):
        _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 128, 0, B, C, 128, 4, bits, word="bits")
        _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, bits, C, D, E, 0, 128, 16, 1, word="bits")
    for dtype in (-1, 3):
        _refused(q4mm, DIM, q4mm.mx_swiglu_ptr, A, 128, B, 128, dtype, C, D, 128, 4, 8, word="type")
        _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, dtype, 128, 16, 1, word="type")
    _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, 0, 128, 0, 1, word="outputDim")
    _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, 0, 128, 16, -1, word="tokens")
    _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 128, 0, B, C, 128, -1, 8, word="rows")
    for many in (0x7FFFFE01, 0x7FFFFFFF):      # indexes of the last tiles would not fit
        _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 128, 0, B, C, 128, many, 8, word="rows")
        _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, 0, 128, many, 1, word="outputDim")
        _refused(q4mm, DIM, q4mm.mx_matmul_ptr, A, B, 8, C, D, E, 0, 128, 16, many, word="tokens")
    _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 127, 0, B, C, 128, 2, 8, word="stride")
    _refused(q4mm, DIM, q4mm.mx_quantize_ptr, A, 1 << 62, 0, B, C, 128, 1 << 30, 8, word="memory")
    _refused(q4mm, DIM, q4mm.mx_rmsnorm_ptr, A, 128, 0, 0, 0, 0, 1, B, 2, 1e-5, C, D, 128, 2, 8, word="weight")
    for eps in (-1.0, float("nan")):
        _refused(q4mm, DIM, q4mm.mx_rmsnorm_ptr, A, 128, 0, 0, 0, 0, 0, B, 0, eps, C, D, 128, 2, 8, word="eps")


def test_no_rows_is_nothing_to_do(q4mm):
    # Nothing is looked at or launched, so no pointer is needed (nor a GPU).
    q4mm.mx_quantize_ptr(0, 0, 0, 0, 0, 128, 0, 8)
    q4mm.mx_swiglu_ptr(0, 0, 0, 0, 2, 0, 0, 100, 0, 4)
    q4mm.mx_rmsnorm_ptr(0, 0, 0, 0, 0, 0, 1, 0, 0, 1e-5, 0, 0, 128, 0, 8)
    q4mm.mx_dequantize_ptr(0, 0, 0, 0, 0, 128, 0, 8)
    q4mm.mx_matmul_ptr(0, 0, 8, 0, 0, 0, 0, 128, 16, 0)


def test_null_is_refused(q4mm):
    for args in ((0, B, C), (A, 0, C), (A, B, 0)):
        _refused(q4mm, NULL, q4mm.mx_quantize_ptr, args[0], 128, 0, args[1], args[2], 128, 4, 8)
        _refused(q4mm, NULL, q4mm.mx_dequantize_ptr, *args, 128, 0, 128, 4, 8)
        _refused(q4mm, NULL, q4mm.mx_rmsnorm_ptr, args[0], 128, 0, 0, 0, 0, 0, D, 0, 1e-5, args[1], args[2], 128, 4, 8)
    _refused(q4mm, NULL, q4mm.mx_rmsnorm_ptr, A, 128, 0, 0, 0, 0, 0, 0, 0, 1e-5, B, C, 128, 4, 8)
    _refused(q4mm, NULL, q4mm.mx_swiglu_ptr, A, 128, 0, 128, 0, B, C, 128, 4, 8)
    for i in range(5):
        p = [A, B, C, D, E]
        p[i] = 0
        _refused(q4mm, NULL, q4mm.mx_matmul_ptr, p[0], p[1], 8, p[2], p[3], p[4], 0, 128, 16, 1)


def test_alignment_is_checked(q4mm):
    _refused(q4mm, ALIGN, q4mm.mx_quantize_ptr, A + 2, 128, 0, B, C, 128, 4, 8)       # float32
    _refused(q4mm, ALIGN, q4mm.mx_quantize_ptr, A + 1, 128, 1, B, C, 128, 4, 8)       # float16
    _refused(q4mm, ALIGN, q4mm.mx_quantize_ptr, A, 128, 0, B + 16, C, 128, 4, 8)      # codes
    _refused(q4mm, ALIGN, q4mm.mx_quantize_ptr, A, 128, 0, B, C + 8, 128, 4, 8)       # scales
    _refused(q4mm, ALIGN, q4mm.mx_matmul_ptr, A + 16, B, 8, C, D, E, 0, 128, 16, 1)
    _refused(q4mm, ALIGN, q4mm.mx_matmul_ptr, A, B, 8, C, D + 4, E, 0, 128, 16, 1)
    _refused(q4mm, ALIGN, q4mm.mx_matmul_ptr, A, B, 8, C, D, E + 2, 0, 128, 16, 1)
    _refused(q4mm, ALIGN, q4mm.mx_rmsnorm_ptr, A, 128, 0, 0, B + 1, 128, 2, D, 2, 1e-5, E, F, 128, 4, 8)


def test_overlap_is_refused(q4mm):
    # 4 rows of 128 float32 reach over 2048 bytes, their 8-bit codes over 512.
    _refused(q4mm, ALIAS, q4mm.mx_quantize_ptr, A, 128, 0, A + 2016, C, 128, 4, 8)
    _refused(q4mm, ALIAS, q4mm.mx_quantize_ptr, A, 128, 0, B, B + 496, 128, 4, 8)
    _refused(q4mm, ALIAS, q4mm.mx_dequantize_ptr, A, B, B + 508, 128, 0, 128, 4, 8)
    # y inside the weight's codes (16 rows of 64 bytes).
    _refused(q4mm, ALIAS, q4mm.mx_matmul_ptr, A, B, 8, C, D, C + 1020, 0, 128, 16, 1)
    # h may be x or the residual, not one shifted against the other.
    _refused(q4mm, ALIAS, q4mm.mx_rmsnorm_ptr, A, 128, B, 128, B + 4, 128, 0, C, 0, 1e-5, D, E, 128, 4, 8)
    _refused(q4mm, ALIAS, q4mm.mx_rmsnorm_ptr, A, 128, B, 128, A, 256, 0, C, 0, 1e-5, D, E, 128, 4, 8)
    _refused(q4mm, ALIAS, q4mm.mx_rmsnorm_ptr, A, 128, B, 128, C, 128, 0, C + 64, 0, 1e-5, D, E, 128, 4, 8)


# Refusals of the Python calls (host tensors never reach the library).

def test_python_refuses_host_tensors_and_types(q4mm):
    import torch
    x = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        q4mm.mx_quantize(x)
    with pytest.raises(ValueError):
        q4mm.mx_swiglu(x, x)
    with pytest.raises(ValueError):
        q4mm.mx_rmsnorm(x, torch.ones(128))
    q = q4mm.MxTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8), 128, 8)
    with pytest.raises(ValueError):
        q4mm.mx_dequantize(q)
    with pytest.raises(ValueError):
        q4mm.mx_matmul(q, q)


def test_symbols_take_the_declared_arguments(q4mm):
    lib = q4mm.library()
    for name, n in (("mx_quantize", 9), ("mx_swiglu", 11), ("mx_rmsnorm", 16), ("mx_dequantize", 9),
                    ("mx_matmul", 11)):
        fn = getattr(lib, name)
        assert len(fn.argtypes) == n and fn.restype is ctypes.c_int
