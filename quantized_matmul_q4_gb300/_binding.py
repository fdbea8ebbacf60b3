"""ctypes binding of libq4mm.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import math
import os
from typing import NamedTuple

PKG = os.path.dirname(os.path.abspath(__file__))
Q4K_VALUES = 256
Q4K_BYTES = 144

_SYMBOLS = ("q4k_matmul", "q4k_matmul_tc", "q4k_matmul_tc_noalloc", "q4k_relayout_tc", "q4k_matmul_tc_relayouted",
            "q4_0_gemv", "q6k_gemv", "q4k_ffn_swiglu", "ternary_gemv",
            "mx_quantize", "mx_swiglu", "mx_rmsnorm", "mx_dequantize", "mx_matmul",
            "q4mm_last_error", "q4mm_device_status", "q4mm_version", "q4mm_test_fail_next_wait")


class Q4mmError(RuntimeError):
    """A q4mm entry point returned a negative status."""

    def __init__(self, code: int, message: str):
        super().__init__(f"q4mm status {code}: {message}")
        self.code = code


def library_path() -> str:
    return os.environ.get("Q4MM_LIB", os.path.join(PKG, "libq4mm.so"))


def _load() -> ctypes.CDLL:
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"libq4mm.so not found at {path}: build it with `python quantized_matmul_q4_gb300/_build.py` "
            "(needs nvcc); there is no fallback implementation")
    lib = ctypes.CDLL(path)
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    for name in ("q4k_matmul", "q4k_matmul_tc", "q4k_matmul_tc_noalloc", "q4k_matmul_tc_relayouted", "q4_0_gemv",
                 "q6k_gemv"):
        fn = getattr(lib, name)
        fn.argtypes = [vp, vp, vp, i32, i32, i32, vp]
        fn.restype = i32
    lib.q4k_relayout_tc.argtypes = [vp, vp, i32, i32, vp]
    lib.q4k_relayout_tc.restype = i32
    lib.q4k_ffn_swiglu.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
    lib.q4k_ffn_swiglu.restype = i32
    lib.ternary_gemv.argtypes = [vp, vp, f32, vp, i32, i32, i32, vp]
    lib.ternary_gemv.restype = i32
    i64 = ctypes.c_longlong
    lib.mx_quantize.argtypes = [vp, i64, i32, vp, vp, i32, i32, i32, vp]
    lib.mx_swiglu.argtypes = [vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, vp]
    lib.mx_rmsnorm.argtypes = [vp, i64, vp, i64, vp, i64, i32, vp, i32, f32, vp, vp, i32, i32, i32, vp]
    lib.mx_dequantize.argtypes = [vp, vp, vp, i64, i32, i32, i32, i32, vp]
    lib.mx_matmul.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, vp]
    for name in ("mx_quantize", "mx_swiglu", "mx_rmsnorm", "mx_dequantize", "mx_matmul"):
        getattr(lib, name).restype = i32
    lib.q4mm_last_error.argtypes = []
    lib.q4mm_last_error.restype = ctypes.c_char_p
    lib.q4mm_device_status.argtypes = [vp, i32]
    lib.q4mm_device_status.restype = i32
    lib.q4mm_version.argtypes = []
    lib.q4mm_version.restype = i32
    lib.q4mm_test_fail_next_wait.argtypes = [i32, ctypes.c_longlong]
    lib.q4mm_test_fail_next_wait.restype = i32
    return lib


_LIB = _load()


def library() -> ctypes.CDLL:
    return _LIB


def last_error() -> str:
    return _LIB.q4mm_last_error().decode()


def version() -> int:
    return _LIB.q4mm_version()


def _check(rc: int) -> None:
    if rc != 0:
        raise Q4mmError(rc, last_error())


def _stream_ptr(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


# Raw-pointer entry points (device pointers, sizes, stream handle).

def q4k_matmul_ptr(x: int, w: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q4k_matmul(x, w, y, K, N, T, stream))


def q4k_matmul_tc_ptr(x: int, w: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q4k_matmul_tc(x, w, y, K, N, T, stream))


def q4k_matmul_tc_noalloc_ptr(x: int, w: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q4k_matmul_tc_noalloc(x, w, y, K, N, T, stream))


def q4k_relayout_tc_ptr(w: int, w_tc: int, K: int, N: int, stream: int = 0) -> None:
    _check(_LIB.q4k_relayout_tc(w, w_tc, K, N, stream))


def q4k_matmul_tc_relayouted_ptr(x: int, w_tc: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q4k_matmul_tc_relayouted(x, w_tc, y, K, N, T, stream))


def q4_0_gemv_ptr(x: int, w: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q4_0_gemv(x, w, y, K, N, T, stream))


def q6k_gemv_ptr(x: int, w: int, y: int, K: int, N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.q6k_gemv(x, w, y, K, N, T, stream))


def q4k_ffn_swiglu_ptr(x: int, w_gate: int, w_up: int, h: int, K: int, N: int, T: int,
                       stream: int = 0) -> None:
    _check(_LIB.q4k_ffn_swiglu(x, w_gate, w_up, h, K, N, T, stream))


def ternary_gemv_ptr(x: int, w: int, scale: float, y: int, K: int, N: int, T: int,
                     stream: int = 0) -> None:
    _check(_LIB.ternary_gemv(x, w, ctypes.c_float(scale), y, K, N, T, stream))


# (dtype: 0 float32, 1 float16, 2 bfloat16; strides in elements.)

def mx_quantize_ptr(x: int, x_stride: int, dtype: int, codes: int, scales: int, K: int, rows: int, bits: int,
                    stream: int = 0) -> None:
    _check(_LIB.mx_quantize(x, x_stride, dtype, codes, scales, K, rows, bits, stream))


def mx_swiglu_ptr(gate: int, gate_stride: int, up: int, up_stride: int, dtype: int, codes: int, scales: int, K: int,
                  rows: int, bits: int, stream: int = 0) -> None:
    _check(_LIB.mx_swiglu(gate, gate_stride, up, up_stride, dtype, codes, scales, K, rows, bits, stream))


def mx_rmsnorm_ptr(x: int, x_stride: int, residual: int, residual_stride: int, h: int, h_stride: int, dtype: int,
                   weight: int, weight_dtype: int, eps: float, codes: int, scales: int, K: int, rows: int, bits: int,
                   stream: int = 0) -> None:
    _check(_LIB.mx_rmsnorm(x, x_stride, residual, residual_stride, h, h_stride, dtype, weight, weight_dtype, eps,
                           codes, scales, K, rows, bits, stream))


def mx_dequantize_ptr(codes: int, scales: int, y: int, y_stride: int, dtype: int, K: int, rows: int, bits: int,
                      stream: int = 0) -> None:
    _check(_LIB.mx_dequantize(codes, scales, y, y_stride, dtype, K, rows, bits, stream))


def mx_matmul_ptr(x_codes: int, x_scales: int, x_bits: int, w_codes: int, w_scales: int, y: int, dtype: int, K: int,
                  N: int, T: int, stream: int = 0) -> None:
    _check(_LIB.mx_matmul(x_codes, x_scales, x_bits, w_codes, w_scales, y, dtype, K, N, T, stream))


def arm_wait_failure(stage: int, limit_cycles: int) -> None:
    """Test hook: the calling thread's next call withholds weight stage `stage`
    and bounds its in-kernel waits by `limit_cycles` (see include/q4mm.h)."""
    _check(_LIB.q4mm_test_fail_next_wait(int(stage), int(limit_cycles)))


def device_status(stream=None, clear: bool = True) -> None:
    """Raise Q4mmError if a bounded in-kernel wait ran out on this device."""
    _check(_LIB.q4mm_device_status(_stream_ptr(stream), int(clear)))


# Tensor entry points (torch CUDA tensors; y allocated unless `out` is given).
#
# stream: a torch stream or a stream's handle; the current stream unless given.
# On another stream than the current one nothing waits: the tensors have to be
# ready there, and a user of the results waits for that stream.  Memory is
# safe, though: results come from the pool of the call's stream, and neither
# they nor the tensors given are reused before both streams are past them,
# however early they are dropped.  (A stream given by its handle has to live
# as long as that memory.)

class _Torch:
    """What the calls take from torch, looked up on the first of them (the
    binding itself imports without torch).  A call costs the host about as
    much as an elementwise torch operation, mostly its allocations and the
    launch; what is left is kept short."""
    dtypes: dict = {}
    uint8 = float32 = empty = raw_stream = current_device = None

    @classmethod
    def load(cls):
        import torch
        cls.dtypes = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # q4mm_dtype
        cls.uint8, cls.float32, cls.empty = torch.uint8, torch.float32, torch.empty
        cls.current_device = torch._C._cuda_getDevice
        # The current stream's handle alone: a Stream object costs as much as a launch.
        # Last: who finds it set (every call looks, in _call_stream) finds the others set too.
        cls.raw_stream = torch._C._cuda_getCurrentRawStream


def _call_stream(stream, device: int):
    """The handle of a call's stream, and the stream where it is not the
    current one (else None).  The library launches on the current device, so
    tensors and stream have to be that device's."""
    if _Torch.raw_stream is None:
        _Torch.load()
    if device != _Torch.current_device():
        raise ValueError(f"the tensors are on device {device}, the current device is {_Torch.current_device()}: "
                         "call under torch.cuda.device(...) of the tensors")
    current = _Torch.raw_stream(device)
    if stream is None:
        return current, None
    handle = _stream_ptr(stream)
    if handle == current:
        return current, None
    if not hasattr(stream, "record_event"):
        import torch
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    elif stream.device.index != device:
        raise ValueError("the stream must be of the tensors' device")
    return handle, stream


def _empty_on(side):
    """torch.empty from the pool of the stream `side`, for a call that runs there (None: the current one)."""
    if side is None:
        return _Torch.empty

    def empty(shape, dtype, device):
        import torch
        with torch.cuda.stream(side):
            t = torch.empty(shape, dtype=dtype, device=device)
        t.record_stream(torch.cuda.current_stream(device))   # whose code has it from now on
        return t

    return empty


def _hold(side, *tensors) -> None:
    """Memory of the tensors is not reused before `side` is past the call."""
    for t in tensors:
        if t is not None:
            t.record_stream(side)


def _prep(x, w, K, bytes_per_row, out, N, stream, w2=None):
    import torch
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    if w.dtype != torch.uint8 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("the packed weight must be a contiguous uint8 CUDA tensor")
    device = x.get_device()
    if any(t is not None and t.get_device() != device for t in (w, w2, out)):
        raise ValueError("all tensors of a call must be on one CUDA device")
    x2 = x.reshape(-1, x.shape[-1])
    T, K_ = x2.shape
    if K is not None and K != K_:
        raise ValueError("x's last dimension must equal inputDim")
    if N is None:
        if bytes_per_row(K_) <= 0 or w.numel() % bytes_per_row(K_):
            raise ValueError("weight size is not a whole number of rows")
        N = w.numel() // bytes_per_row(K_)
    if out is not None and (out.dtype != torch.float32 or not out.is_cuda or not out.is_contiguous()
                            or out.numel() != T * N):
        raise ValueError("out must be a contiguous float32 CUDA tensor with tokens·outputDim elements")
    handle, side = _call_stream(stream, device)
    if out is None:
        out = _empty_on(side)((T, N), dtype=torch.float32, device=x.device)
    if side is not None:
        _hold(side, x, w, w2, out)
    return x2, T, K_, N, out, handle


def q4k_matmul(x, w, N: int | None = None, out=None, stream=None):
    """y[T, N] = x[T, K] · dequant(W)ᵀ in FP32 (decode GEMV up to 8 tokens)."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: (k // Q4K_VALUES) * Q4K_BYTES, out, N, stream)
    q4k_matmul_ptr(x2.data_ptr(), w.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


def q4k_matmul_tc(x, w, N: int | None = None, out=None, stream=None):
    """As q4k_matmul on the tensor cores with bf16-rounded operands."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: (k // Q4K_VALUES) * Q4K_BYTES, out, N, stream)
    q4k_matmul_tc_ptr(x2.data_ptr(), w.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


def q4k_matmul_tc_noalloc(x, w, N: int | None = None, out=None, stream=None):
    """As q4k_matmul_tc with its scratch in the library's fixed device array
    (no allocation; calls that overlap on the GPU race on that array)."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: (k // Q4K_VALUES) * Q4K_BYTES, out, N, stream)
    q4k_matmul_tc_noalloc_ptr(x2.data_ptr(), w.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


TC_CHUNK_BYTES = 48  # relayouted bytes per row and 64 values
TC_TILE_ROWS = 256   # rows per tile of the relayouted layout


def tc_relayout_bytes(K: int, N: int) -> int:
    """Size of a relayouted K -> N weight (rows rounded up to whole tiles)."""
    return -(-N // TC_TILE_ROWS) * TC_TILE_ROWS * (K // 64) * TC_CHUNK_BYTES


def q4k_relayout_tc(w, K: int, N: int | None = None, out=None, stream=None):
    """The one-time relayout of a canonical Q4_K weight for
    q4k_matmul_tc_relayouted: a uint8 CUDA tensor of tc_relayout_bytes(K, N)
    bytes (tile-major, zero rows padding the last 256-row tile)."""
    import torch
    if w.dtype != torch.uint8 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("the packed weight must be a contiguous uint8 CUDA tensor")
    row = (K // Q4K_VALUES) * Q4K_BYTES
    if N is None:
        if row <= 0 or w.numel() % row:
            raise ValueError("weight size is not a whole number of rows")
        N = w.numel() // row
    nbytes = tc_relayout_bytes(K, N)
    if out is not None and (out.dtype != torch.uint8 or not out.is_cuda or not out.is_contiguous()
                            or out.numel() != nbytes):
        raise ValueError("out must be a contiguous uint8 CUDA tensor of tc_relayout_bytes(K, N) bytes")
    if out is not None and out.get_device() != w.get_device():
        raise ValueError("all tensors of a call must be on one CUDA device")
    at, side = _call_stream(stream, w.get_device())
    if out is None:
        out = _empty_on(side)(nbytes, dtype=torch.uint8, device=w.device)
    if side is not None:
        _hold(side, w, out)
    q4k_relayout_tc_ptr(w.data_ptr(), out.data_ptr(), K, N, at)
    return out


def q4k_matmul_tc_relayouted(x, w_tc, N: int, out=None, stream=None):
    """q4k_matmul_tc on a weight relayouted by q4k_relayout_tc (N is
    required: the padded layout does not give it)."""
    if w_tc.numel() != tc_relayout_bytes(x.shape[-1], N):
        raise ValueError("w_tc size does not match tc_relayout_bytes(K, N)")
    x2, T, K, N, out, at = _prep(x, w_tc, None, lambda k: (k // 64) * TC_CHUNK_BYTES, out, N, stream)
    q4k_matmul_tc_relayouted_ptr(x2.data_ptr(), w_tc.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


Q40_VALUES, Q40_BYTES = 32, 18


def q4_0_gemv(x, w, N: int | None = None, out=None, stream=None):
    """y[T, N] = x[T, K] · dequant_q4_0(W)ᵀ in FP32 (up to 8 tokens per weight pass)."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: (k // Q40_VALUES) * Q40_BYTES, out, N, stream)
    q4_0_gemv_ptr(x2.data_ptr(), w.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


Q6K_BYTES = 210


def q6k_gemv(x, w, N: int | None = None, out=None, stream=None):
    """y[T, N] = x[T, K] · dequant_q6k(W)ᵀ in FP32 (up to 8 tokens per weight pass)."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: (k // Q4K_VALUES) * Q6K_BYTES, out, N, stream)
    q6k_gemv_ptr(x2.data_ptr(), w.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


def q4k_ffn_swiglu(x, w_gate, w_up, N: int | None = None, out=None, stream=None):
    """h[T, N] = silu(x · dequant(W_gate)ᵀ) · (x · dequant(W_up)ᵀ), both Q4_K."""
    if (w_up.dtype != w_gate.dtype or w_up.numel() != w_gate.numel() or not w_up.is_cuda
            or not w_up.is_contiguous()):
        raise ValueError("w_up must be a contiguous CUDA uint8 tensor of the gate weight's size")
    x2, T, K, N, out, at = _prep(x, w_gate, None, lambda k: (k // Q4K_VALUES) * Q4K_BYTES, out, N, stream, w_up)
    q4k_ffn_swiglu_ptr(x2.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


def ternary_gemv(x, w, scale: float = 1.0, N: int | None = None, out=None, stream=None):
    """y[T, N] = scale · x[T, K] · codes(W)ᵀ, BitNet b1.58 payload, FP32."""
    x2, T, K, N, out, at = _prep(x, w, None, lambda k: k // 4, out, N, stream)
    ternary_gemv_ptr(x2.data_ptr(), w.data_ptr(), float(scale), out.data_ptr(), K, N, T, at)
    return out.view(T, N)


# Microscaled (MX) tensors: layouts and roundings in include/q4mm.h.

MX_BLOCK, MX_TILE_ROWS, MX_TILE_BYTES = 32, 128, 512
MX_MAX_ROWS = 0x7FFFFE00   # rows of a call (Q4MM_MX_MAX_ROWS)


class MxTensor(NamedTuple):
    """`rows` vectors of K values in MX blocks of 32.

    codes:  uint8 [rows, Kp·bits/8], Kp = K rounded up to a multiple of 128
            (E2M1, two to a byte, for 4 bits; E4M3 for 8)
    scales: uint8 [ceil(rows/128), Kp/128, 512], E8M0 bytes in tiles of 128
            rows x 4 blocks
    """
    codes: "torch.Tensor"
    scales: "torch.Tensor"
    K: int
    bits: int

    @property
    def rows(self) -> int:
        return self.codes.shape[0]


def mx_padded(K: int) -> int:
    return -(-K // 128) * 128


def _mx_dtype(t, what: str) -> int:
    if not _Torch.dtypes:
        _Torch.load()
    code = _Torch.dtypes.get(t)
    if code is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16")
    return code


def _mx_rows(x, what: str):
    """x as a CUDA matrix of rows with adjacent values, never copied: the
    matrix, its shape, its row stride and its device."""
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    shape = x.shape
    if len(shape) != 2:
        if not shape:
            raise ValueError(f"{what} must have at least one dimension")
        try:
            # (No row count can be inferred from nothing: 2 x 0 x 96 is no rows, 2 x 3 x 0 six empty ones.)
            x = x.view(-1, shape[-1]) if x.numel() else x.reshape(math.prod(shape[:-1]), shape[-1])
        except RuntimeError:
            raise ValueError(f"the leading dimensions of {what} must collapse into evenly spaced rows") from None
        shape = x.shape
    rows, K = shape
    if rows > MX_MAX_ROWS or K > MX_MAX_ROWS:
        raise ValueError(f"{what} has more rows or columns than a call takes")
    s0, s1 = x.stride()
    if s1 != 1 and K > 1:
        raise ValueError(f"the values of a row of {what} must be adjacent")
    return x, rows, K, s0 if rows > 1 else K, device


def _mx_out(rows: int, K: int, bits: int, x, device: int, out, side) -> MxTensor:
    """`out` checked, or a new MxTensor on x's device."""
    if bits != 4 and bits != 8:
        raise ValueError("bits must be 4 or 8")
    if out is None:
        kt, where, u8 = -(-K // 128), x.device, _Torch.uint8
        new = _Torch.empty if side is None else _empty_on(side)
        return MxTensor(new((rows, kt * 16 * bits), dtype=u8, device=where),
                        new((-(-rows // MX_TILE_ROWS), kt, MX_TILE_BYTES), dtype=u8, device=where), K, bits)
    if _mx_check(out, "out", device) != rows or out.K != K or out.bits != bits:
        raise ValueError(f"out must hold {rows} rows of {K} values in {bits} bits")
    return out


def _mx_check(q: MxTensor, what: str, device: int) -> int:
    """Checks an MxTensor; returns its rows."""
    codes, scales, K, bits = q
    u8 = _Torch.uint8
    if codes.dtype != u8 or scales.dtype != u8:
        if u8 is None:
            _Torch.load()
            return _mx_check(q, what, device)
        raise ValueError(f"{what}: codes and scales must be uint8 tensors")
    if codes.get_device() != device or scales.get_device() != device or device < 0:
        raise ValueError("all tensors of a call must be on one CUDA device")
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what}: codes and scales must be contiguous")
    shape, kt = codes.shape, -(-K // 128)
    if bits not in (4, 8) or len(shape) != 2 or shape[1] != kt * 16 * bits or K <= 0 or shape[0] > MX_MAX_ROWS:
        raise ValueError(f"{what}: codes must be [rows, padded K·bits/8]")
    if scales.numel() != -(-shape[0] // MX_TILE_ROWS) * kt * MX_TILE_BYTES:
        raise ValueError(f"{what}: scales must hold ceil(rows/128)·(padded K/128) tiles of 512 bytes")
    return shape[0]


def _mx_device(device: int, t) -> None:
    if t.get_device() != device:
        raise ValueError("all tensors of a call must be on one CUDA device")


def mx_quantize(x, bits: int = 8, out: MxTensor | None = None, stream=None) -> MxTensor:
    """x [..., K] (float32, float16 or bfloat16) to an MX tensor of `bits` (4 or 8) bits."""
    x, rows, K, stride, device = _mx_rows(x, "x")
    dtype = _mx_dtype(x.dtype, "x")
    at, side = _call_stream(stream, device)
    out = _mx_out(rows, K, bits, x, device, out, side)
    if side is not None:
        _hold(side, x, out[0], out[1])
    rc = _LIB.mx_quantize(x.data_ptr(), stride, dtype, out[0].data_ptr(), out[1].data_ptr(), K, rows, bits, at)
    if rc:
        _check(rc)
    return out


def mx_swiglu(gate, up, bits: int = 8, out: MxTensor | None = None, stream=None) -> MxTensor:
    """silu(gate)·up as an MX tensor, in one pass."""
    gate, rows, K, gs, device = _mx_rows(gate, "gate")
    up, urows, uK, us, udevice = _mx_rows(up, "up")
    if rows != urows or K != uK or gate.dtype != up.dtype:
        raise ValueError("gate and up must have the same shape and type")
    if device != udevice:
        raise ValueError("all tensors of a call must be on one CUDA device")
    dtype = _mx_dtype(gate.dtype, "gate")
    at, side = _call_stream(stream, device)
    out = _mx_out(rows, K, bits, gate, device, out, side)
    if side is not None:
        _hold(side, gate, up, out[0], out[1])
    rc = _LIB.mx_swiglu(gate.data_ptr(), gs, up.data_ptr(), us, dtype, out[0].data_ptr(), out[1].data_ptr(), K, rows,
                        bits, at)
    if rc:
        _check(rc)
    return out


def mx_rmsnorm(x, weight, eps: float = 1e-5, residual=None, bits: int = 8, out: MxTensor | None = None, h_out=None,
               stream=None):
    """RMS norm of h = x + residual, as an MX tensor.

    With a residual returns (MxTensor, h), h in x's type, written to h_out
    where that is given (which may be x or residual itself); without one
    returns the MxTensor alone.
    """
    shape, xtype = x.shape, x.dtype
    x, rows, K, xs, device = _mx_rows(x, "x")
    dtype = _mx_dtype(xtype, "x")
    if weight.numel() != K or not weight.is_contiguous():
        raise ValueError("weight must be contiguous and hold one value per column of x")
    _mx_device(device, weight)
    at, side = _call_stream(stream, device)
    res_ptr, rs, h_ptr, hs = 0, K, 0, K
    if residual is not None:
        if residual.shape != shape or residual.dtype != xtype:
            raise ValueError("residual must have x's shape and type")
        _mx_device(device, residual)
        r, _, _, rs, _ = _mx_rows(residual, "residual")
        res_ptr = r.data_ptr()
        if h_out is None:
            new = _Torch.empty if side is None else _empty_on(side)
            h = h_out = new(shape, dtype=xtype, device=x.device)
        else:
            if h_out.shape != shape or h_out.dtype != xtype:
                raise ValueError("h_out must have x's shape and type")
            _mx_device(device, h_out)
            h, _, _, hs, _ = _mx_rows(h_out, "h_out")
        h_ptr = h.data_ptr()
    elif h_out is not None:
        raise ValueError("h_out needs a residual: without one h is x")
    out = _mx_out(rows, K, bits, x, device, out, side)
    if side is not None:
        _hold(side, x, weight, residual, h_out, out[0], out[1])
    rc = _LIB.mx_rmsnorm(x.data_ptr(), xs, res_ptr, rs, h_ptr, hs, dtype, weight.data_ptr(),
                         _mx_dtype(weight.dtype, "weight"), float(eps), out[0].data_ptr(), out[1].data_ptr(), K, rows,
                         bits, at)
    if rc:
        _check(rc)
    return out if residual is None else (out, h_out)


def mx_dequantize(q: MxTensor, dtype=None, out=None, stream=None):
    """The values [rows, K] that an MX tensor stands for (float32 unless dtype or out says otherwise)."""
    codes, scales, K, bits = q
    device = codes.get_device()
    rows = _mx_check(q, "q", device)
    at, side = _call_stream(stream, device)
    stride = K
    if out is None:
        new = _Torch.empty if side is None else _empty_on(side)
        out = new((rows, K), dtype=dtype or _Torch.float32, device=codes.device)
    else:
        if out.shape != (rows, K) or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must be [rows, K] of the given type")
        _mx_device(device, out)
        _, _, _, stride, _ = _mx_rows(out, "out")
    if side is not None:
        _hold(side, codes, scales, out)
    rc = _LIB.mx_dequantize(codes.data_ptr(), scales.data_ptr(), out.data_ptr(), stride, _mx_dtype(out.dtype, "out"), K,
                            rows, bits, at)
    if rc:
        _check(rc)
    return out


def mx_matmul(x: MxTensor, w: MxTensor, dtype=None, out=None, stream=None):
    """y[T, N] = x·wᵀ on the tensor cores: x in 4 or 8 bits, w in 4 bits,
    y in float32 unless dtype or out says otherwise."""
    x_codes, x_scales, K, x_bits = x
    w_codes, w_scales, w_K, w_bits = w
    device = x_codes.get_device()
    T, N = _mx_check(x, "x", device), _mx_check(w, "w", device)
    if w_bits != 4:
        raise ValueError("w must be a 4-bit MX tensor")
    if K != w_K:
        raise ValueError("x and w must have the same K")
    at, side = _call_stream(stream, device)
    if out is None:
        new = _Torch.empty if side is None else _empty_on(side)
        out = new((T, N), dtype=dtype or _Torch.float32, device=x_codes.device)
    else:
        if out.shape != (T, N) or not out.is_contiguous() or (dtype is not None and out.dtype != dtype):
            raise ValueError("out must be contiguous, [tokens, outputDim] of the given type")
        _mx_device(device, out)
    if side is not None:
        _hold(side, x_codes, x_scales, w_codes, w_scales, out)
    rc = _LIB.mx_matmul(x_codes.data_ptr(), x_scales.data_ptr(), x_bits, w_codes.data_ptr(), w_scales.data_ptr(),
                        out.data_ptr(), _mx_dtype(out.dtype, "out"), K, N, T, at)
    if rc:
        _check(rc)
    return out
