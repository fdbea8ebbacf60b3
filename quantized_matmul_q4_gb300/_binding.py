"""ctypes binding of libq4mm.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple

PKG = os.path.dirname(os.path.abspath(__file__))
Q4K_VALUES = 256
Q4K_BYTES = 144

_SYMBOLS = ("q4k_matmul", "q4k_matmul_tc", "q4k_matmul_tc_noalloc", "q4k_relayout_tc", "q4k_matmul_tc_relayouted",
            "q4_0_gemv", "q6k_gemv", "q4k_ffn_swiglu", "ternary_gemv",
            "mx_quantize", "mx_swiglu", "mx_rmsnorm", "mx_dequantize", "mx_matmul",
            "rope_rotate", "mx_cache_write", "mx_cache_read", "mx_attention", "mx_attention_workspace",
            "q4mm_call",
            "q4mm_last_error", "q4mm_device_status", "q4mm_version", "q4mm_test_fail_next_wait",
            "q4mm_test_attention_kernel")


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
    heads, cache, batch = [vp, i64, i64], [vp, vp, vp, vp, i32, i32, i32, i32, i32], [vp, vp, vp, i32, i32]
    lib.rope_rotate.argtypes = [*heads, i32, vp, i32, vp, i32, i32, f32, *heads, i32, i32, i32, vp]
    lib.mx_cache_write.argtypes = [*heads, *heads, i32, vp, i32, i32, f32, *cache, *batch, i32, vp]
    lib.mx_cache_read.argtypes = [*cache, *batch, *heads, *heads, i32, i32, vp]
    lib.mx_attention.argtypes = [*heads, i32, *cache, *batch, f32, i32, *heads, i32, i32, vp, ctypes.c_size_t, vp]
    lib.mx_attention_workspace.argtypes = [i32] * 7
    lib.mx_attention_workspace.restype = ctypes.c_size_t
    lib.q4mm_call.argtypes = [i32, ctypes.c_char_p]
    lib.q4mm_call.restype = i32
    for name in ("mx_quantize", "mx_swiglu", "mx_rmsnorm", "mx_dequantize", "mx_matmul", "rope_rotate",
                 "mx_cache_write", "mx_cache_read", "mx_attention"):
        getattr(lib, name).restype = i32
    lib.q4mm_last_error.argtypes = []
    lib.q4mm_last_error.restype = ctypes.c_char_p
    lib.q4mm_device_status.argtypes = [vp, i32]
    lib.q4mm_device_status.restype = i32
    lib.q4mm_version.argtypes = []
    lib.q4mm_version.restype = i32
    lib.q4mm_test_fail_next_wait.argtypes = [i32, ctypes.c_longlong]
    lib.q4mm_test_fail_next_wait.restype = i32
    lib.q4mm_test_attention_kernel.argtypes = [i32]
    lib.q4mm_test_attention_kernel.restype = i32
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


# (x, k, v, q, out, y: pointer, token stride, head stride; cache: the pointers of k's codes and scales and of v's, then
# pages, kvHeads, pageTokens, headDim, bits; batch: the pointers starts, lengths, table, then sequences, tableWidth.)

def rope_rotate_ptr(x, dtype: int, positions: int, positions_64: int, frequencies: int, rotated: int, interleaved: int,
                    magnitude: float, out, tokens: int, heads: int, head_dim: int, stream: int = 0) -> None:
    _check(_LIB.rope_rotate(*x, dtype, positions, positions_64, frequencies, rotated, interleaved, magnitude, *out,
                            tokens, heads, head_dim, stream))


def mx_cache_write_ptr(k, v, dtype: int, frequencies: int, rotated: int, interleaved: int, magnitude: float, cache,
                       batch, tokens: int, stream: int = 0) -> None:
    _check(_LIB.mx_cache_write(*k, *v, dtype, frequencies, rotated, interleaved, magnitude, *cache, *batch, tokens,
                               stream))


def mx_cache_read_ptr(cache, batch, k, v, dtype: int, tokens: int, stream: int = 0) -> None:
    _check(_LIB.mx_cache_read(*cache, *batch, *k, *v, dtype, tokens, stream))


def mx_attention_ptr(q, dtype: int, cache, batch, scale: float, causal: int, y, tokens: int, heads: int,
                     workspace: int = 0, workspace_bytes: int = 0, stream: int = 0) -> None:
    _check(_LIB.mx_attention(*q, dtype, *cache, *batch, scale, causal, *y, tokens, heads, workspace, workspace_bytes,
                             stream))


def arm_wait_failure(stage: int, limit_cycles: int) -> None:
    """Test hook: the calling thread's next call withholds weight stage `stage`
    and bounds its in-kernel waits by `limit_cycles` (see include/q4mm.h)."""
    _check(_LIB.q4mm_test_fail_next_wait(int(stage), int(limit_cycles)))


def force_attention_kernel(which: str | None) -> None:
    """Test hook: the calling thread's mx_attention takes the kernel for "few"
    rows, or for "many", until None leaves the choice to the library."""
    _check(_LIB.q4mm_test_attention_kernel((None, "few", "many").index(which)))


def device_status(stream=None, clear: bool = True) -> None:
    """Raise Q4mmError if a bounded in-kernel wait ran out on this device, or
    a call met a page number or a position outside its cache or table."""
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
    uint8 = float32 = int32 = int64 = float64 = empty = raw_stream = current_device = None

    @classmethod
    def load(cls):
        import torch
        # (Whoever finds the dtypes, or uint8, set finds these set.)
        cls.int32, cls.int64, cls.float64 = torch.int32, torch.int64, torch.float64
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


# Attention on a paged MX cache: layouts, limits and precision in include/q4mm.h.

# The words of q4mm_call, which takes its arguments in a buffer: one by one they
# cost ctypes 2.5 us, more than the launch.
_ROPE_WORDS = struct.Struct("=9qd7q").pack
_WRITE_WORDS = struct.Struct("=10qd16q").pack
_READ_WORDS = struct.Struct("=23q").pack
_ATTENTION_WORDS = struct.Struct("=18qd9q").pack
_ROPE, _WRITE, _READ, _ATTENTION = range(4)     # Q4MM_CALL_...


class Rope(NamedTuple):
    """Rotary positions of a head's first 2·len(frequencies) values.

    frequencies: float64 CUDA tensor, radians per position of each pair
    interleaved: pairs (2i, 2i + 1); else (i, i + len(frequencies))
    magnitude:   factor of the rotated values
    """
    frequencies: "torch.Tensor"
    interleaved: bool = False
    magnitude: float = 1.0


def rope_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int | None = None, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """Frequencies base^(-2i/dim) of a head's dim / 2 pairs, stretched for a
    context `factor` times the `original` one by `scaling`:
      None      not at all
      "linear"  every frequency divided by factor
      "ntk"     base multiplied by factor^(dim / (dim - 2)): the slowest pair
                is divided by factor, the fastest left
      "parts"   by the turns r that a pair makes in the original context:
                divided by factor below `slow` of them, left above `fast`, in
                between mixed linearly (rope_magnitude goes with it)
    """
    import torch
    if dim <= 0 or dim % 2:
        raise ValueError("dim must be positive and even")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "ntk", "parts"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'parts'")
    if scaling == "ntk":
        if dim < 4:
            raise ValueError("'ntk' needs at least two pairs")
        base *= factor ** (dim / (dim - 2))
    f = torch.tensor([base ** (-2 * i / dim) for i in range(dim // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original is None or not original > 0 or not fast > slow:
            raise ValueError("'parts' needs the original context, and fast above slow")
        kept = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * kept + f / factor * (1 - kept)
    return f.to(device)


def rope_magnitude(factor: float) -> float:
    """The magnitude that goes with "parts": 0.1·ln(factor) + 1 for a stretched context."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


class MxCache(NamedTuple):
    """Keys and values of pages of tokens, quantised in MX blocks along the head.

    k_codes, v_codes:   uint8 [pages, kv heads, page, head_dim·bits/8]
    k_scales, v_scales: uint8 [pages, kv heads, page, 4]

    A batch of sequences in it is three int32 CUDA tensors that every call
    takes: starts [sequences + 1], lengths [sequences] and pages [sequences,
    width].  Rows starts[i] .. starts[i + 1] of a call's tensors are the last of
    the lengths[i] tokens that sequence i has in the cache; its position p is
    place p % page of page pages[i, p // page].  Their contents are read on
    the device: see device_status for those that lie outside the cache.
    """
    k_codes: "torch.Tensor"
    k_scales: "torch.Tensor"
    v_codes: "torch.Tensor"
    v_scales: "torch.Tensor"
    head_dim: int
    bits: int


def mx_cache(pages: int, kv_heads: int, head_dim: int, page: int = 64, bits: int = 8, device="cuda") -> MxCache:
    """An empty cache."""
    import torch
    if head_dim not in (32, 64, 96, 128) or bits not in (4, 8) or page <= 0 or page % 16:
        raise ValueError("head_dim must be 32, 64, 96 or 128, bits 4 or 8, and page a multiple of 16")
    if pages <= 0 or kv_heads <= 0:
        raise ValueError("pages and kv_heads must be positive")
    def side():
        return (torch.zeros(pages, kv_heads, page, head_dim * bits // 8, dtype=torch.uint8, device=device),
                torch.zeros(pages, kv_heads, page, 4, dtype=torch.uint8, device=device))
    return MxCache(*side(), *side(), head_dim, bits)


def _heads_arg(x, what: str, shape=None):
    """A [tokens, heads, head_dim] CUDA tensor: the C ABI's three arguments."""
    got = x.shape
    if len(got) != 3 or (shape is not None and got != shape):
        raise ValueError(f"{what} must be [tokens, heads, head_dim]" + (f" = {list(shape)}" if shape is not None else ""))
    s0, s1, s2 = x.stride()
    if s2 != 1 and got[2] > 1:
        raise ValueError(f"the values of a head of {what} must be adjacent")
    return x.data_ptr(), s0, s1


def _cache_arg(c: MxCache, device: int):
    kc, ks, vc, vs, D, bits = c
    u8 = _Torch.uint8
    if u8 is None:
        _Torch.load()
        u8 = _Torch.uint8
    shape = kc.shape
    if len(shape) != 4 or (bits != 8 and bits != 4) or shape[3] * 8 != D * bits:
        raise ValueError("cache: codes must be [pages, kv heads, page, head_dim·bits/8]")
    pages, heads, page, _ = shape
    if vc.shape != shape or ks.shape != (pages, heads, page, 4) or vs.shape != ks.shape:
        raise ValueError("cache: scales must be [pages, kv heads, page, 4], and v's tensors like k's")
    for t in (kc, ks, vc, vs):
        if t.dtype != u8 or not t.is_contiguous():
            raise ValueError("cache: codes and scales must be contiguous uint8 tensors")
        if t.get_device() != device:
            raise ValueError("all tensors of a call must be on one CUDA device")
    return kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, heads, page, D, bits


def _batch_arg(starts, lengths, pages, device: int):
    i32 = _Torch.int32
    for t in (starts, lengths, pages):
        if t.dtype != i32 or not t.is_contiguous():
            raise ValueError("starts, lengths and pages must be contiguous int32 tensors")
        if t.get_device() != device:
            raise ValueError("all tensors of a call must be on one CUDA device")
    if lengths.dim() != 1 or pages.dim() != 2 or starts.dim() != 1:
        raise ValueError("starts and lengths must have one dimension, pages two")
    n = lengths.shape[0]
    if starts.shape[0] != n + 1 or pages.shape[0] != n:
        raise ValueError("starts must be [sequences + 1], lengths [sequences] and pages [sequences, width]")
    return starts.data_ptr(), lengths.data_ptr(), pages.data_ptr(), n, pages.shape[1]


_NO_ROPE = (0, 0, 0, 1.0)


def _rope_arg(rope: Rope, head_dim: int, device: int):
    f, interleaved, magnitude = rope
    if _Torch.float64 is None:
        _Torch.load()
    if f.dtype != _Torch.float64 or f.dim() != 1 or not f.is_contiguous():
        raise ValueError("frequencies must be a contiguous float64 tensor of one dimension")
    if f.get_device() != device:
        raise ValueError("all tensors of a call must be on one CUDA device")
    n = 2 * f.shape[0]
    if n > head_dim:
        raise ValueError("there are more frequencies than pairs in a head")
    return f.data_ptr(), n, 1 if interleaved else 0, float(magnitude)


def _cuda_device(x, what: str) -> int:
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{what} must be a CUDA tensor")
    return device


def rope_rotate(x, positions, rope: Rope, out=None, stream=None):
    """x [tokens, heads, head_dim] (float32, float16 or bfloat16) with its
    rotary positions (int32 or int64, one per token); out may be x itself."""
    device = _cuda_device(x, "x")
    dtype = _mx_dtype(x.dtype, "x")
    xa = _heads_arg(x, "x")
    T, H, D = shape = x.shape
    if positions.dim() != 1 or positions.shape[0] != T or not positions.is_contiguous() or \
            positions.dtype not in (_Torch.int32, _Torch.int64):
        raise ValueError("positions must be a contiguous int32 or int64 tensor with one value per token")
    _mx_device(device, positions)
    ra = _rope_arg(rope, D, device)
    at, side = _call_stream(stream, device)
    if out is None:
        new = _Torch.empty if side is None else _empty_on(side)
        out = new(shape, dtype=x.dtype, device=x.device)
    elif out.dtype != x.dtype:
        raise ValueError("out must have x's type")
    else:
        _mx_device(device, out)
    oa = _heads_arg(out, "out", shape)
    if side is not None:
        _hold(side, x, positions, rope.frequencies, out)
    rc = _LIB.q4mm_call(_ROPE, _ROPE_WORDS(*xa, dtype, positions.data_ptr(), positions.dtype == _Torch.int64, *ra, *oa, T, H,
                                           D, at))
    if rc:
        _check(rc)
    return out


def mx_cache_write(cache: MxCache, k, v, starts, lengths, pages, rope: Rope | None = None, stream=None) -> MxCache:
    """k (turned by rope, where it is given, at its positions) and v
    [tokens, kv heads, head_dim] of a batch's new tokens into the cache."""
    device = _cuda_device(k, "k")
    dtype = _mx_dtype(k.dtype, "k")
    if v.dtype != k.dtype:
        raise ValueError("k and v must have the same type")
    _mx_device(device, v)
    ca = _cache_arg(cache, device)
    ba = _batch_arg(starts, lengths, pages, device)
    T = k.shape[0]
    shape = (T, ca[5], ca[7])
    ka, va = _heads_arg(k, "k", shape), _heads_arg(v, "v", shape)
    ra = _NO_ROPE if rope is None else _rope_arg(rope, ca[7], device)
    at, side = _call_stream(stream, device)
    if side is not None:
        _hold(side, k, v, *cache[:4], starts, lengths, pages, rope and rope[0])
    rc = _LIB.q4mm_call(_WRITE, _WRITE_WORDS(*ka, *va, dtype, *ra, *ca, *ba, T, at))
    if rc:
        _check(rc)
    return cache


def mx_cache_read(cache: MxCache, starts, lengths, pages, tokens: int | None = None, dtype=None, out=None, stream=None):
    """The values (k, v), each [tokens, kv heads, head_dim], of a batch's rows
    (float32 unless dtype or out = (k, v) says otherwise).  Rows that are not in
    the cache, and those behind the last sequence, are left as they were (without
    `out`: as the allocator gave them)."""
    device = _cuda_device(cache[0], "cache")
    ca = _cache_arg(cache, device)
    ba = _batch_arg(starts, lengths, pages, device)
    at, side = _call_stream(stream, device)
    if out is None:
        if tokens is None or tokens < 0:
            raise ValueError("tokens must say how many rows the result has")
        shape = (tokens, ca[5], ca[7])
        new = _Torch.empty if side is None else _empty_on(side)
        dtype = dtype or _Torch.float32
        k, v = new(shape, dtype=dtype, device=cache[0].device), new(shape, dtype=dtype, device=cache[0].device)
    else:
        k, v = out
        shape = (k.shape[0] if tokens is None else tokens, ca[5], ca[7])
        if k.dtype != v.dtype or (dtype is not None and k.dtype != dtype):
            raise ValueError("k and v must have the same, and the given, type")
        _mx_device(device, k), _mx_device(device, v)
    ka, va = _heads_arg(k, "k", shape), _heads_arg(v, "v", shape)
    if side is not None:
        _hold(side, *cache[:4], starts, lengths, pages, k, v)
    rc = _LIB.q4mm_call(_READ, _READ_WORDS(*ca, *ba, *ka, *va, _mx_dtype(k.dtype, "out"), shape[0], at))
    if rc:
        _check(rc)
    return k, v


def mx_attention(q, cache: MxCache, starts, lengths, pages, scale: float | None = None, causal: bool = True, out=None,
                 stream=None):
    """softmax(scale·q·kᵀ)·v of a batch's queries [tokens, heads, head_dim]
    over their sequences' cached tokens (causal: up to their own), heads a
    multiple of the cache's; scale is head_dim^-1/2 unless given.  A row that
    sees nothing gives zeros; rows behind the last sequence are left as they were
    (without `out`: as the allocator gave them)."""
    device = _cuda_device(q, "q")
    dtype = _mx_dtype(q.dtype, "q")
    ca = _cache_arg(cache, device)
    ba = _batch_arg(starts, lengths, pages, device)
    qa = _heads_arg(q, "q")
    T, H, D = shape = q.shape
    if D != ca[7] or H == 0 or ca[5] == 0 or H % ca[5]:
        raise ValueError("q must have the cache's head_dim, and a multiple of its heads")
    at, side = _call_stream(stream, device)
    if out is None:
        new = _Torch.empty if side is None else _empty_on(side)
        out = new(shape, dtype=q.dtype, device=q.device)
    elif out.dtype != q.dtype:
        raise ValueError("out must have q's type")
    else:
        _mx_device(device, out)
    oa = _heads_arg(out, "out", shape)
    # Few rows over a long cache: sums of its parts meet in a workspace.  (The
    # library has the rule; it is asked only where there may be one.)
    ws, nbytes, kv = None, 0, ca[5]
    if (T * (H // kv) // 8 + ba[3]) * kv < 64:
        nbytes = _LIB.mx_attention_workspace(kv, ca[6], D, ba[3], ba[4], T, H)
        if nbytes:
            new = _Torch.empty if side is None else _empty_on(side)
            ws = new((nbytes,), dtype=_Torch.uint8, device=q.device)
    if side is not None:
        _hold(side, q, *cache[:4], starts, lengths, pages, out, ws)
    rc = _LIB.q4mm_call(_ATTENTION, _ATTENTION_WORDS(*qa, dtype, *ca, *ba, D ** -0.5 if scale is None else float(scale),
                                                     1 if causal else 0, *oa, T, H, 0 if ws is None else ws.data_ptr(),
                                                     nbytes, at))
    if rc:
        _check(rc)
    return out
