"""Cases, plain forms and 64-bit definitions of the microscaled (MX) operators.

An MX tensor holds `rows` vectors of `K` values in blocks of 32 along K.  A
block has one power-of-two scale, kept as a biased exponent in a byte (E8M0:
byte b stands for 2^(b - 127), 255 for NaN), and 32 small floating-point
codes: E2M1 (4 bits, two per byte, the even value in the low nibble) or E4M3
(8 bits).  K is padded with zeros to `Kp`, a multiple of 128.  Codes are
stored row by row; scales are stored in tiles of 128 rows x 4 blocks, the byte
of (row r, block b) at

    tile (r / 128, b / 4), byte 16 * (r % 32) + 4 * (r % 128 / 32) + b % 4,

with zero bytes for the padding.  Block scale of values v: with amax = max |v|,
2^(floor(log2 amax) - emax), emax = 2 (E2M1) or 8 (E4M3); a code is v / scale
rounded to nearest even and cut at the largest code (6 or 448).  A block that
holds an infinity or a NaN has scale NaN.

Operators (`op` of a case):
  matmul     y[t][n] = sum_k x[t][k] w[n][k], x in 8 or 4 bits, w in 4 bits
  quantize   x -> 8-bit codes and scales (returned as the E4M3 and E8M0 values)
  roundtrip  x -> 4-bit codes and scales -> the values that they stand for
  rmsnorm    h = x + residual; h / sqrt(mean h^2 + eps) * g -> 8-bit, and h
  swiglu     silu(gate) * up -> 8-bit
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EMAX = {4: 2, 8: 8}       # exponent of the largest power of two that a code holds
EMIN = {4: 0, 8: -6}      # exponent below which codes are spaced evenly
MANT = {4: 1, 8: 3}       # mantissa bits
LARGEST = {4: 6.0, 8: 448.0}
EPS = 1e-5


def listed():
    return [
        # Decode: one token through a 4096 x 4096 projection (attention q or o of Llama-2-7B).
        {"name": "matmul_8b_t1_4096x4096", "op": "matmul", "T": 1, "K": 4096, "N": 4096, "bits": 8, "dtype": "f32"},
        # A ragged batch of tokens through the 2560 -> 6912 layer (BitNet b1.58 2B's FFN shape), 4-bit activations.
        {"name": "matmul_4b_t77_2560x6912", "op": "matmul", "T": 77, "K": 2560, "N": 6912, "bits": 4, "dtype": "f32"},
        # A prompt of 1000 tokens through Llama-2-7B's FFN down projection, 8-bit activations.
        {"name": "matmul_8b_t1000_11008x4096", "op": "matmul", "T": 1000, "K": 11008, "N": 4096, "bits": 8,
         "dtype": "bf16"},
        # Many prompts at once through the FFN gate, 4-bit activations: the largest product.
        {"name": "matmul_4b_t8192_4096x11008", "op": "matmul", "T": 8192, "K": 4096, "N": 11008, "bits": 4,
         "dtype": "bf16"},
        # Three decoded tokens' FFN hidden rows on their way to the down projection.
        {"name": "quantize_8b_t3_11008", "op": "quantize", "T": 3, "K": 11008, "bits": 8, "dtype": "f32"},
        # Attention outputs of a large prefill batch on their way to the output projection.
        {"name": "quantize_8b_t8192_4096", "op": "quantize", "T": 8192, "K": 4096, "bits": 8, "dtype": "bf16"},
        # A few odd rows to 4 bits and back: checking one slice of a weight.
        {"name": "roundtrip_4b_r5_1000", "op": "roundtrip", "T": 5, "K": 1000, "bits": 4, "dtype": "f32"},
        # A whole FFN weight to 4 bits and back, as when a checkpoint is converted and its error taken.
        {"name": "roundtrip_4b_r11008_4096", "op": "roundtrip", "T": 11008, "K": 4096, "bits": 4, "dtype": "bf16"},
        # Decode: one token's residual stream into the next layer's projections, in the FP32 stream of this framework.
        {"name": "rmsnorm_8b_t1_4096", "op": "rmsnorm", "T": 1, "K": 4096, "bits": 8, "dtype": "f32"},
        # The same for a large prefill batch with a bf16 stream.
        {"name": "rmsnorm_8b_t8192_4096", "op": "rmsnorm", "T": 8192, "K": 4096, "bits": 8, "dtype": "bf16"},
        # Decode: one token's gate and up products into the down projection.
        {"name": "swiglu_8b_t1_11008", "op": "swiglu", "T": 1, "K": 11008, "bits": 8, "dtype": "f32"},
        # The same for a ragged prefill batch.
        {"name": "swiglu_8b_t4099_11008", "op": "swiglu", "T": 4099, "K": 11008, "bits": 8, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["matmul", "matmul", "matmul", "quantize", "roundtrip", "rmsnorm", "swiglu"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "matmul":
        # Shares of the range: single tokens and small batches, middling ones, prompts.
        T = rng.choice([1, _log_int(rng, 2, 64), _log_int(rng, 2, 64), _log_int(rng, 65, 512), _log_int(rng, 513, 8192)])
        K, N = _log_int(rng, 500, 16384), _log_int(rng, 500, 16384)
        if rng.random() < 0.5:  # model widths are mostly multiples of 128
            K, N = max(512, K // 128 * 128), max(512, N // 128 * 128)
        while T * K * N > 8192 * 4096 * 11008:
            T = T // 2 + 1
        return {"op": op, "T": T, "K": K, "N": N, "bits": rng.choice([4, 8]), "dtype": dtype}
    T, K = _log_int(rng, 1, 11008), _log_int(rng, 500, 16384)
    if rng.random() < 0.5:
        K = max(512, K // 128 * 128)
    while T * K * SIZE[dtype] > 8192 * 4096 * 2:
        T = T // 2 + 1
    return {"op": op, "T": T, "K": K, "bits": 4 if op == "roundtrip" else 8, "dtype": dtype}


def _padded(K):
    return -(-K // 128) * 128


# Plain form: elementary operations in 32 bits.

def _blocks(v):
    """v [rows, K] in float32, padded to blocks of 32: [rows, Kp / 32, 32]."""
    rows, K = v.shape
    v = torch.nn.functional.pad(v, (0, _padded(K) - K))
    return v.view(rows, -1, 32)


def _quantized(v, bits):
    """The code values [rows, Kp] in float32 and the scale bytes [rows, Kp / 32] of v [rows, K]."""
    b = _blocks(v)
    amax = b.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    amax = torch.where(bad, torch.ones_like(amax), amax)
    e = torch.frexp(amax)[1] - 1 - EMAX[bits]
    byte = torch.where(amax > 0, (e + 127).clamp(0, 254), torch.zeros_like(e))
    s = torch.ldexp(b, (127 - byte).unsqueeze(-1))
    step = (torch.frexp(s)[1] - 1).clamp(min=EMIN[bits]) - MANT[bits]
    q = torch.ldexp(torch.round(torch.ldexp(s, -step)), step).clamp(-LARGEST[bits], LARGEST[bits])
    q = torch.where(bad.unsqueeze(-1), torch.zeros_like(q), q)
    byte = torch.where(bad, torch.full_like(byte, 255), byte)
    return q.reshape(v.shape[0], -1), byte.to(torch.uint8)


def _tiled(bytes_):
    """Scale bytes [rows, Kp / 32] in tiles [ceil(rows / 128), Kp / 128, 512]."""
    rows, nb = bytes_.shape
    b = torch.nn.functional.pad(bytes_, (0, 0, 0, -rows % 128)).view(-1, 4, 32, nb // 4, 4)
    return b.permute(0, 3, 2, 1, 4).reshape(-1, nb // 4, 512)


def _untiled(scales, rows):
    """The scale bytes [rows, Kp / 32] of _tiled's layout."""
    nt, nk = scales.shape[:2]
    return scales.view(nt, nk, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(nt * 128, nk * 4)[:rows]


def _packed(q):
    """E2M1 values [rows, Kp] as codes, two to a byte, the even value in the low nibble."""
    a = q.abs()
    mag = (2 * a).where(a < 2, (a + 2).where(a < 4, a / 2 + 4)).to(torch.uint8)
    c = mag | ((q < 0).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _values(codes, bits):
    """Codes as float32 values [rows, Kp]."""
    if bits == 8:
        return codes.view(torch.float8_e4m3fn).float()
    c = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).int()
    e, m = (c >> 1) & 3, (c & 1).float()
    v = torch.where(e > 0, torch.ldexp(1 + 0.5 * m, e - 1), 0.5 * m)
    return torch.where(c >= 8, -v, v)


def _scale(bytes_):
    """Scale bytes as float32."""
    s = torch.ldexp(torch.ones_like(bytes_, dtype=torch.float32), bytes_.int() - 127)
    return torch.where(bytes_ == 255, torch.full_like(s, float("nan")), s)


def _dequantized(codes, scales, bits):
    v = _values(codes, bits)
    s = _scale(_untiled(scales, codes.shape[0]))
    return (v.view(v.shape[0], -1, 32) * s.unsqueeze(-1)).view(v.shape)


# Inputs.

def _stream(g, T, K, dtype):
    """Activations: rows of normal values whose channels differ in size, a few of them much larger."""
    size = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
    size = torch.where(torch.rand(K, generator=g, device="cuda") < 0.004, 30 * size, size)
    return (torch.randn(T, K, generator=g, device="cuda") * size).to(DTYPES[dtype])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T, K, bits, dtype = case["T"], case["K"], case["bits"], case["dtype"]
    s = {"case": case}
    if case["op"] == "matmul":
        xq, xb = _quantized(_stream(g, T, K, "f32"), bits)
        s["x_codes"] = xq.to(torch.float8_e4m3fn).view(torch.uint8) if bits == 8 else _packed(xq)
        s["x_scales"] = _tiled(xb)
        del xq
        wq, wb = _quantized(0.02 * torch.randn(case["N"], K, generator=g, device="cuda"), 4)
        s["w_codes"], s["w_scales"] = _packed(wq), _tiled(wb)
    elif case["op"] == "roundtrip":
        s["x"] = (0.02 * torch.randn(T, K, generator=g, device="cuda")).to(DTYPES[dtype])
    elif case["op"] == "rmsnorm":
        s["x"] = _stream(g, T, K, dtype)
        s["residual"] = (4 * torch.randn(T, K, generator=g, device="cuda")).to(DTYPES[dtype])
        s["g"] = (1 + 0.2 * torch.randn(K, generator=g, device="cuda")).to(DTYPES[dtype])
    elif case["op"] == "swiglu":
        s["gate"] = (2 * torch.randn(T, K, generator=g, device="cuda")).to(DTYPES[dtype])
        s["up"] = _stream(g, T, K, dtype)
    else:
        s["x"] = _stream(g, T, K, dtype)
    return s


# One pass.

def _as_8bit(codes, scales):
    return {"codes": codes.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}


def _plain_8bit(v):
    q, byte = _quantized(v, 8)
    return _as_8bit(q.to(torch.float8_e4m3fn), _tiled(byte))


def _run_plain(s):
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        x = _dequantized(s["x_codes"], s["x_scales"], case["bits"])
        w = _dequantized(s["w_codes"], s["w_scales"], 4)
        return (x @ w.T).to(dtype)
    if case["op"] == "quantize":
        return _plain_8bit(s["x"].float())
    if case["op"] == "roundtrip":
        q, byte = _quantized(s["x"].float(), 4)
        v = q.view(q.shape[0], -1, 32) * _scale(byte).unsqueeze(-1)
        return v.view(q.shape)[:, :case["K"]].to(dtype)
    if case["op"] == "rmsnorm":
        h = s["x"].float() + s["residual"].float()
        n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["g"].float()
        return {**_plain_8bit(n), "h": h.to(dtype)}
    gate = s["gate"].float()
    return _plain_8bit(gate / (1 + torch.exp(-gate)) * s["up"].float())


def _run_own(s):
    import quantized_matmul_q4_gb300 as q4mm
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "matmul":
        x = q4mm.MxTensor(s["x_codes"], s["x_scales"], case["K"], case["bits"])
        w = q4mm.MxTensor(s["w_codes"], s["w_scales"], case["K"], 4)
        return q4mm.mx_matmul(x, w, dtype=dtype)
    if case["op"] == "quantize":
        q = q4mm.mx_quantize(s["x"], bits=8)
        return _as_8bit(q.codes, q.scales)
    if case["op"] == "roundtrip":
        return q4mm.mx_dequantize(q4mm.mx_quantize(s["x"], bits=4), dtype=dtype)
    if case["op"] == "rmsnorm":
        q, h = q4mm.mx_rmsnorm(s["x"], s["g"], eps=EPS, residual=s["residual"], bits=8)
        return {**_as_8bit(q.codes, q.scales), "h": h}
    q = q4mm.mx_swiglu(s["gate"], s["up"], bits=8)
    return _as_8bit(q.codes, q.scales)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# What a pass cannot do without.

def _mx_bytes(rows, K, bits):
    return rows * _padded(K) * bits // 8 + rows * _padded(K) // 32


def work(case):
    T, K, bits, size = case["T"], case["K"], case["bits"], SIZE[case["dtype"]]
    if case["op"] == "matmul":
        N = case["N"]
        return {"bytes": _mx_bytes(T, K, bits) + _mx_bytes(N, K, 4) + T * N * size, "flops": 2 * T * N * K}
    if case["op"] == "quantize":
        return {"bytes": T * K * size + _mx_bytes(T, K, 8), "flops": 4 * T * K}
    if case["op"] == "roundtrip":  # x read, codes written and read, values written
        return {"bytes": 2 * T * K * size + 2 * _mx_bytes(T, K, 4), "flops": 5 * T * K}
    if case["op"] == "rmsnorm":
        return {"bytes": 3 * T * K * size + K * size + _mx_bytes(T, K, 8), "flops": 9 * T * K}
    return {"bytes": 2 * T * K * size + _mx_bytes(T, K, 8), "flops": 8 * T * K}


# The definitions in 64 bits.

def _code_grid(bits):
    """The non-negative code values, in order."""
    if bits == 4:
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_mx(v, bits):
    """Code values and scales in float64 of v [rows, K] in float64 (finite): each value goes to the nearest
    code, found by search among the codes; halfway goes to the code of even index."""
    rows, K = v.shape
    b = torch.zeros(rows, _padded(K), dtype=torch.float64, device=v.device)
    b[:, :K] = v
    b = b.view(rows, -1, 32)
    top = b.abs().max(-1).values
    power = torch.floor(torch.log2(top.clamp(min=2.0 ** -160)))
    power = power - (torch.exp2(power) > top).double() + (torch.exp2(power + 1) <= top).double()
    power = (power - EMAX[bits]).clamp(-127, 127)
    power = torch.where(top > 0, power, torch.full_like(power, -127.0))
    grid = torch.tensor(_code_grid(bits), dtype=torch.float64, device=v.device)
    half = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(b)
    for i in range(0, rows, 1024):
        u = b[i:i + 1024] * torch.exp2(-power[i:i + 1024]).unsqueeze(-1)
        a = u.abs()
        lo = torch.bucketize(a, half, right=False)   # halfway values go down here,
        hi = torch.bucketize(a, half, right=True)    # and up here
        out[i:i + 1024] = torch.copysign(grid[torch.where(lo % 2 == 0, lo, hi)], u)
    return out, power


def _exact_8bit(v):
    q, power = _exact_mx(v, 8)
    rows, nb = power.shape
    s = torch.full((-(-rows // 128) * 128, nb), 2.0 ** -127, dtype=torch.float64, device=v.device)
    s[:rows] = torch.exp2(power)
    r, b = torch.arange(s.shape[0], device=v.device).view(-1, 1), torch.arange(nb, device=v.device)
    t = torch.empty(s.shape[0] // 128, nb // 4, 512, dtype=torch.float64, device=v.device)
    t[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = s
    return {"codes": q.reshape(rows, -1), "scales": t}


def _exact_values(codes, scales, bits):
    """What codes and tiled scales stand for, looked up value by value."""
    rows = codes.shape[0]
    if bits == 4:
        table = _code_grid(4)
        table = table + [-x for x in table]
        c = torch.empty(rows, 2 * codes.shape[1], dtype=torch.int64, device=codes.device)
        c[:, 0::2], c[:, 1::2] = (codes % 16).long(), (codes // 16).long()
    else:
        table = _code_grid(8) + [math.nan]
        table = table + [-x for x in table]
        c = codes.long()
    v = torch.tensor(table, dtype=torch.float64, device=codes.device)[c]
    r = torch.arange(rows, device=codes.device).view(-1, 1)
    b = torch.arange(v.shape[1] // 32, device=codes.device)
    s = torch.exp2(scales[r // 128, b // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4].double() - 127)
    return v * s.repeat_interleave(32, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "matmul":
        w = _exact_values(s["w_codes"], s["w_scales"], 4)
        x = _exact_values(s["x_codes"], s["x_scales"], case["bits"])
        return x @ w.T
    if case["op"] == "quantize":
        return _exact_8bit(s["x"].double())
    if case["op"] == "roundtrip":
        q, power = _exact_mx(s["x"].double(), 4)
        return (q * torch.exp2(power).unsqueeze(-1)).reshape(q.shape[0], -1)[:, :case["K"]].contiguous()
    if case["op"] == "rmsnorm":
        h = s["x"].double() + s["residual"].double()
        n = h / torch.sqrt((h ** 2).sum(-1, keepdim=True) / case["K"] + EPS) * s["g"].double()
        return {**_exact_8bit(n), "h": h}
    g = s["gate"].double()
    return _exact_8bit(g * torch.sigmoid(g) * s["up"].double())
