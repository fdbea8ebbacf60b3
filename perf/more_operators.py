"""Cases, plain forms and 64-bit definitions of the attention operators on a quantised, paged cache.

The cache keeps keys and values of `pages` pages of `page` tokens for each
key/value head in microscaled (MX) blocks of 32 values along the head: codes
[pages, kv heads, page, D * bits / 8] (E2M1, two per byte, the even value in
the low nibble, or E4M3) and power-of-two scales [pages, kv heads, page, 4]
(E8M0 bytes, block b of the head in byte b, zero bytes past the head).

A batch is described by `starts` (rows starts[i] .. starts[i + 1] of q, k and v
are the new tokens of sequence i), `lengths` (tokens of sequence i in the cache,
the new ones last among them) and a table `pages`: position p of sequence i lies
in page pages[i][p / page] at place p % page.

Operators (`op` of a case):
  rope       pairs of a head's values turned by position * frequency
  write      k (turned) and v of the new tokens -> codes and scales in their pages
  roundtrip  the same in 4 bits, and the values of the new tokens read back
  read       the values of the new tokens
  attention  softmax(scale q k^T) v of the new tokens' queries over the cache, each
             key/value head shared by heads / kv_heads query heads
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
BASE = 10000.0


def listed():
    return [
        # Decode: one token's 32 query heads (Llama-2-7B's), in the FP32 stream of this framework.
        {"name": "rope_t1_h32", "op": "rope", "T": 1, "heads": 32, "D": 128, "rotated": 128, "interleaved": False,
         "stretch": 1.0, "far": 4000, "dtype": "f32"},
        # A large prefill batch, half of each head rotated in interleaved pairs, positions of a stretched long context.
        {"name": "rope_t8192_h32_part", "op": "rope", "T": 8192, "heads": 32, "D": 128, "rotated": 64,
         "interleaved": True, "stretch": 32.0, "far": 120000, "dtype": "bf16"},
        # A decoding step of 64 sequences: each one's new key and value into its last page.
        {"name": "write_8b_s64", "op": "write", "seqs": 64, "new": 1, "context": 2000, "ragged": True, "heads": 32,
         "kv_heads": 32, "D": 128, "page": 16, "bits": 8, "rotated": 128, "interleaved": False, "dtype": "bf16"},
        # Prompts of uneven lengths, some behind a cached prefix, written at once.
        {"name": "write_8b_s5_t8700", "op": "write", "seqs": 5, "new": 2801, "context": 3500, "ragged": True, "heads": 32,
         "kv_heads": 32, "D": 128, "page": 64, "bits": 8, "rotated": 128, "interleaved": False, "dtype": "f16"},
        # A short sequence of a 4-bit cache taken out for inspection.
        {"name": "read_4b_t333", "op": "read", "seqs": 1, "new": 333, "context": 333, "ragged": False, "heads": 20,
         "kv_heads": 5, "D": 128, "page": 16, "bits": 4, "dtype": "f32"},
        # Eight sequences' caches taken out whole, as when they move to another store.
        {"name": "read_8b_s8_t28000", "op": "read", "seqs": 8, "new": 4000, "context": 4000, "ragged": True, "heads": 32,
         "kv_heads": 8, "D": 128, "page": 64, "bits": 8, "dtype": "bf16"},
        # Decode of one sequence: one token's heads over a thousand cached tokens.
        {"name": "attention_8b_s1_c1000", "op": "attention", "seqs": 1, "new": 1, "context": 1000, "ragged": False,
         "heads": 32, "kv_heads": 32, "D": 128, "page": 16, "bits": 8, "causal": True, "dtype": "bf16"},
        # Decode of 64 sequences of uneven lengths, every head with keys of its own: all of the cache is read.
        {"name": "attention_8b_s64_c4096", "op": "attention", "seqs": 64, "new": 1, "context": 4096, "ragged": True,
         "heads": 32, "kv_heads": 32, "D": 128, "page": 16, "bits": 8, "causal": True, "dtype": "f16"},
        # Decode of one long sequence, four query heads to a key head, 4-bit cache.
        {"name": "attention_4b_s1_c131071", "op": "attention", "seqs": 1, "new": 1, "context": 131071, "ragged": False,
         "heads": 20, "kv_heads": 5, "D": 128, "page": 64, "bits": 4, "causal": True, "dtype": "bf16"},
        # Three odd prompts together, small heads, an odd page size, FP32 stream.
        {"name": "attention_4b_s3_n301_f32", "op": "attention", "seqs": 3, "new": 301, "context": 700, "ragged": True,
         "heads": 12, "kv_heads": 4, "D": 64, "page": 48, "bits": 4, "causal": True, "dtype": "f32"},
        # A chunk of a long prompt: 512 new tokens over what is cached already.
        {"name": "attention_8b_n512_c8192", "op": "attention", "seqs": 1, "new": 512, "context": 8192, "ragged": False,
         "heads": 32, "kv_heads": 8, "D": 128, "page": 64, "bits": 8, "causal": True, "dtype": "bf16"},
        # A whole long prompt at once: the largest.
        {"name": "attention_8b_n8192_c8192", "op": "attention", "seqs": 1, "new": 8192, "context": 8192, "ragged": False,
         "heads": 32, "kv_heads": 32, "D": 128, "page": 64, "bits": 8, "causal": True, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "roundtrip", "read"] + 5 * ["attention"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    D = rng.choice([64, 96, 128, 128])
    if op == "rope":
        T, heads = _log_int(rng, 1, 16384), _log_int(rng, 1, 64)
        while T * heads * D * SIZE[dtype] > 8192 * 32 * 128 * 2:
            T = T // 2 + 1
        return {"op": op, "T": T, "heads": heads, "D": D, "rotated": rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)]),
                "interleaved": rng.random() < 0.5, "stretch": rng.choice([1.0, 4.0, 32.0]),
                "far": _log_int(rng, 100, 500000), "dtype": dtype}
    kv_heads = rng.choice([1, 2, 4, 5, 8, 32])
    heads = kv_heads * rng.choice([1, 1, 2, 4, 7, 8] if kv_heads <= 8 else [1])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "D": D, "page": rng.choice([16, 32, 48, 64, 128]),
            "bits": 4 if op == "roundtrip" else 8 if op == "write" else rng.choice([4, 8]), "ragged": rng.random() < 0.7,
            "dtype": dtype}
    if op == "attention":
        kind = rng.choice(["decode", "decode", "chunk", "prompt"])
        seqs = _log_int(rng, 1, 64) if kind == "decode" else rng.randint(1, 6)
        new = rng.choice([1, 1, 1, rng.randint(2, 9)]) if kind == "decode" else _log_int(rng, 10, 8192)
        context = new if kind == "prompt" else new + _log_int(rng, 10, 131072)
        case.update(seqs=seqs, new=new, context=context, causal=rng.random() < 0.85)
        # No more than the largest listed one computes, and tokens for no more than a few GB in 32 bits.
        while case["seqs"] * case["new"] * case["context"] * heads * D * {"f32": 2, "f16": 1, "bf16": 1}[dtype] > 8192 ** 2 * 32 * 64 \
                or case["seqs"] * case["context"] * kv_heads * D > 64 * 4096 * 32 * 64:
            shorter = case["context"] // 2 + 1
            case["new"] = min(case["new"], max(1, case["new"] // 2)) if kind != "prompt" else shorter
            case["context"] = max(shorter, case["new"])
        return case
    rotated = rng.choice([D, D, D // 2])
    case.update(seqs=_log_int(rng, 1, 64), new=_log_int(rng, 1, 8192))
    case["context"] = case["new"] + _log_int(rng, 1, 4000)
    if op != "read":
        case.update(rotated=rotated, interleaved=rng.random() < 0.5)
    while case["seqs"] * case["new"] * kv_heads * D > 8192 * 32 * 128:
        case["new"] = case["new"] // 2 + 1
    while case["seqs"] * case["context"] * kv_heads * D > 2 * 8192 * 32 * 128 and case["context"] > case["new"]:
        case["context"] = max(case["new"], case["context"] // 2)
    return case


def _spread(case):
    """New tokens and lengths of each sequence: alike, or between a quarter and the whole."""
    new, prior = case["new"], case["context"] - case["new"]
    out = []
    for i in range(case["seqs"]):
        a = 0.25 + 0.75 * ((i + 1) * 0.618034 % 1) if case["ragged"] else 1.0
        b = 0.25 + 0.75 * ((i + 1) * 0.414214 % 1) if case["ragged"] else 1.0
        n = max(1, round(a * new))
        out.append((n, n + round(b * prior)))
    return [n for n, _ in out], [m for _, m in out]


# Codes, scales and angles of the plain form.

def _quantized(v, bits):
    """Code values (float32, v's shape) and scale bytes [..., 4] of v [..., D]."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 1 - EMAX[bits]
    byte = torch.where(amax > 0, (e + 127).clamp(0, 254), torch.zeros_like(e))
    s = torch.ldexp(b, (127 - byte).unsqueeze(-1))
    step = (torch.frexp(s)[1] - 1).clamp(min=EMIN[bits]) - MANT[bits]
    q = torch.ldexp(torch.round(torch.ldexp(s, -step)), step).clamp(-LARGEST[bits], LARGEST[bits])
    return q.flatten(-2), torch.nn.functional.pad(byte, (0, 4 - byte.shape[-1])).to(torch.uint8)


def _packed(q, bits):
    """Code values as bytes [..., D * bits / 8]."""
    if bits == 8:
        return q.to(torch.float8_e4m3fn).view(torch.uint8)
    a = q.abs()
    mag = (2 * a).where(a < 2, (a + 2).where(a < 4, a / 2 + 4)).to(torch.uint8)
    c = mag | ((q < 0).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _values(codes, scales, bits):
    """float32 values [..., D] of codes and their scale bytes [..., 4]."""
    if bits == 8:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
        e, m = (c >> 1) & 3, (c & 1).float()
        v = torch.where(e > 0, torch.ldexp(1 + 0.5 * m, e - 1), 0.5 * m)
        v = torch.where(c >= 8, -v, v)
    b = v.unflatten(-1, (-1, 32))
    s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)[..., :b.shape[-2]]
    return (b * s.unsqueeze(-1)).flatten(-2)


def _turned(x, positions, frequencies, interleaved):
    """x [T, H, D] in float32 with its first pairs turned; angles in 64 bits, their sines and cosines in 32."""
    R = 2 * frequencies.numel()
    a = torch.remainder(positions.double().unsqueeze(-1) * frequencies, 2 * math.pi)
    c, s = torch.cos(a).float().unsqueeze(1), torch.sin(a).float().unsqueeze(1)
    if interleaved:
        u, v = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2)
    else:
        u, v = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat((u * c - v * s, v * c + u * s), -1)
    return torch.cat((turned, x[..., R:]), -1)


# Inputs.

def _frequencies(rotated, stretch):
    return torch.tensor([BASE ** (-2 * i / rotated) / stretch for i in range(rotated // 2)], dtype=torch.float64, device="cuda")


def _heads(g, T, H, D):
    """Rows of heads whose channels differ in size, a few of them much larger, as keys and queries have them."""
    size = torch.exp(0.4 * torch.randn(H, D, generator=g, device="cuda"))
    size = torch.where(torch.rand(H, D, generator=g, device="cuda") < 0.01, 5 * size, size)
    return torch.randn(T, H, D, generator=g, device="cuda") * size


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "rope":
        return {"case": case, "x": _heads(g, case["T"], case["heads"], case["D"]).to(dtype),
                "positions": torch.randint(0, case["far"], (case["T"],), generator=g, device="cuda", dtype=torch.int32),
                "frequencies": _frequencies(case["rotated"], case["stretch"])}
    D, page, Hk, bits = case["D"], case["page"], case["kv_heads"], case["bits"]
    new, lengths = _spread(case)
    T = sum(new)
    used = [-(-m // page) for m in lengths]
    total = sum(used) + 3                            # some pages are another program's
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(used), max(used), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(used):
        table[i, :n] = order[at:at + n]
        at += n
    ints = dict(dtype=torch.int32, device="cuda")
    s = {"case": case, "new": new, "lengths_list": lengths, "T": T, "pages": table,
         "starts": torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], **ints), "lengths": torch.tensor(lengths, **ints)}
    writes = case["op"] in ("write", "roundtrip")
    for what in ("k", "v"):
        if writes:
            codes = torch.zeros(total, Hk, page, D * bits // 8, dtype=torch.uint8, device="cuda")
            scales = torch.zeros(total, Hk, page, 4, dtype=torch.uint8, device="cuda")
            s[what] = _heads(g, T, Hk, D).to(dtype)
        else:
            codes = torch.empty(total, Hk, page, D * bits // 8, dtype=torch.uint8, device="cuda")
            scales = torch.empty(total, Hk, page, 4, dtype=torch.uint8, device="cuda")
            step = max(1, 2 ** 27 // (Hk * page * D))
            for p in range(0, total, step):
                n = min(step, total - p)
                q, byte = _quantized(_heads(g, n * page, Hk, D).view(n, page, Hk, D).transpose(1, 2), bits)
                codes[p:p + n], scales[p:p + n] = _packed(q, bits), byte
        s[what + "_codes"], s[what + "_scales"] = codes, scales
    if writes:
        s["frequencies"] = _frequencies(case["rotated"], 1.0)
    if case["op"] == "attention":
        # Scores of a few units, so that some keys matter and most matter little.
        s["q"] = (1.5 * torch.randn(T, case["heads"], D, generator=g, device="cuda")).to(dtype)
    return s


# One pass.

def _places(s):
    """Of each new token its sequence and position, and the page and place it lies in."""
    starts, lengths = s["starts"].long(), s["lengths"].long()
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(starts, t, right=True) - 1
    pos = lengths[seq] - starts[seq + 1] + t
    page = s["case"]["page"]
    return seq, pos, s["pages"].long()[seq, pos // page], pos % page


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        return _turned(s["x"].float(), s["positions"], s["frequencies"], case["interleaved"]).to(s["x"].dtype)
    bits, dtype = case["bits"], DTYPES[case["dtype"]]
    seq, pos, page, place = _places(s)
    if case["op"] in ("write", "roundtrip"):
        kq, kb = _quantized(_turned(s["k"].float(), pos, s["frequencies"], case["interleaved"]), bits)
        vq, vb = _quantized(s["v"].float(), bits)
        s["k_codes"][page, :, place], s["k_scales"][page, :, place] = _packed(kq, bits), kb
        s["v_codes"][page, :, place], s["v_scales"][page, :, place] = _packed(vq, bits), vb
    if case["op"] == "write":
        return _cache_values(s)
    if case["op"] in ("read", "roundtrip"):
        return (_values(s["k_codes"][page, :, place], s["k_scales"][page, :, place], bits).to(dtype),
                _values(s["v_codes"][page, :, place], s["v_scales"][page, :, place], bits).to(dtype))
    # Every sequence padded to the longest: queries [B, kv heads, group, n, D], keys [B, kv heads, L, D].
    B, Hk, D, n, L = case["seqs"], case["kv_heads"], case["D"], max(s["new"]), max(s["lengths_list"])
    table = s["pages"].long()
    k = _values(s["k_codes"][table], s["k_scales"][table], bits).transpose(1, 2).reshape(B, Hk, -1, D)[:, :, :L]
    v = _values(s["v_codes"][table], s["v_scales"][table], bits).transpose(1, 2).reshape(B, Hk, -1, D)[:, :, :L]
    row = torch.arange(s["T"], device="cuda") - s["starts"].long()[seq]
    q = torch.zeros(B, n, Hk, case["heads"] // Hk, D, device="cuda")
    q[seq, row] = s["q"].float().unflatten(1, (Hk, -1))
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, D)
    p = q @ k.transpose(-1, -2)
    p *= D ** -0.5
    j = torch.arange(L, device="cuda")
    lengths, new = s["lengths"].long(), s["starts"].long().diff()
    last = torch.where(torch.tensor(case["causal"], device="cuda"),
                       (lengths - new).unsqueeze(-1) + torch.arange(n, device="cuda"), (lengths - 1).unsqueeze(-1))
    hidden = j > torch.minimum(last, (lengths - 1).unsqueeze(-1)).unsqueeze(-1)          # [B, n, L]
    p = p.view(B, Hk, -1, n, L).masked_fill_(hidden.view(B, 1, 1, n, L), -math.inf)
    p -= p.amax(-1, keepdim=True)
    p.exp_()
    p /= p.sum(-1, keepdim=True)
    y = (p.view(B, Hk, -1, L) @ v).view(B, Hk, -1, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, -1, D)
    return y[seq, row].to(dtype)


def _cache_values(s):
    return {"k_codes": s["k_codes"].view(torch.float8_e4m3fn), "k_scales": s["k_scales"].view(torch.float8_e8m0fnu),
            "v_codes": s["v_codes"].view(torch.float8_e4m3fn), "v_scales": s["v_scales"].view(torch.float8_e8m0fnu)}


def _run_own(s):
    import quantized_matmul_q4_gb300 as q4mm
    case = s["case"]
    if case["op"] == "rope":
        return q4mm.rope_rotate(s["x"], s["positions"], q4mm.Rope(s["frequencies"], case["interleaved"]))
    cache = q4mm.MxCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], case["D"], case["bits"])
    batch = (s["starts"], s["lengths"], s["pages"])
    if case["op"] in ("write", "roundtrip"):
        q4mm.mx_cache_write(cache, s["k"], s["v"], *batch, rope=q4mm.Rope(s["frequencies"], case["interleaved"]))
    if case["op"] == "write":
        return _cache_values(s)
    if case["op"] in ("read", "roundtrip"):
        return q4mm.mx_cache_read(cache, *batch, tokens=s["T"], dtype=DTYPES[case["dtype"]])
    return q4mm.mx_attention(s["q"], cache, *batch, causal=case["causal"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# What a pass cannot do without.

def work(case):
    D, size = case["D"], SIZE[case["dtype"]]
    if case["op"] == "rope":
        n = case["T"] * case["heads"]
        return {"bytes": 2 * n * D * size + 4 * case["T"] + 4 * case["rotated"], "flops": 3 * n * case["rotated"]}
    new, lengths = _spread(case)
    Hk, held = case["kv_heads"], D * case["bits"] // 8 + D // 32    # bytes of a token's key, or value, of a head
    if case["op"] in ("write", "roundtrip", "read"):
        n, twice = 2 * sum(new) * Hk, case["op"] == "roundtrip"
        return {"bytes": (1 + twice) * n * (D * size + held), "flops": n * D * (2 if case["op"] == "read" else 7)}
    keys = sum(n * m - (n * (n - 1) // 2 if case["causal"] else 0) for n, m in zip(new, lengths))
    return {"bytes": 2 * sum(lengths) * Hk * held + 2 * sum(new) * case["heads"] * D * size,
            "flops": 4 * keys * case["heads"] * D}


# The definitions in 64 bits.

def _code_grid(bits):
    """The non-negative code values, in order."""
    if bits == 4:
        return [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1]


def _exact_mx(v, bits):
    """Code values [T, H, D] and scales [T, H, 4] in float64 of v: the nearest code by search, halfway the even one."""
    T, H, D = v.shape
    b = v.reshape(T, H, D // 32, 32)
    top = b.abs().max(-1).values
    power = torch.floor(torch.log2(top.clamp(min=2.0 ** -160)))
    power = power - (torch.exp2(power) > top).double() + (torch.exp2(power + 1) <= top).double()
    power = torch.where(top > 0, (power - EMAX[bits]).clamp(-127, 127), torch.full_like(power, -127.0))
    grid = torch.tensor(_code_grid(bits), dtype=torch.float64, device=v.device)
    half = (grid[1:] + grid[:-1]) / 2
    out = torch.empty_like(b)
    for i in range(0, T, 512):
        u = b[i:i + 512] * torch.exp2(-power[i:i + 512]).unsqueeze(-1)
        lo, hi = torch.bucketize(u.abs(), half, right=False), torch.bucketize(u.abs(), half, right=True)
        out[i:i + 512] = torch.copysign(grid[torch.where(lo % 2 == 0, lo, hi)], u)
    scales = torch.full((T, H, 4), 2.0 ** -127, dtype=torch.float64, device=v.device)
    scales[..., :D // 32] = torch.exp2(power)
    return out.reshape(T, H, D), scales


def _exact_values(codes, scales, bits):
    """What codes [..., D * bits / 8] with scales [..., 4] stand for, looked up value by value."""
    table = _code_grid(bits) + ([math.nan] if bits == 8 else [])
    table = torch.tensor(table + [-x for x in table], dtype=torch.float64, device=codes.device)
    c = codes.long() if bits == 8 else torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)
    return table[c] * s[..., :c.shape[-1]]


def _exact_turned(x, positions, frequencies, interleaved):
    out = x.clone()
    R = 2 * frequencies.numel()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        angle = (positions.double() * frequencies[i]).unsqueeze(-1)
        out[..., a] = x[..., a] * torch.cos(angle) - x[..., b] * torch.sin(angle)
        out[..., b] = x[..., a] * torch.sin(angle) + x[..., b] * torch.cos(angle)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_turned(s["x"].double(), s["positions"], s["frequencies"], case["interleaved"])
    page, table, new, lengths = case["page"], s["pages"].tolist(), s["new"], s["lengths_list"]
    places = [[(table[i][p // page], p % page) for p in range(m)] for i, m in enumerate(lengths)]
    fresh = [at for n, all_of in zip(new, places) for at in all_of[len(all_of) - n:]]
    fp, fo = (torch.tensor(x, device="cuda") for x in zip(*fresh))
    if case["op"] in ("write", "roundtrip"):
        pos = torch.tensor([p for n, m in zip(new, lengths) for p in range(m - n, m)], device="cuda")
        kq, ks = _exact_mx(_exact_turned(s["k"].double(), pos, s["frequencies"], case["interleaved"]), case["bits"])
        vq, vs = _exact_mx(s["v"].double(), case["bits"])
        if case["op"] == "roundtrip":
            return (kq * ks.repeat_interleave(32, dim=-1)[..., :case["D"]], vq * vs.repeat_interleave(32, dim=-1)[..., :case["D"]])
        out = {}
        for what, q, sc in (("k", kq, ks), ("v", vq, vs)):
            out[what + "_codes"] = torch.zeros(s[what + "_codes"].shape, dtype=torch.float64, device="cuda")
            out[what + "_scales"] = torch.full(s[what + "_scales"].shape, 2.0 ** -127, dtype=torch.float64, device="cuda")
            out[what + "_codes"][fp, :, fo], out[what + "_scales"][fp, :, fo] = q, sc
        return out
    if case["op"] == "read":
        return tuple(_exact_values(s[w + "_codes"][fp, :, fo], s[w + "_scales"][fp, :, fo], case["bits"]) for w in ("k", "v"))
    group = case["heads"] // case["kv_heads"]
    y, at = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for n, m, all_of in zip(new, lengths, places):
        p, o = (torch.tensor(x, device="cuda") for x in zip(*all_of))
        last = torch.arange(m - n, m, device="cuda") if case["causal"] else torch.full((n,), m - 1, device="cuda")
        for h in range(case["kv_heads"]):
            k, v = (_exact_values(s[w + "_codes"][p, h, o], s[w + "_scales"][p, h, o], case["bits"]) for w in ("k", "v"))
            for f in range(h * group, (h + 1) * group):
                score = s["q"][at:at + n, f].double() @ k.T / math.sqrt(case["D"])
                score = torch.where(torch.arange(m, device="cuda") <= last.unsqueeze(-1), score, -math.inf)
                y[at:at + n, f] = torch.softmax(score, -1) @ v
        at += n
    return y
