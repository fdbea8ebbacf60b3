"""Attention over caches whose lengths and values lie at the ends of what the types hold.

Tolerances as derived in test_gpu_attention.
"""
import numpy as np
import pytest

import attention_reference as ref
import test_gpu_attention as base
import test_gpu_attention_batches as batches
from test_gpu_attention import KERNELS, Case, kernel  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def test_lengths_up_to_the_last_position():
    """A sequence of 2^31 - 256 tokens, whose table repeats one page of 2^24, gives what that page gives; a longer one is
    reported, as is one that is longer than its table.  The keys are shared by 15 clusters of 8 CTAs of 8 warps at least, each
    of which adds 2^31 / 960 / 16 < 2^18 times and drops at most 2^-23 of the sum each time."""
    q, torch = _q(), _torch()
    page = 2 ** 24
    cache = q.mx_cache(1, 1, 32, page=page, bits=4)
    g = torch.Generator(device="cuda").manual_seed(1)
    cache.k_codes.random_(0, 256, generator=g), cache.v_codes.fill_(0x22)       # values of v: 1
    cache.k_scales.fill_(125), cache.v_scales.fill_(127)
    x = torch.randn(1, 8, 32, generator=g, device="cuda")
    starts, table = base._i32([0, 1]), torch.zeros(1, 129, dtype=torch.int32, device="cuda")
    q.device_status()
    for dtype in (torch.float32, torch.bfloat16):
        y = q.mx_attention(x.to(dtype), cache, starts, base._i32([2 ** 31 - 256]), table)
        q.device_status()
        assert float((y.float() - 1).abs().max()) <= 2.0 ** -5 + base._half(str(dtype)[6:])
    for n, width in ((2 ** 31 - 1, 129), (2 ** 31 - 200, 129), (2 ** 24 + 1, 1)):
        q.mx_attention(x, cache, starts, base._i32([n]), table[:, :width].contiguous())
        with pytest.raises(q.Q4mmError) as e:
            q.device_status()
        assert e.value.code == -7


# Powers of two by which the values of neighbouring groups of tokens differ, in turn; None: all zeros.
POWERS = {"zeros": [None, 0, None], "zeros beside 2^50": [None, 50], "2^50 beside zeros": [50, None, None], "2^100, then zeros": [100, None],
          "far apart": [0, -60, 60, 100, None, -100], "up": [-100, 0, 100], "down": [100, 0, -100], "a step": [0, 0, 45], "tiny": [-112],
          "tiny, and zeros": [None, -112], "huge": [112, 112, 90]}


def _spread(scales, codes, powers, run):
    """Scale bytes [..., places, 4] and codes of v, in runs of `run` tokens, moved by the powers in turn."""
    torch = _torch()
    at = torch.arange(scales[..., 0].numel(), device=scales.device).view(scales.shape[:-1]) // run % len(powers)
    for i, p in enumerate(powers):
        mine = (at == i)[..., None]
        if p is None:
            scales.masked_fill_(mine, 0), codes.masked_fill_(mine, 0)
        else:
            scales.copy_(torch.where(mine, (scales.int() + p).clamp(0, 246), scales.int()).to(torch.uint8))


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("run", [1, 16, 64])
@pytest.mark.parametrize("news,lengths,bits", [([1], [900], 8), ([1], [30000], 4), ([150], [700], 8), ([3, 20], [60, 333], 4)])
@pytest.mark.parametrize("powers", POWERS)
def test_values_of_any_powers(powers, news, lengths, bits, run, dtype):
    """Groups of tokens whose values differ by any powers of two, zeros among them: each counts in the sum of probabilities
    by its scores alone."""
    q = _q()
    b = batches.Batch(news, lengths, 2, 64, 64, bits, seed=run)
    _spread(b.cache.v_scales, b.cache.v_codes, POWERS[powers], run)
    x = b.queries(4, dtype, size=1.0)
    y = q.mx_attention(x, b.cache, *b.batch)
    q.device_status()
    assert bool(_torch().isfinite(y).all())
    b.check(x, y)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("high,low", [(60, -60), (100, -20), (20, -110), (0, -110)])
def test_small_values_of_large_probability(high, low, dtype):
    """Keys of tiny values whose probability makes them as large a part of the output as the huge values of keys of
    little probability, and far larger scores of keys without values."""
    q, torch = _q(), _torch()
    for n, m in ((1, 600), (140, 600)):
        c = Case(17, [n], [m], 1, 64, 16, 8).fill(size=0.01)
        gap = (high - low) * np.log(2)
        for p in range(m):
            pg, at, kind = c.table[0, p // 16], p % 16, p // 16 % 3
            s = c.cache["v_scales"][pg, 0, at]
            s[:2] = np.clip(s[:2].astype(int) + 6 + (high, low, 0)[kind], 0, 246)
            if kind == 2:
                c.cache["v_codes"][pg, 0, at], s[:] = 0, 0
            # k's first value alone makes the score: 0 for huge values, gap for tiny ones, a little less for none
            codes, byte = ref.head_codes(np.concatenate([[(0, 16, 15)[kind]], np.zeros(63)]), 8)
            c.cache["k_codes"][pg, 0, at], c.cache["k_scales"][pg, 0, at] = codes, byte
        x = np.zeros((n, 2, 64))
        x[..., 0] = gap / 16 * c.rng.uniform(0.9, 1.1, (n, 2))
        x, xv = base._dev(x, dtype)
        y = q.mx_attention(x, c.device_cache(), *c.device_batch(), scale=1.0)
        base._check(c, x, y, xv, dtype, scale=1.0)


@KERNELS
@pytest.mark.parametrize("D,bits,keys,rows,dtype", [
    (64, 8, 0, 152, "float16"), (128, 8, 0, 152, "float16"), (128, 4, 0, 152, "float16"), (64, 4, 0, 152, "float16"),
    (128, 8, 1, 152, "float16"), (64, 4, 1, 152, "float16"), (128, 8, 2, 8, "bfloat16"), (96, 4, 2, 8, "bfloat16")])
def test_long_16_bit_sums_do_not_drift(kernel, D, bits, keys, rows, dtype):
    """Values of one over more keys than a sum in the tensor cores may hold, which drops up to 2^-23 of itself a step of 16
    keys: outputs are one, whatever the keys that a CTA takes.  (Probabilities of 16 bits round by chance, and an fp16
    output is one as long as its value is within 2^-12.)"""
    q, torch = _q(), _torch()
    keys, page = ((3_000_000, 500_000), (5_000_000, 600_000), (3_000_000, 5_000_000))[keys][kernel == "many"], 4096
    cache = q.mx_cache(1, 2, D, page=page, bits=bits)
    g = torch.Generator(device="cuda").manual_seed(D + bits)
    k = torch.randn(page, 2, D, generator=g, device="cuda")
    q.mx_cache_write(cache, k, torch.ones_like(k), base._i32([0, page]), base._i32([page]), base._i32([[0]]))
    x = torch.randn(rows, 4, D, generator=g, device="cuda").to(getattr(torch, dtype))
    table = torch.zeros(rows, -(-keys // page), dtype=torch.int32, device="cuda")
    y = q.mx_attention(x, cache, torch.arange(rows + 1, dtype=torch.int32, device="cuda"),
                       torch.full((rows,), keys, dtype=torch.int32, device="cuda"), table)
    q.device_status()
    assert bool((y == 1).all())


def test_long_16_bit_sums_without_a_workspace():
    """One row over more keys than one cluster's sums may hold, the parts' workspace left out."""
    q, torch = _q(), _torch()
    keys, page = 5_000_000, 4096
    c = q.mx_cache(1, 1, 64, page=page)
    k = torch.randn(page, 1, 64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    q.mx_cache_write(c, k, torch.ones_like(k), base._i32([0, page]), base._i32([page]), base._i32([[0]]))
    x = torch.randn(1, 4, 64, device="cuda").half()
    table, starts, lengths = torch.zeros(1, -(-keys // page), dtype=torch.int32, device="cuda"), base._i32([0, 1]), base._i32([keys])
    y = torch.empty_like(x)
    q.mx_attention_ptr((x.data_ptr(), 256, 64), 1, (*[t.data_ptr() for t in c[:4]], 1, 1, page, 64, 8),
                       (starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), 1, table.shape[1]), 0.125, 1,
                       (y.data_ptr(), 256, 64), 1, 4, 0, 0, torch.cuda.current_stream().cuda_stream)
    q.device_status()
    assert bool((y == 1).all())


@pytest.mark.filterwarnings("ignore:All-NaN slice")
@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("news,lengths,D", [([5], [40], 128), ([5], [40], 64), ([1, 1], [700, 90], 96), ([150], [400], 128), ([300, 20], [300, 333], 32)])
def test_nan_codes_stay_where_they_are_seen(news, lengths, D, dtype):
    """Codes of v that are NaN (the format has them; no call here writes them) reach the rows that see them, in their value
    alone; those under a NaN scale, in its block.  Codes of k reach the rows that see them whole."""
    q, torch = _q(), _torch()
    c = Case(sum(lengths) + D, news, lengths, 2, D, 16, 8).fill()
    n = news[0]
    last = int(c.lengths[0])
    def put(what, head, p, d, code):
        c.cache[what + "_codes"][c.table[0, p // 16], head, p % 16, d] = code
    if n > 1:
        put("v", 0, last - 1, 3, 0x7F), put("v", 0, last - n // 2, D - 1, 0xFF), put("v", 0, last - n // 2, 7, 0x7F)
        put("v", 1, last - 2, 5, 0x7F)
        c.cache["v_scales"][c.table[0, (last - 2) // 16], 1, (last - 2) % 16, 0] = 255
        put("k", 1, last - 1, 0, 0x7F)
    else:
        put("v", 0, 17, 40, 0xFF), put("v", 0, last - 1, 8, 0x7F)
    x, xv = base._dev(c.rng.normal(size=(c.T, 4, D)), dtype)
    y = q.mx_attention(x, c.device_cache(), *c.device_batch())
    q.device_status()
    assert bool(torch.isnan(y).any())
    base._check(c, x, y, xv, dtype)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("causal,scale", [(True, None), (False, 0.3), (True, 0.0)])
@pytest.mark.parametrize("news,lengths,group,D,page,bits", [
    ([1], [45], 1, 32, 16, 8), ([1], [3000], 4, 96, 48, 4), ([9, 0, 3], [9, 40, 1], 3, 128, 16, 8), ([40, 5], [200, 3], 2, 96, 16, 8),
    ([150], [333], 2, 32, 64, 4), ([300], [300], 1, 128, 32, 8)])
def test_far_values_in_every_shape(news, lengths, group, D, page, bits, causal, scale, dtype):
    """Values that the kernels' own sums cannot take, over head sizes, groups, rows that see nothing, unaligned and
    strided rows, with and without a mask, scores of zero among them."""
    q, torch = _q(), _torch()
    c = Case(sum(lengths) + D, news, lengths, 2, D, page, bits, offset=2).fill()
    for i, n in enumerate(lengths):
        for p in range(n):          # every fifth token tiny, some none at all; fp16 holds what the others give
            s = c.cache["v_scales"][c.table[i, p // page], :, p % page]
            if p % 5 == 0:
                s[:] = np.clip(s.astype(int) - 70, 0, 250)
            elif p % 7 == 0:
                s[:], c.cache["v_codes"][c.table[i, p // page], :, p % page] = 0, 0
    heads = 2 * group
    fused, _ = base._dev(1.5 * c.rng.normal(size=(c.T + 3, heads * D + 5)), dtype)
    x = fused[:, 3:3 + heads * D].view(c.T + 3, heads, D)
    out = torch.full((heads, c.T + 3, D + 1), 7.0, device="cuda", dtype=x.dtype)[..., :D].transpose(0, 1)
    q.mx_attention(x, c.device_cache(), *c.device_batch(), scale=scale, causal=causal, out=out)
    q.device_status()
    assert bool((out[:2] == 7).all()) and bool((out[c.T:] == 7).all())
    base._check(c, x, out, x.double().cpu().numpy(), dtype, causal=causal, scale=scale)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("gap", [20, 50, 65, 80])
def test_tokens_of_zeros_that_outweigh_all_others(gap, dtype):
    """Keys without values, 2^gap times as probable as the others: they shrink the output, and leave it its precision."""
    q = _q()
    for n, m in ((1, 700), (140, 600)):
        c = Case(18, [n], [m], 1, 64, 16, 8).fill()
        for p in range(m):
            pg, at = c.table[0, p // 16], p % 16
            codes, byte = ref.head_codes(np.concatenate([[16 if p // 32 % 4 == 0 else 0], np.zeros(63)]), 8)
            c.cache["k_codes"][pg, 0, at], c.cache["k_scales"][pg, 0, at] = codes, byte
            if p // 32 % 4 == 0:
                c.cache["v_codes"][pg, 0, at], c.cache["v_scales"][pg, 0, at] = 0, 0
        x = np.zeros((n, 2, 64))
        x[..., 0] = gap * np.log(2) / 16
        x, xv = base._dev(x, dtype)
        y = q.mx_attention(x, c.device_cache(), *c.device_batch(), scale=1.0)
        q.device_status()
        base._check(c, x, y, xv, dtype, scale=1.0)


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("n,m", [(1, 50), (5, 700), (150, 300)])
def test_rows_whose_scores_are_all_minus_infinity(n, m, far, dtype):
    """The softmax of such scores is NaN; those of rows that see no keys stay zeros, other rows as they are."""
    q, torch = _q(), _torch()
    c = Case(19, [n, 2], [m, 0], 1, 64, 16, 8).fill()
    c.cache["k_codes"] &= 0x7F          # k is positive,
    c.cache["k_codes"][..., 0] |= 0x38  # and not zero where the infinity is
    c.cache["k_codes"] = np.where(c.cache["k_codes"] == 0x7F, 0x78, c.cache["k_codes"]).astype(np.uint8)
    c.cache["k_scales"] = np.where(c.cache["k_scales"] > 140, 120, c.cache["k_scales"]).astype(np.uint8)
    if far:
        c.cache["v_scales"][c.table[0, 0], 0, 3] = 70
    x, xv = base._dev(c.rng.normal(size=(c.T, 2, 64)), dtype)
    x[0, 1, 0] = xv[0, 1, 0] = -np.inf
    y = q.mx_attention(x, c.device_cache(), *c.device_batch())
    assert bool(torch.isnan(y[0, 1]).all()) and int(torch.isnan(y).sum()) == 64 and bool((y[n:] == 0).all())
    xv[0, 1, 0] = 0
    x, xv = base._dev(xv, dtype)
    other = q.mx_attention(x, c.device_cache(), *c.device_batch())
    keep = ~torch.isnan(y)
    assert bool((y[keep] == other[keep]).all())
