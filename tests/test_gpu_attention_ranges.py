"""Attention over caches whose lengths and values lie at the ends of what the types hold.

Tolerances as derived in test_gpu_attention.
"""
import numpy as np
import pytest

import attention_reference as ref
import test_gpu_attention as base
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
