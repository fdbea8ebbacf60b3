"""Sizes of attention calls that its 32-bit row numbers and positions cannot hold: refused by the C ABI before any CUDA call, or
counted as beyond the table."""
import ctypes
import os
import subprocess

import pytest

DIM = -1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D, E, F, G, H, I = (0x10000000 * i for i in range(1, 10))   # fake device addresses, far apart


@pytest.fixture(scope="module")
def q4mm():
    import quantized_matmul_q4_gb300 as m
    return m


@pytest.mark.parametrize("tokens,heads", [(2 ** 24, 256), (2 ** 30, 4), (0x7FFFFE00, 4), (2 ** 15, 65536)])
def test_rows_of_a_key_head_stay_below_32_bits(q4mm, tokens, heads):
    """tokens·heads / kvHeads rows share a key head and are numbered in 32 bits; queries may be broadcast, so that as many
    fit in memory."""
    kv = 1 if heads == 65536 else 2
    with pytest.raises(q4mm.Q4mmError) as e:
        q4mm.mx_attention_ptr((H, 0, 0), 1, (A, B, C, D, 4, kv, 16, 32, 8), (E, F, G, 1, 4), 0.125, 1, (I, 32 * heads, 32),
                              tokens, heads)
    assert e.value.code == DIM and "rows" in q4mm.last_error(), q4mm.last_error()
    assert q4mm.library().mx_attention_workspace(kv, 16, 32, 1, 4, tokens, heads) == 0


@pytest.fixture(scope="module")
def limits(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("att_limits") / "libatt_limits.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    f"-I{os.path.join(ROOT, 'quantized_matmul_q4_gb300', 'csrc')}",
                    os.path.join(ROOT, "tests", "attention_limits_shim.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.att_chain.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 7 + [ctypes.POINTER(ctypes.c_int)]
    return lib


def test_keys_of_a_table_leave_room_for_a_tile_in_32_bits(limits):
    """The kernels round the number of keys up to whole tiles, and look a tile ahead, in 32-bit integers."""
    for width, page in ((2 ** 31 - 1, 2 ** 24), (128, 2 ** 24), (129, 2 ** 24), (2 ** 27, 16), (2 ** 27 - 1, 16), (2 ** 31 - 1, 16)):
        assert limits.att_table_keys(width, page) + 2 * limits.att_tile_keys() <= 2 ** 31
    assert limits.att_table_keys(127, 2 ** 24) == 127 * 2 ** 24 and limits.att_table_keys(0, 16) == 0


def test_sums_of_16_bit_rows_have_a_bounded_number_of_steps(limits):
    """However long a table, a tensor-core sum of 16 keys a step has no more steps than drop a third of half a step of the
    output, or the rows take the form for fp32; where all fits, plans are as without the bound."""
    out, free = (ctypes.c_int * 7)(), (ctypes.c_int * 7)()
    for bf16 in (0, 1):
        chain = limits.att_chain_of(bf16)
        assert chain * 1.7e-8 < 2.0 ** (-9 if bf16 else -12) / 3
        for tokens, group, seqs, kv in ((1, 1, 1, 1), (1, 8, 1, 1), (64, 4, 64, 8), (2048, 4, 1, 8), (8192, 1, 1, 32), (152, 2, 152, 2), (65536, 4, 1, 8)):
            for keys in (1000, 60000, 131072, 2 ** 19, 2 ** 20, 3000000, 2 ** 23, 2 ** 26, 2 ** 31 - 1):
                limits.att_chain(tokens, group, seqs, kv, -(-keys // 16), 16, chain, 152, out)
                limits.att_chain(tokens, group, seqs, kv, -(-keys // 16), 16, 0, 152, free)
                many, split, many32, _, cluster, parts, few32 = out
                assert few32 or -(-keys // 16) <= chain * 8 * cluster * parts
                assert many32 or -(--(-keys // 128) // split) * 8 <= chain
                if keys <= 16 * chain:
                    assert list(out) == list(free) and not many32 and not few32
                assert not free[2] and not free[6]


def test_a_cache_of_no_heads_is_refused(monkeypatch):
    """Queries of any number of heads have no key heads there."""
    import torch
    import quantized_matmul_q4_gb300 as q
    from quantized_matmul_q4_gb300 import _binding as b
    b._Torch.load()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)     # (no call here reaches a launch)
    monkeypatch.setattr(b._Torch, "current_device", lambda: 0)
    monkeypatch.setattr(b._Torch, "raw_stream", lambda device: 0)
    monkeypatch.setattr(b, "_LIB", None)
    codes, scales = torch.zeros(4, 0, 16, 64, dtype=torch.uint8), torch.zeros(4, 0, 16, 4, dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)
    batch = torch.tensor([0, 3], **i32), torch.tensor([3], **i32), torch.zeros(1, 2, **i32)
    with pytest.raises(ValueError):
        q.mx_attention(torch.zeros(3, 4, 64), q.MxCache(codes, scales, codes, scales, 64, 8), *batch)
