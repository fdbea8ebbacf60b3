"""Sizes of attention calls that its 32-bit row numbers and positions cannot hold: refused by the C ABI before any CUDA call."""
import pytest

DIM = -1
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
