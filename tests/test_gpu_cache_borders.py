"""Keys that the rotation takes beside the borders of the cache's scales, and keys of position 0, against their exact values.

What is held: where values 2^-25 to both sides of the exact one (the angles and what is made of them are good to 2^-26)
have the same scale byte and code, those are the ones written.
"""
import numpy as np
import pytest
import attention_reference as ref
import mx_reference as mx
import test_gpu_attention as base
from test_gpu_attention import Case, _q
pytestmark = pytest.mark.gpu


def _held(c, cache, want, bits, D):
    """Scale bytes and codes of k are those of the exact values, wherever those of values 2^-25 to both sides are alike.
    Returns how many blocks and codes the fp32 arithmetic, 2^-22 to both sides, leaves open."""
    codes, scales = cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy()
    open_blocks = open_codes = 0
    for t, _, _, pg, at in ref.places(c.batch, c.page):
        w = want[t, 0]
        def byte(e):
            return ref.head_codes(w * (1 + e), bits)[1][:D // 32]
        sure = byte(-2.0 ** -25) == byte(2.0 ** -25)
        assert np.array_equal(scales[pg, 0, at][:D // 32][sure], byte(0)[sure]), t
        open_blocks += int((sure & (byte(-2.0 ** -22) != byte(2.0 ** -22))).sum())
        unit = np.repeat(np.exp2(byte(0).astype(float) - 127), 32)
        got = mx.unpack(codes[pg, 0, at][None], bits)[0]
        lo, hi = (mx.nearest_code(w * (1 + e) / unit, bits) for e in (-2.0 ** -25, 2.0 ** -25))
        mine = np.repeat(sure, 32) & (lo == hi)
        assert np.array_equal(got[mine], lo[mine]), (t, np.flatnonzero(mine & (got != lo)))
        wide = [mx.nearest_code(w * (1 + e) / unit, bits) for e in (-2.0 ** -22, 2.0 ** -22)]
        open_codes += int((mine & (wide[0] != wide[1])).sum())
    return open_blocks, open_codes


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("magnitude", [1.0, 1.1])
@pytest.mark.parametrize("R,interleaved,D", [(128, False, 128), (128, True, 128), (64, False, 64), (72, False, 96)])
def test_largest_values_beside_powers_of_two(R, interleaved, D, magnitude, bits):
    """A block's largest value, taken by the rotation to within a unit or two of a power of two, gives the block the scale,
    and hence the codes, of the exact value."""
    q = _q()
    T = 150
    c = Case(R + bits, [T], [T + 3000], 1, D, 16, bits)
    pos = np.arange(3000, 3000 + T)
    f = q.rope_frequencies(R)
    a = pos[:, None] * f.cpu().numpy()
    x = c.rng.uniform(-0.3, 0.3, (T, 1, D))
    pairs = [((2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)) for i in range(R // 2)]
    for t in range(T):
        for block in range(R // 32):
            mine = [(i, s) for i, p in enumerate(pairs) for s in (0, 1) if p[s] // 32 == block and abs(np.cos(a[t, i])) > 0.78
                    and (x[t, 0, list(p)] != 0).all()]
            if mine:        # its partner becomes tan(a), at most 0.81
                i, s = mine[c.rng.integers(len(mine))]
                x[t, 0, list(pairs[i])] = 0
                x[t, 0, pairs[i][s]] = (1 + c.rng.integers(-3, 4) * 2.0 ** -25) / (magnitude * np.cos(a[t, i]))
    k, kv = base._dev(x, "float32")
    cache, batch = c.device_cache(), c.device_batch()
    q.mx_cache_write(cache, k, k, *batch, rope=q.Rope(f, interleaved, magnitude))
    want = ref.turned(kv, pos, f.cpu().numpy(), interleaved, float(np.float32(magnitude)))
    blocks, _ = _held(c, cache, want, bits, D)
    assert blocks > T // 2      # these are what is tested


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R,interleaved,D", [(128, False, 128), (64, True, 128), (36, False, 96), (64, False, 64)])
def test_position_zero_with_a_magnitude(R, interleaved, D, bits):
    """Keys of position 0 are multiplied by the magnitude, which may take them beside a border as any angle does."""
    q = _q()
    n = 150
    c = Case(R + bits, [1] * n, [1] * n, 1, D, 16, bits)
    steps = 16 if bits == 8 else 4
    m = float(np.float32(1.1))
    x = (1 + (2 * c.rng.integers(0, steps // 2, (n, 1, D)) + 1) / steps) / m
    x[..., ::16] = 3.9 / m
    k, kv = base._dev(x, "float32")
    cache, batch = c.device_cache(), c.device_batch()
    f = q.rope_frequencies(R)
    q.mx_cache_write(cache, k, k, *batch, rope=q.Rope(f, interleaved, 1.1))
    want = kv.copy()
    want[..., :R] *= m
    _, codes = _held(c, cache, want, bits, D)
    assert codes > n * R // 16
