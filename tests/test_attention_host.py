"""Attention operators without a GPU: the tests' 64-bit restatement against
values worked out by hand, how the kernels' work is split, the numbering of
row tiles, and the refusals of the C ABI and of the Python calls."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import attention_reference as ref

DIM, NULL, ALIGN, ALIAS = -1, -2, -3, -6
A, B, C, D, E, F, G, H, I, J = (0x10000000 * i for i in range(1, 11))   # fake device addresses, far apart
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def q4mm():
    import quantized_matmul_q4_gb300 as m
    return m


@pytest.fixture(scope="module")
def geo(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("att_geo") / "libatt_geo.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC",
                    f"-I{os.path.join(ROOT, 'quantized_matmul_q4_gb300', 'csrc')}",
                    os.path.join(ROOT, "tests", "attention_geometry_shim.cpp"), "-o", out], check=True)
    lib = ctypes.CDLL(out)
    lib.att_geo.argtypes = [ctypes.c_longlong] + [ctypes.c_int] * 7 + [ctypes.POINTER(ctypes.c_int)]
    return lib


# The restatement.

def test_turned_pairs():
    x = np.arange(1.0, 7).reshape(1, 1, 6)
    quarter = [np.pi / 2, np.pi]
    assert np.allclose(ref.turned(x, [1], quarter), [[[-3, -2, 1, -4, 5, 6]]])           # pairs (1, 3), (2, 4)
    assert np.allclose(ref.turned(x, [1], quarter, interleaved=True), [[[-2, 1, -3, -4, 5, 6]]])
    assert np.allclose(ref.turned(x, [-1], quarter, magnitude=2), [[[6, -4, -2, -8, 5, 6]]])


def test_places_of_a_batch():
    batch = (np.array([0, 2, 2, 5]), np.array([17, 4, 2]), np.array([[3, 9], [7, 0], [1, 0]]))
    assert list(ref.places(batch, 16)) == [(0, 0, 15, 3, 15), (1, 0, 16, 9, 0), (3, 2, 0, 1, 0), (4, 2, 1, 1, 1)]


def test_attention_by_hand():
    """One head of 32 values, two keys of 8-bit ones and twos: scores 0 and ln 3."""
    cache = {w + "_codes": np.zeros((1, 1, 16, 32), np.uint8) for w in "kv"}
    cache |= {w + "_scales": np.zeros((1, 1, 16, 4), np.uint8) for w in "kv"}
    cache["k_codes"][0, 0, 1, 0], cache["k_scales"][0, 0, :, 0] = 0x38, 127          # k[1] = (1, 0, ...)
    cache["v_codes"][0, 0, 0, 5], cache["v_codes"][0, 0, 1, 5], cache["v_scales"][0, 0, :, 0] = 0x38, 0x40, 127
    q = np.zeros((2, 1, 32))
    q[:, 0, 0] = 2 * np.log(3)
    batch = (np.array([0, 2]), np.array([2]), np.array([[0]]))
    y = ref.attention(q, cache, batch, 8, 0.5)[0]
    assert np.allclose(y[:, 0, 5], [1, 0.25 * 1 + 0.75 * 2]) and np.allclose(np.delete(y[:, 0], 5, 1), 0)
    assert np.allclose(ref.attention(q, cache, batch, 8, 0.5, causal=False)[0][0, 0, 5], 1.75)


def test_frequencies_refuse_what_they_cannot_be(q4mm):
    for kw in (dict(dim=0), dict(dim=7), dict(dim=64, scaling="x"), dict(dim=64, scaling="parts"), dict(dim=64, base=0),
               dict(dim=64, scaling="linear", factor=0), dict(dim=2, scaling="ntk", factor=2),
               dict(dim=64, scaling="parts", original=4096, fast=1, slow=2)):
        with pytest.raises(ValueError):
            q4mm.rope_frequencies(**kw, device="cpu")
    assert abs(q4mm.rope_magnitude(8) - (0.1 * np.log(8) + 1)) < 1e-15 and q4mm.rope_magnitude(0.5) == 1


# How the work is split.

def test_few_rows_split(geo):
    out = (ctypes.c_int * 6)()
    for sms, f32 in ((1, 0), (132, 1), (152, 0), (152, 1)):
        for tokens, seqs in ((1, 1), (1, 3), (2, 50), (64, 64), (300, 7), (5, 5), (8192, 1000), (1, 2 ** 24)):
            for group in (1, 4, 7, 16):
                for kv in (1, 5, 8, 32):
                    for width, page in ((1, 16), (63, 16), (40, 48), (8192, 16), (2 ** 21, 4096), (0, 16)):
                        geo.att_geo(tokens, group, seqs, kv, width, page, f32, sms, out)
                        nr, tiles, cluster, parts, _, split = out
                        assert split in (1, 2, 3, 4, 5, 6, 8) and split <= max(1, -(-min(width * page, 0x7FFFFFFF) // 128))
                        assert nr in (1, 2) and tiles == tokens * group // (8 * nr) + seqs
                        assert nr == 1 or tokens * group > 8 * seqs
                        assert cluster in (1, 2, 3, 4, 5, 6, 8) and parts >= 1 and (parts == 1 or cluster == 8)
                        groups = min(width * page, 0x7FFFFFFF) // 16
                        if parts > 1:   # a group a warp, and all of them resident; what is shared in vain costs
                            some = min(tokens, seqs)
                            even = some * -(-tokens * group // (8 * nr * some))
                            assert cluster * parts * 8 <= groups and even * kv * cluster * parts <= 2 * sms
                            assert (tokens * group // 8 + seqs) * kv < 64   # where the Python call asks for a workspace
                        if groups <= 8:
                            assert cluster == 1


def test_which_kernel(geo):
    out = (ctypes.c_int * 6)()
    for tokens, group, seqs, kv, keys, f32, many, split in (
            (1, 1, 1, 32, 1000, 0, 0, None), (64, 1, 64, 32, 4096, 0, 0, None), (1, 8, 1, 1, 2 ** 20, 0, 0, None),
            (8192, 1, 1, 32, 8192, 0, 1, 1), (512, 8, 1, 4, 8192, 0, 1, 2), (2000, 4, 1, 8, 2000, 0, 1, None), (200, 4, 1, 1, 500, 0, 0, None),
            (64, 4, 8, 8, 30000, 0, 0, None), (96, 4, 8, 8, 30000, 0, 1, 2), (2000, 4, 1, 8, 2000, 1, 1, None)):
        geo.att_geo(tokens, group, seqs, kv, -(-keys // 16), 16, f32, 152, out)
        assert out[4] == many and (split is None or out[5] == split), (tokens, group, seqs, kv, keys, list(out))


def test_numbers_of_row_tiles():
    """Tiles of sequence i start at floor(starts[i]·group / R) + i: room for its rows, and none beyond the last."""
    r = np.random.default_rng(0)
    for _ in range(200):
        R, group, n = int(r.choice([8, 16, 128, 256])), int(r.integers(1, 9)), int(r.integers(1, 12))
        news = r.integers(0, int(r.choice([2, 40, 700])), n)
        starts = np.concatenate([[0], np.cumsum(news)])
        first = [int(s) * group // R + i for i, s in enumerate(starts)]
        for i in range(n):
            assert first[i + 1] - first[i] >= -(-int(news[i]) * group // R)
        assert first[n] <= int(starts[n]) * group // R + n


# Refusals of the C ABI, before any CUDA call.

def _refused(q4mm, code, fn, *args, word=None):
    with pytest.raises(q4mm.Q4mmError) as e:
        fn(*args)
    assert e.value.code == code, q4mm.last_error()
    if word:
        assert word in q4mm.last_error()


def _cache(pages=4, heads=2, page=16, dim=64, bits=8, at=(A, B, C, D)):
    return (*at, pages, heads, page, dim, bits)


def _batch(n=1, width=4, at=(E, F, G)):
    return (*at, n, width)


X = (H, 128, 64)      # 2 heads of 64 a token
Y = (I, 128, 64)


def test_rope_is_refused(q4mm):
    def rope(x=X, dtype=0, positions=A, wide=0, frequencies=B, rotated=64, magnitude=1.0, out=Y, tokens=3, heads=2, dim=64):
        return (x, dtype, positions, wide, frequencies, rotated, 0, magnitude, out, tokens, heads, dim)
    fn = q4mm.rope_rotate_ptr
    for bad, word in ((dict(rotated=63), "rotated"), (dict(rotated=66), "rotated"), (dict(rotated=-2), "rotated"),
                      (dict(dtype=3), "type"), (dict(dim=0), "headDim"), (dict(dim=257), "headDim"), (dict(heads=0), "heads"),
                      (dict(tokens=-1), "tokens"), (dict(magnitude=float("inf")), "magnitude"),
                      (dict(magnitude=float("nan")), "magnitude"), (dict(x=(H, -1, 64)), "strides"),
                      (dict(x=(H, 2 ** 60, 64)), "fit")):
        _refused(q4mm, DIM, fn, *rope(**bad), word=word)
    for bad in (dict(x=(0, 128, 64)), dict(positions=0), dict(frequencies=0), dict(out=(0, 128, 64))):
        _refused(q4mm, NULL, fn, *rope(**bad))
    for bad in (dict(x=(H + 2, 128, 64)), dict(positions=A + 2), dict(positions=A + 4, wide=1), dict(frequencies=B + 4),
                dict(out=(I + 1, 128, 64), dtype=2)):
        _refused(q4mm, ALIGN, fn, *rope(**bad))
    # out a part of x, shifted; out whose heads lie on each other; out over the positions.
    for bad in (dict(out=(H + 4, 128, 64)), dict(out=(I, 128, 63)), dict(out=(I, 100, 64)), dict(out=(A, 128, 64))):
        _refused(q4mm, ALIAS, fn, *rope(**bad))


CALLS = {
    "write": lambda q, c=None, b=None, k=X, v=Y, dtype=0, tokens=3, rotated=0, frequencies=0: q.mx_cache_write_ptr(
        k, v, dtype, frequencies, rotated, 0, 1.0, c or _cache(), b or _batch(), tokens),
    "read": lambda q, c=None, b=None, k=X, v=Y, dtype=0, tokens=3: q.mx_cache_read_ptr(
        c or _cache(), b or _batch(), k, v, dtype, tokens),
    "attention": lambda q, c=None, b=None, k=X, v=Y, dtype=0, tokens=3, scale=0.125, heads=2, ws=(0, 0): q.mx_attention_ptr(
        k, dtype, c or _cache(), b or _batch(), scale, 1, v, tokens, heads, *ws),
}


@pytest.mark.parametrize("name", CALLS)
def test_cache_calls_are_refused(q4mm, name):
    def call(**kw):
        CALLS[name](q4mm, **kw)
    def refused(code, word=None, **kw):
        _refused(q4mm, code, lambda: call(**kw), word=word)
    for kw, word in ((dict(dim=48), "headDim"), (dict(dim=160), "headDim"), (dict(dim=0), "headDim"), (dict(bits=6), "bits"),
                     (dict(page=8), "pageTokens"), (dict(page=24), "pageTokens"), (dict(page=0), "pageTokens"),
                     (dict(pages=0), "pages"), (dict(heads=0), "kvHeads")):
        refused(DIM, word, c=_cache(**kw))
    refused(DIM, "type", dtype=4)
    refused(DIM, "sequences", b=_batch(n=-1))
    refused(DIM, "tableWidth", b=_batch(width=-1))
    refused(DIM, "tokens", tokens=-3)
    refused(DIM, "strides", k=(H, -128, 64))
    for i in range(4):
        at = [A, B, C, D]
        at[i] = 0
        refused(NULL, c=_cache(at=at))
        at[i] = (A, B, C, D)[i] + 8
        refused(ALIGN, c=_cache(at=at))
    for i in range(3):
        at = [E, F, G]
        at[i] = 0
        refused(NULL, b=_batch(at=at))
        at[i] = (E, F, G)[i] + 2
        refused(ALIGN, b=_batch(at=at))
    refused(NULL, k=(0, 128, 64))
    refused(NULL, v=(0, 128, 64))
    refused(ALIGN, k=(H + 2, 128, 64))
    refused(ALIGN, v=(I + 1, 128, 64), dtype=1)
    # What is written lies on what is read: 4 pages of 2 heads of 16 tokens of 64 bytes are 8192.
    refused(ALIAS, k=(A + 8188, 128, 64), v=(A + 8188, 128, 64))
    if name != "write":
        refused(ALIAS, v=(E, 128, 64))
        refused(ALIAS, v=(I, 128, 32))       # heads on each other
    if name == "read":
        refused(ALIAS, k=(I + 64, 128, 64))
    if name == "attention":
        for scale in (-1.0, float("nan"), float("inf")):
            refused(DIM, "scale", scale=scale)
        refused(DIM, "heads", heads=3)
        refused(DIM, "heads", heads=0)
        refused(ALIAS, v=(H + 64, 128, 64))
        refused(NULL, ws=(0, 1024))
        refused(ALIGN, ws=(J + 8, 1024))
        for at in (A, H, I + 16, G):
            refused(ALIAS, ws=(at, 1024))


def test_workspace_of_nothing(q4mm):
    lib = q4mm.library()
    for args in ((0, 16, 64, 1, 4, 1, 2), (2, 0, 64, 1, 4, 1, 2), (2, 16, 64, 0, 4, 1, 2), (2, 16, 64, 1, -4, 1, 2),
                 (2, 16, 64, 1, 4, 0, 2), (2, 16, 64, 1, 4, 1, 3), (2, 16, 64, 1, 4, 100, 2)):
        assert lib.mx_attention_workspace(*args) == 0


def test_symbols_take_the_declared_arguments(q4mm):
    lib = q4mm.library()
    for name, n in (("rope_rotate", 17), ("mx_cache_write", 27), ("mx_cache_read", 23), ("mx_attention", 28)):
        fn = getattr(lib, name)
        assert len(fn.argtypes) == n and fn.restype is ctypes.c_int


def test_packed_calls_check_the_same(q4mm):
    """The calls with their arguments in words: each bad one is refused as it is by the call itself."""
    import struct
    lib = q4mm.library()
    def pack(fmt, *a):
        return struct.pack(fmt, *a)
    rope = ["=9qd7q", H, 128, 64, 0, A, 0, B, 64, 0, 1.0, I, 128, 64, 3, 2, 64, 0]
    write = ["=10qd16q", H, 128, 64, I, 128, 64, 0, 0, 0, 0, 1.0, A, B, C, D, 4, 2, 16, 64, 8, E, F, G, 1, 4, 3, 0]
    read = ["=23q", A, B, C, D, 4, 2, 16, 64, 8, E, F, G, 1, 4, H, 128, 64, I, 128, 64, 0, 3, 0]
    att = ["=18qd9q", H, 128, 64, 0, A, B, C, D, 4, 2, 16, 64, 8, E, F, G, 1, 4, 0.125, 1, I, 128, 64, 3, 2, 0, 0, 0]
    for which, words, bad in (
            (0, rope, ((0, 0, NULL, "x"), (1, -1, DIM, "strides"), (3, 7, DIM, "type"), (4, A + 2, ALIGN, "positions"), (6, 0, NULL, "frequencies"),
                       (7, 66, DIM, "rotated"), (9, float("inf"), DIM, "magnitude"), (10, 0, NULL, "out"), (12, 32, ALIAS, "out"),
                       (13, -5, DIM, "tokens"), (14, 0, DIM, "heads"), (15, 500, DIM, "headDim"), (13, 2 ** 40, DIM, "tokens"))),
            (1, write, ((0, 0, NULL, "k"), (3, 0, NULL, "v"), (6, 9, DIM, "type"), (8, 3, DIM, "rotated"), (10, float("nan"), DIM, "magnitude"),
                        (11, 0, NULL, "k_codes"), (14, D + 4, ALIGN, "v_scales"), (15, 0, DIM, "pages"), (16, 0, DIM, "kvHeads"), (17, 20, DIM, "pageTokens"),
                        (18, 65, DIM, "headDim"), (19, 5, DIM, "bits"), (20, 0, NULL, "starts"), (21, 0, NULL, "lengths"), (22, 0, NULL, "table"),
                        (23, -1, DIM, "sequences"), (24, -1, DIM, "tableWidth"), (25, -1, DIM, "tokens"))),
            (2, read, ((3, 0, NULL, "v_scales"), (8, 7, DIM, "bits"), (9, E + 1, ALIGN, "starts"), (12, -1, DIM, "sequences"), (14, 0, NULL, "k"), (17, H, ALIAS, "overlap"),
                       (20, 5, DIM, "type"), (21, -1, DIM, "tokens"))),
            (3, att, ((0, 0, NULL, "q"), (3, 3, DIM, "type"), (4, 0, NULL, "k_codes"), (12, 3, DIM, "bits"), (15, 0, NULL, "table"), (17, -2, DIM, "tableWidth"),
                      (18, -0.5, DIM, "scale"), (20, 0, NULL, "y"), (22, 32, ALIAS, "y"), (23, -1, DIM, "tokens"), (24, 5, DIM, "heads"), (26, 64, NULL, "workspace")))):
        for at, value, code, word in bad:
            w = words.copy()
            w[1 + at] = value
            assert lib.q4mm_call(which, pack(*w)) == code, (which, at, q4mm.last_error())
            assert word in q4mm.last_error(), (which, at, q4mm.last_error())
    assert lib.q4mm_call(9, b"") == DIM and lib.q4mm_call(0, None) == NULL


# Refusals of the Python calls.

@pytest.fixture
def q(monkeypatch):
    """The package, for CPU tensors that pass for those of device 0 (no call here reaches a launch)."""
    import torch
    import quantized_matmul_q4_gb300 as m
    from quantized_matmul_q4_gb300 import _binding as b
    b._Torch.load()
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(b._Torch, "current_device", lambda: 0)
    monkeypatch.setattr(b._Torch, "raw_stream", lambda device: 0)
    monkeypatch.setattr(b, "_LIB", None)
    return m


def test_python_refuses(q):
    import torch
    def i32(*a):
        return torch.tensor(a, dtype=torch.int32)
    c = q.mx_cache(4, 2, 64, page=16, device="cpu")
    batch = (i32(0, 3), i32(3), i32(0, 1).view(1, 2))
    x, k = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    f = torch.ones(32, dtype=torch.float64)
    bad_caches = [c._replace(bits=4), c._replace(head_dim=32), c._replace(k_scales=c.k_scales[..., :2]),
                  c._replace(v_codes=c.v_codes[:3]), c._replace(k_codes=c.k_codes.int()), c._replace(v_scales=c.v_scales.char()),
                  c._replace(k_codes=c.k_codes.transpose(0, 1).contiguous().transpose(0, 1))]
    bad_batches = [(batch[0].long(), *batch[1:]), (i32(0), *batch[1:]), (*batch[:2], i32(0, 1)),
                   (*batch[:2], i32(0, 1, 2, 3).view(2, 2)), (batch[0], batch[1].view(1, 1), batch[2])]
    calls = []
    for cache, b in [(z, batch) for z in bad_caches] + [(c, z) for z in bad_batches]:
        calls += [lambda cache=cache, b=b: q.mx_attention(x, cache, *b), lambda cache=cache, b=b: q.mx_cache_write(cache, k, k, *b),
                  lambda cache=cache, b=b: q.mx_cache_read(cache, *b, tokens=3)]
    calls += [
        lambda: q.mx_attention(x[:, :3], c, *batch), lambda: q.mx_attention(x[..., :32], c, *batch),
        lambda: q.mx_attention(x.double(), c, *batch), lambda: q.mx_attention(x, c, *batch, out=x[:2]),
        lambda: q.mx_attention(x, c, *batch, out=x.half()), lambda: q.mx_attention(x[0], c, *batch),
        lambda: q.mx_attention(x.transpose(1, 2).contiguous().transpose(1, 2), c, *batch),
        lambda: q.mx_cache_write(c, k, k.half(), *batch), lambda: q.mx_cache_write(c, k, k[:2], *batch),
        lambda: q.mx_cache_write(c, x, x, *batch), lambda: q.mx_cache_write(c, k, k, *batch, rope=q.Rope(f.float())),
        lambda: q.mx_cache_write(c, k, k, *batch, rope=q.Rope(torch.ones(33, dtype=torch.float64))),
        lambda: q.mx_cache_read(c, *batch), lambda: q.mx_cache_read(c, *batch, out=(k, k.half())),
        lambda: q.mx_cache_read(c, *batch, out=(k, k[:2])), lambda: q.mx_cache_read(c, *batch, tokens=4, out=(k, k)),
        lambda: q.rope_rotate(x, i32(1, 2), q.Rope(f)), lambda: q.rope_rotate(x, i32(1, 2, 3).float(), q.Rope(f)),
        lambda: q.rope_rotate(x, i32(1, 2, 3), q.Rope(f), out=x.half()), lambda: q.rope_rotate(x[0], i32(1, 2, 3), q.Rope(f)),
        lambda: q.rope_rotate(x, i32(1, 2, 3), q.Rope(torch.ones(33, dtype=torch.float64))),
        lambda: q.mx_cache(4, 2, 48, device="cpu"), lambda: q.mx_cache(4, 2, 64, page=24, device="cpu"),
        lambda: q.mx_cache(0, 2, 64, device="cpu"), lambda: q.mx_cache(4, 2, 64, bits=5, device="cpu")]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"call {i} was taken")
