"""Attention over larger caches, in company, after a time-out, and as a block.

Where a case is too large for the restatement value by value, the cache's
values are read back (which test_gpu_attention holds to the format) and the
formula is taken over them in float64 by torch; tolerances as derived there.
"""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _torch():
    import torch
    return torch


@pytest.fixture(autouse=True)
def kernel(request):
    """The attention kernel that a test's calls take: as planned, or the one that `KERNELS` says."""
    which = getattr(request, "param", None)
    if which:
        _q().force_attention_kernel(which)
    yield which
    if which:
        _q().force_attention_kernel(None)


KERNELS = pytest.mark.parametrize("kernel", ["few", "many"], indirect=True)
MANY = pytest.mark.parametrize("kernel", ["many"], indirect=True)


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def _i32(*a):
    return _torch().tensor(a, dtype=_torch().int32, device="cuda")


class Batch:
    """Sequences with a filled cache, the pages dealt at random."""

    def __init__(self, news, lengths, kv, D, page, bits, seed=0, width=None, scale=1.0):
        q, torch = _q(), _torch()
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.news, self.lens = news, lengths
        used = [-(-n // page) for n in lengths]
        order = torch.randperm(sum(used) + 3, generator=self.g, device="cuda").int()
        width = max(used) if width is None else width
        table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(used):
            table[i, :n] = order[at:at + n]
            at += n
        def ends(a):
            return _i32(*np.concatenate([[0], np.cumsum(a)]).tolist())
        self.cache = q.mx_cache(sum(used) + 3, kv, D, page=page, bits=bits)
        self.batch = ends(news), _i32(*lengths), table
        self.whole = ends(lengths), _i32(*lengths), table      # every cached token as a row
        n = sum(lengths)
        self.k, self.v = (scale * torch.randn(n, kv, D, generator=self.g, device="cuda") for _ in "kv")
        q.mx_cache_write(self.cache, self.k, self.v, *self.whole)

    def queries(self, heads, dtype, size=1.5):
        torch = _torch()
        shape = (sum(self.news), heads, self.cache.head_dim)
        return (size * torch.randn(shape, generator=self.g, device="cuda")).to(getattr(torch, dtype))

    def check(self, x, y, causal=True):
        q, torch = _q(), _torch()
        D, name = self.cache.head_dim, str(x.dtype)[6:]
        k, v = (t.double() for t in q.mx_cache_read(self.cache, *self.whole, tokens=sum(self.lens)))
        group = x.shape[1] // k.shape[1]
        at = row = 0
        for n, m in zip(self.news, self.lens):
            last = torch.arange(m - n, m, device="cuda") if causal else torch.full((n,), m - 1, device="cuda")
            hidden = torch.arange(m, device="cuda") > last[:, None]
            for h in range(x.shape[1]):
                qh, kh, vh = x[row:row + n, h].double(), k[at:at + m, h // group], v[at:at + m, h // group]
                s = (qh @ kh.T * D ** -0.5).masked_fill(hidden, -float("inf"))
                p = torch.softmax(s, -1)
                want, spread = p @ vh, p @ vh.abs()
                A = (qh.abs() @ kh.abs().T * D ** -0.5).amax(-1, keepdim=True)
                e = ((D / 16 + 8) * A + 1.45 * A + 160) * 2.0 ** -23 * np.log(2) + 2.0 ** -21
                e = 2 * e + (m / 16 + 30) * 2.0 ** -23 + (2.0 ** -22 + 2.0 ** -21 * A if name == "float32" else 2.0 ** -11)
                most = (p * vh.abs().amax(-1)).amax(-1, keepdim=True)
                f = torch.finfo(x.dtype)
                bound = e * spread + m * 2.0 ** -30 * most + f.eps / 2 * want.abs() * 1.01 + f.smallest_normal * f.eps / 2
                off = (y[row:row + n, h].double() - want).abs() - bound
                assert float(off.max()) <= 0, (h, float(off.max()), float(want.abs().max()))
            at, row = at + m, row + n


LARGE = [  # new tokens, lengths, kv heads, group, D, page, bits
    ([1], [40000], 1, 8, 128, 16, 8), ([1], [70001], 2, 1, 64, 64, 4), ([1], [30000], 3, 2, 96, 48, 8),
    ([1, 1, 1], [9000, 1, 300], 2, 4, 128, 16, 8), ([2], [33000], 1, 7, 128, 128, 4), ([1] * 40, [17 * i + 1 for i in range(40)], 4, 1, 128, 32, 8),
    ([520], [4100], 2, 1, 128, 16, 8), ([33], [20000], 1, 4, 128, 64, 4), ([1000, 7, 333], [1000, 2000, 333], 2, 2, 64, 32, 8),
    ([2049], [2049], 1, 1, 128, 64, 8), ([700], [1500], 2, 3, 96, 16, 4), ([257], [5000], 1, 1, 128, 128, 8)]


@KERNELS
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("news,lengths,kv,group,D,page,bits", LARGE)
def test_large(news, lengths, kv, group, D, page, bits, dtype):
    q = _q()
    b = Batch(news, lengths, kv, D, page, bits, seed=len(news) + D)
    x = b.queries(kv * group, dtype)
    y = q.mx_attention(x, b.cache, *b.batch)
    q.device_status()
    b.check(x, y)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_workspace_of_any_size(dtype):
    """Without a workspace, or with too little, a call is slower, not wrong; nothing beyond it is written."""
    q, torch = _q(), _torch()
    b = Batch([1], [50000], 1, 64, 64, 8)
    x = b.queries(4, dtype)
    need = q.library().mx_attention_workspace(1, 64, 64, 1, b.batch[2].shape[1], 1, 4)
    assert need > 0
    code = {"float32": 0, "bfloat16": 2}[dtype]
    c = b.cache
    for nbytes in (0, 16, need // 2 // 16 * 16, need, need + 4096):
        ws = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        y = torch.empty_like(x)
        q.mx_attention_ptr((x.data_ptr(), 256, 64), code, (*[t.data_ptr() for t in c[:4]], *c.k_codes.shape[:3], 64, 8),
                           (*[t.data_ptr() for t in b.batch], 1, b.batch[2].shape[1]), 0.125, 1, (y.data_ptr(), 256, 64), 1, 4,
                           ws.data_ptr() if nbytes else 0, nbytes, torch.cuda.current_stream().cuda_stream)
        b.check(x, y)
        assert (ws[nbytes:] == 0x5A).all()
    q.device_status()


@KERNELS
def test_long_fp32_sums_do_not_drift(kernel):
    """Values of one over 60000 keys that no other CTA shares: outputs are one, and not always short of it.  A tensor-core
    sum drops at most a step, 2^-23, each of the 33 times that it is added to, and fp32 additions round by
    chance: over 16 rows and 60000 / 128 additions by sqrt(470) 2^-24 / 4 = 3.2e-7 on average."""
    q, torch = _q(), _torch()
    b = Batch([60000], [60000], 2, 64, 16, 8)
    ones = torch.ones(60000, 2, 64, device="cuda")
    q.mx_cache_write(b.cache, b.k, ones, *b.whole)
    x = torch.randn(200, 8, 64, generator=b.g, device="cuda")
    y = q.mx_attention(x, b.cache, torch.arange(201, dtype=torch.int32, device="cuda"), b.batch[1].expand(200).contiguous(),
                       b.batch[2].expand(200, -1).contiguous())
    q.device_status()
    assert abs(float((y.double() - 1).mean())) < 33 * 2.0 ** -23 + 3.2e-7
    assert float((y.double() - 1).abs().max()) < 2 * (33 + 60000 / 128) * 2.0 ** -23


@KERNELS
def test_a_sequence_alone_and_among_others():
    """A row's bits do not depend on the sequences beside it, as long as the keys are shared alike."""
    q, torch = _q(), _torch()
    for news, lengths in (([1, 1, 1], [700, 33, 1290]), ([140, 200], [300, 260])):
        b = Batch(news, lengths, 2, 128, 32, 8, width=64)
        x = b.queries(4, "bfloat16")
        together = q.mx_attention(x, b.cache, *b.batch)
        at = 0
        for i, n in enumerate(news):
            alone = q.mx_attention(x[at:at + n], b.cache, _i32(0, n), b.batch[1][i:i + 1].contiguous(), b.batch[2][i:i + 1].contiguous())
            assert float((together[at:at + n].float() - alone.float()).abs().max()) <= 2.0 ** -7 * float(alone.float().abs().max())
            at += n
        b.check(x, together)


@KERNELS
def test_new_tokens_in_any_chunks():
    """A prompt written and attended to in chunks gives, to the tolerance of both, what it gives at once."""
    q, torch = _q(), _torch()
    b = Batch([600], [600], 2, 128, 32, 8)
    x = b.queries(8, "float32")
    at_once = q.mx_attention(x, b.cache, *b.batch)
    other = q.mx_cache(*b.cache.k_codes.shape[:2], 128, page=32)
    at = 0
    for n in (1, 2, 40, 257, 3, 1, 200, 96):
        batch = _i32(0, n), _i32(at + n), b.batch[2]
        q.mx_cache_write(other, b.k[at:at + n], b.v[at:at + n], *batch)
        y = q.mx_attention(x[at:at + n], other, *batch)
        assert float((y - at_once[at:at + n]).abs().max()) < 2e-5
        at += n
    assert at == 600
    for s, t in zip(b.cache[:4], other[:4]):
        assert torch.equal(s, t)


@KERNELS
def test_streams_at_once():
    """Calls on four streams at once, parted ones with a workspace each among them, one on top of the next."""
    q, torch = _q(), _torch()
    sets = [(Batch([1], [30000 + i], 1, 64, 64, 8, seed=i), 4) for i in range(2)] + [(Batch([300], [900 + i], 2, 128, 16, 8, seed=i), 2) for i in range(2)]
    xs = [b.queries(h, "bfloat16") for b, h in sets]
    want = [q.mx_attention(x, b.cache, *b.batch) for (b, _), x in zip(sets, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[] for _ in sets]
    for _ in range(20):
        for i, ((b, _), x, s) in enumerate(zip(sets, xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(q.mx_attention(x, b.cache, *b.batch))
    torch.cuda.synchronize()
    q.device_status()
    for w, g in zip(want, got):
        assert all(torch.equal(w, y) for y in g)


def test_two_graphs_of_parted_calls():
    """Two captured calls that take workspaces, replayed at once on two streams and again."""
    q, torch = _q(), _torch()
    made = []
    for i in range(2):
        b = Batch([1], [25000 + 16 * i], 1, 128, 16, 8, seed=i)
        x = b.queries(8, "bfloat16")
        want = q.mx_attention(x, b.cache, *b.batch)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = q.mx_attention(x, b.cache, *b.batch)
        made.append((b, x, want, graph, y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for *_, graph, y, stream in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, want, _, y, _ in made:
        assert torch.equal(want, y)


@MANY
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("news,lengths,bits", [([300], [900], 8), ([200, 100], [200, 4000], 4)])
def test_wait_runs_out_then_next_call_is_right(news, lengths, bits, dtype):
    import time
    q, torch = _q(), _torch()
    b = Batch(news, lengths, 2, 128, 32, bits)
    x = b.queries(4, dtype)
    q.device_status()
    for stage in (0, 1):
        q.arm_wait_failure(stage, 2_000_000)
        t0 = time.perf_counter()
        q.mx_attention(x, b.cache, *b.batch)
        torch.cuda.synchronize()
        assert time.perf_counter() - t0 < 1.0
        with pytest.raises(q.Q4mmError) as e:
            q.device_status()
        assert e.value.code == -5
        y = q.mx_attention(x, b.cache, *b.batch)
        q.device_status()
        b.check(x, y)


def _example():
    spec = importlib.util.spec_from_file_location("llama_attention_mx", os.path.join(ROOT, "examples", "llama_attention_mx.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("heads,kv,bits", [(4, 4, 8), (8, 2, 8), (4, 1, 4)])
def test_the_block_stage_by_stage(heads, kv, bits):
    """The example's block: each stage from what the one before it left, in float64; chunks and single tokens alike."""
    q, torch, m = _q(), _torch(), _example()
    weights, x, r = m.make(heads, kv, 64, 150, seed=heads, dtype=torch.float32)
    block = m.MxAttention(**weights, head_dim=64, pages=14, page=16, bits=bits)
    table = torch.randperm(14, device="cuda").int()[None, :10].contiguous()
    pos = torch.arange(150, dtype=torch.int32, device="cuda")
    y, h = block(x, r, pos, _i32(0, 150), _i32(150), table)
    n, h2 = q.mx_rmsnorm(x, weights["norm"], residual=r)
    assert torch.equal(h, h2)
    qkv = (q.mx_dequantize(n).double() @ q.mx_dequantize(block.qkv).double().T).view(150, -1, 64)
    a = pos.double()[:, None] * block.rope.frequencies
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = qkv[:, :heads + kv].chunk(2, -1)
    turned = torch.cat((lo * c - hi * s, hi * c + lo * s), -1)
    ck, cv = (t.double() for t in q.mx_cache_read(block.cache, _i32(0, 150), _i32(150), table, tokens=150))
    # A code is off by at most half a step, 2^-4 or 2^-2 of the value, or by its cut: of a block's largest, which is below
    # 512 (8) scales, at 448 (6), 64 of 512 (2 of 8).
    step = 0.125 if bits == 8 else 0.25
    for got, want in ((ck, turned[:, heads:]), (cv, qkv[:, heads + kv:])):
        top = want.abs().unflatten(-1, (2, 32)).amax(-1, keepdim=True).expand(-1, -1, -1, 32).flatten(-2)
        assert bool(((got - want).abs() <= step * top + 1e-4).all())
    ck, cv = ck.repeat_interleave(heads // kv, 1), cv.repeat_interleave(heads // kv, 1)
    p = torch.einsum("thd,shd->hts", turned[:, :heads], ck) / 8
    p = p.masked_fill(torch.ones(150, 150, device="cuda").triu(1).bool(), -float("inf")).softmax(-1)
    att = torch.einsum("hts,shd->thd", p, cv).flatten(1)
    codes = q.mx_quantize(att.float())
    want = q.mx_dequantize(codes).double() @ q.mx_dequantize(block.out).double().T
    assert float((y.double() - want).norm() / want.norm()) < 2e-3       # codes beside ties of a few of its inputs
    served, _ = m.serve(m.MxAttention(**weights, head_dim=64, pages=14, page=16, bits=bits), x, r, 140, 60, 16)
    assert float((served - y).norm() / y.norm()) < 2e-3
    q.device_status()
