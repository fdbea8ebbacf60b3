"""Calls on another stream than the current one: memory that is dropped early,
or that the other stream still uses, is not reused too soon.  (What a result
holds is compared with the same call on the current stream: equal bits.)"""
import pytest

pytestmark = pytest.mark.gpu

BUSY = 20_000_000     # cycles, about 10 ms


def _torch():
    import torch
    return torch


def _q():
    import quantized_matmul_q4_gb300 as q
    return q


def _busy(stream):
    torch = _torch()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(BUSY)


def _overwrite(*like):
    """Allocations on the current stream that would get memory just dropped, and are written at once."""
    torch = _torch()
    return [torch.full_like(t, 77) for t in like for _ in range(4)]


def _same(a, b):
    if isinstance(a, tuple):
        return all(_same(x, y) for x, y in zip(a, b))
    return a == b if isinstance(a, int) else _torch().equal(a, b)


@pytest.mark.parametrize("as_handle", [False, True])
def test_temporaries_of_a_chain(as_handle):
    q, torch = _q(), _torch()
    s = torch.cuda.Stream()
    at = s.cuda_stream if as_handle else s
    a = torch.randn(300, 2048, device="cuda")
    w = q.mx_quantize(torch.randn(640, 2048, device="cuda"), bits=4)
    m = q.mx_quantize(a)
    want = q.mx_matmul(m, w)
    like = torch.empty_like(m.codes), torch.empty_like(m.scales), torch.empty_like(want)
    for _ in range(5):
        torch.cuda.synchronize()
        _busy(s)
        y = q.mx_matmul(q.mx_quantize(a, stream=at), w, stream=at)
        kept = _overwrite(*like)
        s.synchronize()
        assert torch.equal(y, want)
        del kept, y


def test_inputs_dropped_at_once():
    q, torch = _q(), _torch()
    s = torch.cuda.Stream()
    x, r = torch.randn(500, 1024, device="cuda"), torch.randn(500, 1024, device="cuda")
    g = torch.randn(1024, device="cuda")
    w4 = torch.randint(0, 100, (64 * 4 * 144,), dtype=torch.uint8, device="cuda")   # Q4_K, 64 rows of 1024
    w4.view(-1, 144)[:, 1] = w4.view(-1, 144)[:, 3] = 0x20
    calls = [lambda x, r, s: q.mx_quantize(x, bits=4, stream=s), lambda x, r, s: q.mx_swiglu(x, r, stream=s),
             lambda x, r, s: q.mx_rmsnorm(x, g, residual=r, stream=s), lambda x, r, s: q.q4k_matmul(x[:8], w4, stream=s)]
    for call in calls:
        want = call(x, r, None)
        x1, r1 = x.clone(), r.clone()
        torch.cuda.synchronize()
        _busy(s)
        got = call(x1, r1, s)
        del x1, r1
        kept = _overwrite(x, r)
        s.synchronize()
        assert _same(got, want)
        del kept


def test_memory_that_the_current_stream_still_reads():
    q, torch = _q(), _torch()
    s = torch.cuda.Stream()
    m = q.mx_quantize(torch.randn(700, 1024, device="cuda"))
    zeros = m._replace(codes=torch.zeros_like(m.codes))
    want = q.mx_dequantize(m)
    torch.cuda.synchronize()
    # A tensor of the current stream, dropped while that still reads it ...
    t = torch.randn(700, 1024, device="cuda")
    copy = t.clone()
    torch.cuda.synchronize()
    _busy(torch.cuda.current_stream())
    again = t.clone()
    del t
    y = q.mx_dequantize(m, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, copy) and torch.equal(y, want)
    # ... and a result of the other stream, dropped while the current one reads it.
    torch.cuda.current_stream().wait_stream(s)
    _busy(torch.cuda.current_stream())
    again = y.clone()
    del y
    y = q.mx_dequantize(zeros, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(again, want) and not y.any()
