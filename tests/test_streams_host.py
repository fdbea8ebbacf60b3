"""Which stream a tensor call uses, whose memory its results have, and what is
kept from reuse: on the host, with stand-ins for the library and for torch's
CUDA streams."""
import contextlib
import types

import pytest

CURRENT, OTHER = 0x10, 0x20


class _Stream:
    """As much of a torch stream as the binding looks at."""

    def __init__(self, handle):
        self.cuda_stream = handle
        self.device = types.SimpleNamespace(index=0)

    def record_event(self):
        raise AssertionError("nothing is recorded on a stream itself")


@pytest.fixture
def host(monkeypatch):
    """CPU tensors that pass for CUDA ones; the calls, and what is allocated and recorded where."""
    import torch
    import quantized_matmul_q4_gb300 as q
    from quantized_matmul_q4_gb300 import _binding as b

    h = types.SimpleNamespace(q=q, torch=torch, calls=[], device=0, under=CURRENT, pools={}, records=[], keep=[])

    class Library:
        def __getattr__(self, name):
            def call(*args):
                h.calls.append((name, args))
                return 0
            return call

    @contextlib.contextmanager
    def under(stream):
        before, h.under = h.under, stream.cuda_stream
        yield
        h.under = before

    def empty(*a, device=None, **kw):
        t = plain(*a, **kw)
        h.keep.append(t)          # (addresses stay unique)
        h.pools[t.data_ptr()] = h.under
        return t

    plain = torch.empty
    b._Torch.load()
    monkeypatch.setattr(b, "_LIB", Library())
    monkeypatch.setattr(b._Torch, "raw_stream", lambda device: CURRENT)
    monkeypatch.setattr(b._Torch, "current_device", lambda: h.device)
    monkeypatch.setattr(b._Torch, "empty", empty)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: h.records.append((t.data_ptr(), s.cuda_stream)))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _Stream(CURRENT))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: _Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: _Stream(handle))
    return h


def _calls(h):
    """Every tensor call: (name, call of a stream, the tensors it reads)."""
    q, torch = h.q, h.torch
    x, w8 = torch.zeros(3, 256), torch.zeros(3, 256)
    q4k, q40 = torch.zeros(2 * 144, dtype=torch.uint8), torch.zeros(2 * 8 * 18, dtype=torch.uint8)
    q6k, tern = torch.zeros(2 * 210, dtype=torch.uint8), torch.zeros(2 * 64, dtype=torch.uint8)
    relaid = torch.zeros(q.tc_relayout_bytes(256, 2), dtype=torch.uint8)
    up = torch.zeros_like(q4k)
    g = torch.zeros(256)
    m = q.MxTensor(torch.zeros(3, 256, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8), 256, 8)
    w = q.MxTensor(torch.zeros(5, 128, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8), 256, 4)
    return [
        ("q4k_matmul", lambda s: q.q4k_matmul(x, q4k, stream=s), [x, q4k]),
        ("q4k_matmul_tc", lambda s: q.q4k_matmul_tc(x, q4k, stream=s), [x, q4k]),
        ("q4k_matmul_tc_noalloc", lambda s: q.q4k_matmul_tc_noalloc(x, q4k, stream=s), [x, q4k]),
        ("q4k_relayout_tc", lambda s: q.q4k_relayout_tc(q4k, 256, stream=s), [q4k]),
        ("q4k_matmul_tc_relayouted", lambda s: q.q4k_matmul_tc_relayouted(x, relaid, 2, stream=s), [x, relaid]),
        ("q4_0_gemv", lambda s: q.q4_0_gemv(x, q40, stream=s), [x, q40]),
        ("q6k_gemv", lambda s: q.q6k_gemv(x, q6k, stream=s), [x, q6k]),
        ("q4k_ffn_swiglu", lambda s: q.q4k_ffn_swiglu(x, q4k, up, stream=s), [x, q4k, up]),
        ("ternary_gemv", lambda s: q.ternary_gemv(x, tern, stream=s), [x, tern]),
        ("mx_quantize", lambda s: q.mx_quantize(x, stream=s), [x]),
        ("mx_swiglu", lambda s: q.mx_swiglu(x, w8, stream=s), [x, w8]),
        ("mx_rmsnorm", lambda s: q.mx_rmsnorm(x, g, stream=s), [x, g]),
        ("mx_rmsnorm", lambda s: q.mx_rmsnorm(x, g, residual=w8, stream=s), [x, g, w8]),
        ("mx_dequantize", lambda s: q.mx_dequantize(m, stream=s), [m.codes, m.scales]),
        ("mx_matmul", lambda s: q.mx_matmul(m, w, stream=s), [m.codes, m.scales, w.codes, w.scales]),
    ]


def _tensors(result):
    if isinstance(result, tuple):
        return [t for part in result for t in _tensors(part)]
    return [] if isinstance(result, int) else [result]


COUNT = 15


@pytest.mark.parametrize("i", range(COUNT))
@pytest.mark.parametrize("given", [None, CURRENT, _Stream(CURRENT)], ids=["none", "handle", "stream"])
def test_on_the_current_stream_nothing_is_recorded(host, i, given):
    assert len(_calls(host)) == COUNT
    name, call, _ = _calls(host)[i]
    out = _tensors(call(given))
    assert [(c[0], c[1][-1]) for c in host.calls] == [(name, CURRENT)]
    assert out and all(host.pools[t.data_ptr()] == CURRENT for t in out)
    assert not host.records


@pytest.mark.parametrize("i", range(COUNT))
@pytest.mark.parametrize("given", [OTHER, _Stream(OTHER), 0], ids=["handle", "stream", "default"])
def test_on_another_stream_memory_waits_for_both(host, i, given):
    name, call, reads = _calls(host)[i]
    out = _tensors(call(given))
    at = 0 if given == 0 else OTHER
    assert [(c[0], c[1][-1]) for c in host.calls] == [(name, at)]
    # Results lie in that stream's pool and wait for the current one, which has them from now on;
    # what the call reads waits for its stream.
    assert out and all(host.pools[t.data_ptr()] == at for t in out)
    assert {(t.data_ptr(), CURRENT) for t in out} <= set(host.records)
    assert {(t.data_ptr(), at) for t in reads} <= set(host.records)


def test_results_written_into_given_tensors_wait_too(host):
    q, torch = host.q, host.torch
    x, g, h = torch.zeros(3, 128), torch.zeros(128), torch.zeros(3, 128)
    out = q.MxTensor(torch.zeros(3, 128, dtype=torch.uint8), torch.zeros(1, 1, 512, dtype=torch.uint8), 128, 8)
    q.mx_rmsnorm(x, g, residual=x, out=out, h_out=h, stream=OTHER)
    assert {(t.data_ptr(), OTHER) for t in (out.codes, out.scales, h)} <= set(host.records)
    y = torch.zeros(3, 2)
    q.q4k_matmul(torch.zeros(3, 256), torch.zeros(288, dtype=torch.uint8), out=y, stream=OTHER)
    assert (y.data_ptr(), OTHER) in host.records


@pytest.mark.parametrize("i", range(COUNT))
def test_tensors_of_another_device_are_refused(host, i):
    # The library would launch on the current device with the other one's pointers.
    host.device = 1
    for stream in (None, OTHER, _Stream(OTHER)):
        with pytest.raises(ValueError, match="device"):
            _calls(host)[i][1](stream)
    assert not host.calls


@pytest.mark.parametrize("i", range(COUNT))
def test_a_stream_of_another_device_is_refused(host, i):
    stream = _Stream(OTHER)
    stream.device.index = 1
    with pytest.raises(ValueError, match="device"):
        _calls(host)[i][1](stream)
    assert not host.calls


def test_tensors_of_two_devices_are_refused(host, monkeypatch):
    q, torch = host.q, host.torch
    there = []
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: int(any(t is o for o in there)))
    x, g = torch.zeros(3, 256), torch.zeros(256)
    wq, up = torch.zeros(2 * 144, dtype=torch.uint8), torch.zeros(2 * 144, dtype=torch.uint8)
    y, r = torch.zeros(3, 2), torch.zeros(3, 256)
    codes, scales = torch.zeros(3, 256, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8)
    relaid = torch.zeros(q.tc_relayout_bytes(256, 2), dtype=torch.uint8)
    out = q.MxTensor(codes, scales, 256, 8)
    for other, call in [(wq, lambda: q.q4k_matmul(x, wq)), (y, lambda: q.q4k_matmul(x, wq, out=y)),
                        (up, lambda: q.q4k_ffn_swiglu(x, wq, up)),
                        (relaid, lambda: q.q4k_relayout_tc(wq, 256, out=relaid)),
                        (r, lambda: q.mx_swiglu(x, r)), (g, lambda: q.mx_rmsnorm(x, g)),
                        (r, lambda: q.mx_rmsnorm(x, g, residual=r)), (scales, lambda: q.mx_quantize(x, out=out)),
                        (codes, lambda: q.mx_dequantize(out))]:
        there[:] = [other]
        with pytest.raises(ValueError, match="device"):
            call()
    assert not host.calls
