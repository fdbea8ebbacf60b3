"""Streams, memory and devices of the attention calls, on the host: what
test_streams_host asks of every other tensor call."""
import struct

import pytest

from test_streams_host import CURRENT, OTHER, _Stream, _tensors, host  # noqa: F401


def _calls(h):
    """(name, call of a stream, the tensors it reads or writes beside its results)"""
    q, torch = h.q, h.torch
    c = q.mx_cache(4, 2, 64, page=16, device="cpu")
    starts, lengths = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    pages, f = torch.zeros(1, 2, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    x, k, v, pos = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    batch = (starts, lengths, pages)
    return [
        ("rope_rotate", lambda s: q.rope_rotate(x, pos, q.Rope(f), stream=s), [x, pos, f]),
        ("mx_cache_write", lambda s: q.mx_cache_write(c, k, v, *batch, rope=q.Rope(f), stream=s) and (),
         [*c[:4], k, v, f, *batch]),
        ("mx_cache_read", lambda s: q.mx_cache_read(c, *batch, tokens=3, stream=s), [*c[:4], *batch]),
        ("mx_attention", lambda s: q.mx_attention(x, c, *batch, stream=s), [x, *c[:4], *batch]),
    ]


NAMES = ("rope_rotate", "mx_cache_write", "mx_cache_read", "mx_attention")


def _words(args):
    """The 8-byte words of a packed call; the last is its stream."""
    return struct.unpack(f"={len(args[1]) // 8}q", args[1])


def _launches(h):
    return [(NAMES[a[0]], _words(a)[-1]) for n, a in h.calls if n != "mx_attention_workspace" and n == "q4mm_call"]


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("given", [None, CURRENT, _Stream(CURRENT)], ids=["none", "handle", "stream"])
def test_on_the_current_stream_nothing_is_recorded(host, i, given):  # noqa: F811
    name, call, _ = _calls(host)[i]
    out = _tensors(call(given))
    assert _launches(host) == [(name, CURRENT)] and not host.records
    assert all(host.pools[t.data_ptr()] == CURRENT for t in out)


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("given", [OTHER, _Stream(OTHER), 0], ids=["handle", "stream", "default"])
def test_on_another_stream_memory_waits_for_both(host, i, given):  # noqa: F811
    name, call, uses = _calls(host)[i]
    out = _tensors(call(given))
    at = 0 if given == 0 else OTHER
    assert _launches(host) == [(name, at)]
    assert all(host.pools[t.data_ptr()] == at for t in out)
    assert {(t.data_ptr(), CURRENT) for t in out} <= set(host.records)
    assert {(t.data_ptr(), at) for t in uses} <= set(host.records)


@pytest.mark.parametrize("i", range(4))
def test_another_device_is_refused(host, i):  # noqa: F811
    host.device = 1
    for stream in (None, OTHER, _Stream(OTHER)):
        with pytest.raises(ValueError, match="device"):
            _calls(host)[i][1](stream)
    host.device = 0
    stream = _Stream(OTHER)
    stream.device.index = 1
    with pytest.raises(ValueError, match="device"):
        _calls(host)[i][1](stream)
    assert not _launches(host)


def test_tensors_of_two_devices_are_refused(host, monkeypatch):  # noqa: F811
    for i in range(4):
        _, call, uses = _calls(host)[i]
        for other in uses:
            monkeypatch.setattr(host.torch.Tensor, "get_device", lambda t, other=other: int(t is other))
            if other is uses[0]:
                continue
            with pytest.raises(ValueError, match="device"):
                call(None)
    assert not _launches(host)


def test_a_workspace_waits_like_a_result(host):  # noqa: F811
    """A call that is given a workspace takes it from its stream's pool and keeps it from reuse."""
    name, call, _ = _calls(host)[3]
    from quantized_matmul_q4_gb300 import _binding as b
    lib = b._LIB

    class Asked:
        def __getattr__(self, n):
            return (lambda *a: 4096) if n == "mx_attention_workspace" else getattr(lib, n)
    b._LIB = Asked()
    try:
        call(OTHER)
    finally:
        b._LIB = lib
    (args,) = [_words(a) for n, a in host.calls if n == "q4mm_call"]
    assert args[-2] == 4096 and host.pools[args[-3]] == OTHER
    assert {(args[-3], OTHER), (args[-3], CURRENT)} <= set(host.records)
