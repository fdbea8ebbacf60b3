"""Tensors without values in the MX calls: no rows are nothing to do, rows of
no values are refused, whatever the number of dimensions."""
import pytest


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
    return m


@pytest.mark.parametrize("shape", [(4, 0), (0, 0), (0,), (2, 3, 0), (0, 3, 0), (2, 0, 0), (1, 2, 3, 0)])
def test_rows_of_no_values_are_refused(q, shape):
    import torch
    x, g = torch.zeros(shape), torch.zeros(0)
    for call in (lambda: q.mx_quantize(x), lambda: q.mx_swiglu(x, x), lambda: q.mx_rmsnorm(x, g),
                 lambda: q.mx_rmsnorm(x, g, residual=x)):
        with pytest.raises(q.Q4mmError) as e:
            call()
        assert e.value.code == -1 and "inputDim (0)" in str(e.value)


@pytest.mark.parametrize("shape", [(0, 96), (0, 3, 96), (2, 0, 96), (2, 0, 3, 96)])
def test_no_rows(q, shape):
    import torch
    x, g = torch.zeros(shape), torch.ones(96)
    for m in (q.mx_quantize(x), q.mx_swiglu(x, x), q.mx_rmsnorm(x, g), q.mx_rmsnorm(x, g, residual=x)[0]):
        assert m.rows == 0 and m.K == 96 and m.codes.shape == (0, 128)
