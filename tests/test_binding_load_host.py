"""The first call looks up what the binding takes from torch; another thread's
call may come at any point of that."""


def test_a_call_in_the_middle_of_the_first_one(monkeypatch):
    import torch
    from quantized_matmul_q4_gb300 import _binding as b

    class Library:
        def __getattr__(self, name):
            return lambda *args: 0

    monkeypatch.setattr(b, "_LIB", Library())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    x, g = torch.zeros(3, 256), torch.zeros(256)
    m = b.MxTensor(torch.zeros(3, 256, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8), 256, 8)
    w = b.MxTensor(torch.zeros(5, 128, dtype=torch.uint8), torch.zeros(1, 2, 512, dtype=torch.uint8), 256, 4)
    q4k = torch.zeros(2 * 144, dtype=torch.uint8)
    calls = [lambda: b.mx_quantize(x), lambda: b.mx_swiglu(x, x), lambda: b.mx_rmsnorm(x, g, residual=x),
             lambda: b.mx_dequantize(m), lambda: b.mx_matmul(m, w), lambda: b.q4k_matmul(x, q4k)]
    points = []
    empty = {name: ({} if name == "dtypes" else None)
             for name, value in vars(b._Torch).items() if not name.startswith("_") and name != "load"}

    for call in calls:
        class AfterEachAssignment(type):
            inside = False

            def __setattr__(cls, name, value):
                super().__setattr__(name, value)
                if not AfterEachAssignment.inside and not name.startswith("_"):
                    AfterEachAssignment.inside = True
                    # The other thread's whole call, from this point of the loading ...
                    state = {n: getattr(cls, n) for n in empty}
                    call()
                    points.append(name)
                    # ... which leaves this thread's own loading where it was.
                    for n, v in state.items():
                        type.__setattr__(cls, n, v)
                    AfterEachAssignment.inside = False

        watched = AfterEachAssignment("_Torch", (b._Torch,), {n: v for n, v in empty.items()})
        monkeypatch.setattr(b, "_Torch", watched)
        call()
        monkeypatch.setattr(b, "_Torch", b._Torch.__mro__[1])
    assert len(points) >= len(calls) * len(empty)
