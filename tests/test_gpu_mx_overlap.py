"""Products on several streams at once: CTAs of both MX forms and of the Q4_K
tensor-core kernel compete for the same SMs and their tensor memory.  Every
result has the bits of a call on its own."""
import pytest

from test_gpu_mx import _random_mx, _rng

pytestmark = pytest.mark.gpu


def test_products_on_several_streams():
    import torch
    import synth
    import quantized_matmul_q4_gb300 as q

    def mx(T, K, N, bits):
        g = _rng(61, T, K, N)
        x, w = _random_mx(g, T, K, bits)[0], _random_mx(g, N, K, 4)[0]
        return lambda out, s: q.mx_matmul(x, w, out=out, stream=s), torch.empty(T, N, device="cuda")

    def q4k(T, K, N):
        x, w = (torch.from_numpy(a).cuda() for a in synth.q4k_case((K, N, T), seed=62)[:2])
        w = w.reshape(-1)
        return lambda out, s: q.q4k_matmul_tc(x, w, N=N, out=out, stream=s), torch.empty(T, N, device="cuda")

    # Per stream: clusters of single CTAs in turn with few columns and many, pairs, Q4_K.
    lanes = [[mx(1, 4096, 4096, 8), mx(64, 8192, 1200, 4), mx(16, 2560, 7000, 8)],
             [mx(100, 4096, 600, 8), mx(17, 4096, 11008, 4)],
             [mx(700, 640, 3400, 8), mx(192, 4224, 9000, 4)],
             [q4k(64, 2048, 4096), q4k(100, 1024, 3000)]]
    want = []
    for lane in lanes:
        for f, out in lane:
            f(out, None)
            torch.cuda.synchronize()
            want.append(out.clone())
            out.fill_(float("nan"))
    streams = [torch.cuda.Stream() for _ in lanes]
    torch.cuda.synchronize()
    for _ in range(60):
        for lane, s in zip(lanes, streams):
            for f, out in lane:
                f(out, s)
    torch.cuda.synchronize()
    q.device_status()
    got = [out for lane in lanes for _, out in lane]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
