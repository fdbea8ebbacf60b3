"""One Llama feed-forward block on microscaled (MX) tensors.

    python examples/llama_ffn_mx.py [--tokens 1 16 1000] [--dim 4096] [--hidden 11008]

The block holds its weights in 4 bits and carries activations in 8 bits
between the kernels:

    n, h = mx_rmsnorm(x, g, residual)        residual added, norm, 8-bit codes
    gu   = mx_matmul(n, W_gate_up)           gate and up as one product
    a    = mx_swiglu(gu[:, :H], gu[:, H:])   silu(gate)·up, 8-bit codes
    y    = mx_matmul(a, W_down)

four launches.  The result is compared with the same block in float32 on the
weights and activations as given, so the difference printed is that of the
formats: about 4 bits of weight and 8 of activation.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matmul_q4_gb300 as q4mm  # noqa: E402


class MxFeedForward:
    """x, residual -> (y, h): the block's output and the residual stream after the addition."""

    def __init__(self, norm, gate, up, down, eps: float = 1e-5):
        self.norm, self.eps, self.hidden = norm, eps, gate.shape[0]
        self.gate_up = q4mm.mx_quantize(torch.cat((gate, up)), bits=4)
        self.down = q4mm.mx_quantize(down, bits=4)

    def __call__(self, x, residual):
        n, h = q4mm.mx_rmsnorm(x, self.norm, eps=self.eps, residual=residual)
        gu = q4mm.mx_matmul(n, self.gate_up, dtype=x.dtype)
        a = q4mm.mx_swiglu(gu[:, :self.hidden], gu[:, self.hidden:])
        return q4mm.mx_matmul(a, self.down, dtype=x.dtype), h


def reference(x, residual, norm, gate, up, down, eps=1e-5):
    """The block in float32, elementary operations."""
    h = x.float() + residual.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * norm.float()
    g = n @ gate.float().T
    return (g * torch.sigmoid(g) * (n @ up.float().T)) @ down.float().T


def make(dim: int, hidden: int, tokens: int, seed: int = 0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    def normal(*s, scale=1.0):
        return (scale * torch.randn(*s, generator=g, device="cuda")).to(dtype)
    weights = dict(norm=1 + normal(dim, scale=0.1), gate=normal(hidden, dim, scale=dim ** -0.5),
                   up=normal(hidden, dim, scale=dim ** -0.5), down=normal(dim, hidden, scale=hidden ** -0.5))
    return weights, normal(tokens, dim), normal(tokens, dim)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, nargs="+", default=[1, 16, 1000])
    ap.add_argument("--dim", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=11008)
    a = ap.parse_args()
    for tokens in a.tokens:
        weights, x, residual = make(a.dim, a.hidden, tokens)
        block = MxFeedForward(**weights)
        y, _ = block(x, residual)
        ref = reference(x, residual, **weights)
        off = float((y.float() - ref).norm() / ref.norm())
        # The block in a CUDA graph, as a serving loop would replay it.
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block(x, residual)
        for _ in range(3):
            graph.replay()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(20):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        q4mm.device_status()
        us = start.elapsed_time(end) / 20 * 1e3
        print(f"{tokens:5d} tokens: {us:8.1f} us a block, {6 * tokens * a.dim * a.hidden / us / 1e6:8.1f} TFLOP/s, "
              f"off from float32 by {off:.3f}")


if __name__ == "__main__":
    main()
