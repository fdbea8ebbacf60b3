"""One Llama attention block on microscaled (MX) tensors: a prompt in chunks,
then single tokens, over a quantised paged cache.

    python examples/llama_attention_mx.py [--heads 32] [--kv-heads 32] [--prompt 1000] [--chunk 512] [--bits 8]

The block holds its weights in 4 bits, carries activations in 8 bits into the
products, and keeps keys and values in MX blocks of 4 or 8 bits:

    n, h = mx_rmsnorm(x, g, residual)                    residual added, norm, 8-bit codes
    qkv  = mx_matmul(n, W_qkv)                           queries, keys and values as one product
    q    = rope_rotate(qkv[:, :H], positions)            rotary positions of the queries
    mx_cache_write(cache, qkv[:, H:H+K], qkv[:, H+K:])   keys turned, both quantised into their pages
    a    = mx_attention(q, cache)                        softmax(q kᵀ) v over all that is cached
    y    = mx_matmul(mx_quantize(a), W_o)

A sequence's pages are dealt as it grows; a batch is described by three
tensors that stay in place, so a decoding step can be captured once in a CUDA
graph and replayed.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_matmul_q4_gb300 as q4mm  # noqa: E402


class MxAttention:
    """x, residual -> (y, h) of one attention block; keeps its own cache."""

    def __init__(self, norm, wq, wk, wv, wo, head_dim: int, pages: int, page: int = 64, bits: int = 8, eps: float = 1e-5):
        self.norm, self.eps, self.head_dim = norm, eps, head_dim
        self.heads, self.kv_heads = wq.shape[0] // head_dim, wk.shape[0] // head_dim
        self.qkv = q4mm.mx_quantize(torch.cat((wq, wk, wv)), bits=4)
        self.out = q4mm.mx_quantize(wo, bits=4)
        self.rope = q4mm.Rope(q4mm.rope_frequencies(head_dim))
        self.cache = q4mm.mx_cache(pages, self.kv_heads, head_dim, page=page, bits=bits)

    def __call__(self, x, residual, positions, starts, lengths, pages):
        n, h = q4mm.mx_rmsnorm(x, self.norm, eps=self.eps, residual=residual)
        qkv = q4mm.mx_matmul(n, self.qkv, dtype=x.dtype).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), dim=1)
        q = q4mm.rope_rotate(q, positions, self.rope)
        q4mm.mx_cache_write(self.cache, k, v, starts, lengths, pages, rope=self.rope)
        a = q4mm.mx_attention(q, self.cache, starts, lengths, pages)
        return q4mm.mx_matmul(q4mm.mx_quantize(a.view(x.shape[0], -1)), self.out, dtype=x.dtype), h


def reference(x, residual, norm, wq, wk, wv, wo, head_dim, eps=1e-5):
    """The block over one whole sequence in float32, elementary operations."""
    h = x.float() + residual.float()
    n = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * norm.float()
    q, k, v = ((n @ w.float().T).unflatten(-1, (-1, head_dim)).transpose(0, 1) for w in (wq, wk, wv))
    pos = torch.arange(x.shape[0], device=x.device, dtype=torch.float64)
    a = pos[:, None] * q4mm.rope_frequencies(head_dim, device=x.device)
    c, s = a.cos().float(), a.sin().float()

    def turned(t):
        lo, hi = t.chunk(2, -1)
        return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)
    q, k = turned(q), turned(k)
    group = q.shape[0] // k.shape[0]
    p = q @ k.repeat_interleave(group, 0).transpose(-1, -2) * head_dim ** -0.5
    p = p.masked_fill(torch.ones(p.shape[-2:], device=x.device).triu(1).bool(), float("-inf")).softmax(-1)
    return (p @ v.repeat_interleave(group, 0)).transpose(0, 1).flatten(1) @ wo.float().T


def make(heads: int, kv_heads: int, head_dim: int, tokens: int, seed: int = 0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dim = heads * head_dim
    def normal(*s, scale=1.0):
        return (scale * torch.randn(*s, generator=g, device="cuda")).to(dtype)
    weights = dict(norm=1 + normal(dim, scale=0.1), wq=normal(dim, dim, scale=1.5 * dim ** -0.5),
                   wk=normal(kv_heads * head_dim, dim, scale=dim ** -0.5),
                   wv=normal(kv_heads * head_dim, dim, scale=dim ** -0.5), wo=normal(dim, dim, scale=dim ** -0.5))
    return weights, normal(tokens, dim), normal(tokens, dim)


def serve(block: MxAttention, x, residual, prompt: int, chunk: int, page: int):
    """The prompt in chunks, then one token at a time by a captured step; returns all outputs and a step's microseconds."""
    total = x.shape[0]
    table = torch.randperm(block.cache.k_codes.shape[0], device="cuda").to(torch.int32)[None, :-(-total // page)].contiguous()
    ys = []
    for a in range(0, prompt, chunk):
        b = min(a + chunk, prompt)
        batch = torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), torch.tensor([b], dtype=torch.int32, device="cuda")
        ys.append(block(x[a:b], residual[a:b], torch.arange(a, b, dtype=torch.int32, device="cuda"), *batch, table)[0])
    if prompt == total:
        return torch.cat(ys), 0.0
    one_x, one_r = x[:1].clone(), residual[:1].clone()
    starts, lengths = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([prompt], dtype=torch.int32, device="cuda")
    pos = lengths - 1       # (the warm-up and the capture write the prompt's last place again, before it is read)
    keep = [t.clone() for t in block.cache[:4]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(one_x, one_r, pos, starts, lengths, table)
    torch.cuda.current_stream().wait_stream(side)
    for t, k in zip(block.cache[:4], keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = block(one_x, one_r, pos, starts, lengths, table)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    spent = 0.0
    for t in range(prompt, total):
        one_x.copy_(x[t:t + 1]), one_r.copy_(residual[t:t + 1])
        lengths.fill_(t + 1), pos.fill_(t)
        begin.record()
        graph.replay()
        end.record()
        ys.append(y.clone())
        end.synchronize()
        spent += begin.elapsed_time(end) * 1e3
    return torch.cat(ys), spent / (total - prompt)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=32)
    ap.add_argument("--head-dim", type=int, default=128)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--tokens", type=int, default=24, help="decoded after the prompt")
    ap.add_argument("--chunk", type=int, default=512)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--bits", type=int, default=8)
    a = ap.parse_args()
    weights, x, residual = make(a.heads, a.kv_heads, a.head_dim, a.prompt + a.tokens)
    block = MxAttention(**weights, head_dim=a.head_dim, pages=-(-(a.prompt + a.tokens) // a.page) + 5, page=a.page, bits=a.bits)
    y, us = serve(block, x, residual, a.prompt, a.chunk, a.page)
    ref = reference(x, residual, **weights, head_dim=a.head_dim)
    q4mm.device_status()
    off = float((y.float() - ref).norm() / ref.norm())
    print(f"{a.prompt} tokens in chunks of {a.chunk}, {a.tokens} one by one: a step takes {us:.1f} us on the device, "
          f"off from float32 by {off:.3f}")


if __name__ == "__main__":
    main()
