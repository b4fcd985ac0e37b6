#!/usr/bin/env python3
"""The attention half of a decoder layer on the library's calls, as a serving loop makes them: int8 activations, the
fused QKV product (w8a8_gemm), norm, rotation and append to the 8-bit paged cache (kv8_append), attention over it
(kv8_attention), int8 again and the output projection (w8a8_gemm).

    python examples/attention_layer.py [--batch 16] [--context 2048] [--steps 64]

The sizes are those of one of four tensor-parallel ranks: hidden 4096, 8 query heads and 2 key-value heads of 128 (QKV
columns 1536).  Weights are random.  A decode step is captured once in a CUDA graph; lengths advance on the device."""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_weight_gemm_gb300 as lib8  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM = 4096, 8, 2, 128
QKV = (Q_HEADS + 2 * KV_HEADS) * DIM
MAX_ROWS = 128          # of a w8a8_gemm call


def rotations(positions: int, dim: int = DIM, base: float = 10000.0) -> torch.Tensor:
    """fp32 [positions, dim]: a position's cosines, then its sines."""
    inv = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class Linear8:
    """An int8 weight [K, N] with its column scales, packed for w8a8_gemm."""

    def __init__(self, K, N, gen):
        w = torch.randn(K, N, device="cuda", generator=gen) / K ** 0.5
        self.scale = w.abs().amax(0) / 127.0
        self.ws = lib8.alloc_workspace(lib8.w8a8_workspace_bytes(MAX_ROWS, K, N))
        self.packed = lib8.w8a8_pack_weights((w / self.scale).round().to(torch.int8), ws=self.ws)
        self.N = N

    def __call__(self, x):
        xq, xs = lib8.w8a8_quantize_activations(x)
        return lib8.w8a8_gemm(xq, xs, self.packed, self.scale, self.ws, self.N)


class AttentionLayer:
    """One layer's projections and cache.  Sequence b's pages are rows of `table`; kv_len is its cached tokens."""

    def __init__(self, batch, max_len, page_tokens=64, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.batch, self.max_len = batch, max_len
        self.qkv, self.proj = Linear8(HIDDEN, QKV, gen), Linear8(Q_HEADS * DIM, HIDDEN, gen)
        width = -(-max_len // page_tokens)
        pages = batch * width
        self.cache = lib8.kv8_cache(pages, KV_HEADS, page_tokens, DIM)
        self.table = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).view(batch, width)
        self.kv_len = torch.zeros(batch, device="cuda", dtype=torch.int32)
        gamma = [(1 + 0.1 * torch.randn(DIM, device="cuda", generator=gen)).to(torch.bfloat16) for _ in range(2)]
        self.prep = lib8.QKPrep(rotations(max_len).cuda(), DIM, *gamma, eps=1e-6)
        self.ws = lib8.alloc_workspace(lib8.kv8_workspace_bytes(Q_HEADS, KV_HEADS, DIM))
        # One row a sequence: a decode step.
        self.one = lib8.KV8Step(torch.arange(batch + 1, device="cuda", dtype=torch.int32), self.kv_len, self.table, batch, 1)
        self.graph = None

    def forward(self, x, step):
        """x [rows, HIDDEN] bf16, the step's rows; kv_len already counts them.  Appends and attends."""
        rows = x.shape[0]
        qkv = self.qkv(x).view(rows, Q_HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)
        q = lib8.kv8_append(self.cache, step, self.prep, k, v, self.ws, q=q)
        self.q, self.context = q, lib8.kv8_attention(self.cache, step, q, self.ws)
        return self.proj(self.context.view(rows, Q_HEADS * DIM))

    def prompt(self, b, x):
        """x [tokens, HIDDEN]: sequence b's next tokens, in chunks that the projections take."""
        out = []
        for part in x.split(MAX_ROWS):
            row0 = torch.zeros(self.batch + 1, dtype=torch.int32)
            row0[b + 1:] = part.shape[0]
            self.kv_len[b] += part.shape[0]
            out.append(self.forward(part, lib8.KV8Step(row0.cuda(), self.kv_len, self.table, part.shape[0], part.shape[0])))
        return torch.cat(out)

    def decode(self, x):
        """x [batch, HIDDEN]: one token of every sequence, through a graph captured at the first call."""
        if self.graph is None:
            self.x = x.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self.kv_len.add_(1)
                self.out = self.forward(self.x, self.one)
        self.x.copy_(x)
        self.graph.replay()
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--context", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    layer = AttentionLayer(a.batch, a.context + a.steps + 1)
    for b in range(a.batch):
        layer.prompt(b, torch.randn(a.context, HIDDEN, device="cuda").to(torch.bfloat16))
    x = torch.randn(a.batch, HIDDEN, device="cuda").to(torch.bfloat16)
    layer.decode(x)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        layer.decode(x)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    assert lib8.w8a8_workspace_status(layer.ws) == 0
    print(f"{a.batch} sequences at {a.context} tokens: {t * 1e6:.1f} us a layer step (QKV, append, attention, projection)")


if __name__ == "__main__":
    main()
