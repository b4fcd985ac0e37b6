#!/usr/bin/env python3
"""A speculative decoding loop on the library's calls, all of a step on the device: the next step's rows and pages
(kv8_plan), the int8 products of a small one-layer model (w8a8_gemm), norm, rotation and append to the 8-bit paged cache
(kv8_append), attention of requests that share a prompt (kv8_attention_shared), the probabilities of the vocabulary
(spec_probs) and the verification of the drafted tokens (spec_verify).

    python examples/speculative_loop.py [--batch 24] [--prompt 2048] [--window 5] [--steps 64]

Weights are random.  Drafts are looked up: a table of each token's likely successor, learnt from what the model has said.
A step is captured once in a CUDA graph; lengths, page tables and windows change in device memory.  (At these sizes
kv8_attention_shared leaves a step to kv8_attention's launch; from a table with room for some 400,000 tokens times kv heads on
it reads the prompt once for all requests.)"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import int8_weight_gemm_gb300 as lib8  # noqa: E402
from attention_layer import Linear8, rotations  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB = 1024, 8, 2, 128, 8192


def i32(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device="cuda")


class SpeculativeLoop:
    """`batch` requests behind one prompt, windows of up to `window` tokens (the last one said, then drafts), until each
    holds max_len tokens."""

    def __init__(self, batch, prompt, window, max_len, page_tokens=64, temperature=0.7, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.gen, self.batch, self.window, self.max_len, self.page = gen, batch, window, max_len, page_tokens
        rows = self.rows = batch * window
        self.qkv, self.proj, self.head = (Linear8(k, n, gen) for k, n in ((HIDDEN, (Q_HEADS + 2 * KV_HEADS) * DIM), (Q_HEADS * DIM, HIDDEN),
                                                                           (HIDDEN, VOCAB)))
        self.embed = torch.randn(VOCAB, HIDDEN, device="cuda", generator=gen).to(torch.bfloat16)
        self.prep = lib8.QKPrep(rotations(max_len, DIM).cuda(), DIM)
        # The prompt's whole pages are the first ones; every request's table begins with them.  The others are free.
        width, shared = -(-max_len // page_tokens), prompt // page_tokens
        pages = shared + batch * (width - shared)
        self.cache = lib8.kv8_cache(pages, KV_HEADS, page_tokens, DIM)
        self.table = i32(batch, width, fill=-1)
        self.table[:, :shared] = torch.arange(shared, device="cuda", dtype=torch.int32)
        ring = torch.arange(shared, pages, device="cuda", dtype=torch.int32)
        self.pool = lib8.KV8Pool(torch.cat([ring, i32(shared, fill=-1)]), torch.tensor([0, pages - shared], dtype=torch.int32, device="cuda"))
        self.prefix = shared * page_tokens
        self.row0, self.kv_len = i32(batch + 1), i32(batch, fill=self.prefix)
        self.held, self.pinned = i32(batch, fill=shared), i32(batch, fill=shared)
        self.step = lib8.KV8Step(self.row0, self.kv_len, self.table, rows, window)
        self.groups = lib8.KV8Groups(torch.tensor([0, batch], dtype=torch.int32, device="cuda"), i32(1, fill=self.prefix), rows)
        self.positions, self.seq_of, self.granted = i32(rows), i32(rows), i32(batch)
        self.take, self.grow = i32(batch), i32(batch, fill=window)
        self.windows = torch.randint(0, VOCAB, (batch, window), device="cuda", generator=gen)     # the next window's tokens
        self.drafts = torch.randint(0, VOCAB, (VOCAB,), device="cuda", generator=gen)             # each token's successor
        self.accept, self.sample = (torch.zeros(rows, device="cuda") for _ in range(2))
        self.inv_temp = torch.full((rows,), 1.0 / temperature, device="cuda")
        self.next = i32(rows, fill=-1)
        self.said = torch.zeros(batch, dtype=torch.int64, device="cuda")                          # tokens that came out
        self.ws = lib8.alloc_workspace(lib8.kv8_shared_workspace_bytes(rows, 1, Q_HEADS, KV_HEADS, DIM))
        self.spec_ws = lib8.alloc_workspace(lib8.spec_workspace_bytes(batch, VOCAB))
        self.graph = None
        self._prompt(torch.randint(0, VOCAB, (self.prefix,), device="cuda", generator=gen))

    def _heads(self, tokens):
        qkv = self.qkv(self.embed[tokens]).view(-1, Q_HEADS + 2 * KV_HEADS, DIM)
        return qkv.split([Q_HEADS, KV_HEADS, KV_HEADS], 1)

    def _prompt(self, tokens):
        """The shared tokens, once, in chunks that the products take."""
        done = 0
        for part in tokens.split(128):
            n = part.shape[0]
            done += n
            step = lib8.KV8Step(torch.tensor([0, n], dtype=torch.int32, device="cuda"), i32(1, fill=done), self.table[:1], n, n)
            _, k, v = self._heads(part)
            lib8.kv8_append(self.cache, step, self.prep, k, v, self.ws)

    def _step(self):
        lib8.kv8_plan(self.step, self.page, self.pool, self.held, self.take, self.grow, self.ws, pinned=self.pinned, granted=self.granted,
                      positions=self.positions, seq_of=self.seq_of)
        # The rows' tokens; rows behind the last sequence compute something that nobody reads.
        seq = self.seq_of.long().clamp(0, self.batch - 1)
        place = (torch.arange(self.rows, device="cuda") - self.row0[seq]).clamp(0, self.window - 1)
        self.tokens = self.windows[seq, place].to(torch.int32)
        q, k, v = self._heads(self.tokens.long())
        self.q = lib8.kv8_append(self.cache, self.step, self.prep, k, v, self.ws, q=q, positions=self.positions)
        self.context = lib8.kv8_attention_shared(self.cache, self.step, self.groups, self.q, self.ws)
        self.logits = self.head(self.proj(self.context.view(self.rows, -1)))
        self.p = lib8.spec_probs(self.logits, self.inv_temp)
        lib8.spec_verify(self.p, self.tokens, self.row0, self.accept, self.sample, self.spec_ws, next=self.next, take=self.take)
        # The next windows: the last token, then its successors by the table, which learns what followed it.
        self.said += self.take
        last_row = (self.row0[1:] - 1 - (self.granted - self.take)).clamp(0, self.rows - 1).long()
        live = self.granted > 0
        last = torch.where(live, self.next[last_row].long(), self.windows[:, 0]).clamp(min=0)
        self.drafts[self.tokens[last_row].long()] = last
        window = [last]
        for _ in range(self.window - 1):
            window.append(self.drafts[window[-1]])
        self.windows.copy_(torch.stack(window, 1))
        # A request that has no room for another window ends: its own pages go back at the next plan.
        kept = self.kv_len - self.granted + self.take
        self.take.copy_(torch.where(live & (kept + self.window > self.max_len), -1, self.take))
        self.grow.mul_((self.take >= 0).to(torch.int32))

    def run(self, accept=None):
        """One step, through a graph captured at the first call.  accept: the random numbers of the tests, drawn if not given."""
        if self.graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph, stream=side):
                self._step()
        self.accept.uniform_(generator=self.gen) if accept is None else self.accept.copy_(accept)
        self.sample.uniform_(generator=self.gen)
        self.graph.replay()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=24)
    ap.add_argument("--prompt", type=int, default=2048)
    ap.add_argument("--window", type=int, default=5)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    loop = SpeculativeLoop(a.batch, a.prompt, a.window, a.prompt + a.steps * a.window + 64)
    loop.run()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(a.steps):
        loop.run()
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / a.steps
    assert lib8.w8a8_workspace_status(loop.ws) == 0 and lib8.w8a8_workspace_status(loop.spec_ws) == 0
    print(f"{a.batch} requests behind {loop.prefix} tokens, windows of {a.window}: {t * 1e6:.1f} us a step, "
          f"{loop.said.float().mean().item() / (a.steps + 1):.2f} tokens a request and step")


if __name__ == "__main__":
    main()
