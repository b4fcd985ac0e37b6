"""kv8_attention where a part of a cache could get lost or count twice: the ends of CTAs' runs, of warps' turns, of pages
and of sequences.

Of each sequence and kv head one granule of 16 tokens (another one in each trial) has values, all others hold zeros, so the
output is made of that granule alone and the bound follows its size: a lost token moves the output by a sixteenth, fp16
weights and fp32 sums by 2^-11 at most.  The queries are small, so that all tokens weigh nearly the same: a lost granule of
L tokens moves the log sum by 16 / L, several times its bound."""
import math

import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import DT, TINY, UNIT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,kv_heads,n,page,window", [
    ([5999, 17, 4100, 3001, 800, 6000, 1, 2049], 8, 1, 64, 0),          # few rows, uneven items over many runs
    ([5999, 32, 4100, 3001, 800, 6000, 24, 2049], 8, 6, 16, 0),         # a verify window
    ([40001], 4, 1, 128, 0),                                            # one sequence over all CTAs
    ([5000, 3333], 8, 5, 32, 1111),
    ([2999, 64, 2100, 1501, 800, 3000, 40, 1025], 8, 40, 64, 0),        # many rows, enough tiles
    ([12001], 2, 300, 128, 0),                                          # many rows over all CTAs
    ([2500, 3333], 4, 290, 32, 1111),
])
def test_one_granule_of_values(lens, kv_heads, n, page, window, dim):
    G, dtype, B = 4, "f16", len(lens)
    gen = torch.Generator(device="cuda").manual_seed(dim + n)
    ns = [min(n, L) for L in lens]
    used = [-(-L // page) for L in lens]
    pages, width = sum(used) + 2, max(used) + 1
    ids = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, :used[b]] = ids[sum(used[:b]):sum(used[:b + 1])]
    shape = (pages, kv_heads, page, dim)
    k = torch.randint(1, 256, shape, device="cuda", generator=gen, dtype=torch.uint8)
    v = torch.full(shape, 128, dtype=torch.uint8, device="cuda")
    ks, vs = (0.01 * torch.exp(0.2 * torch.randn(shape[:2], device="cuda", generator=gen)) for _ in range(2))
    row0 = torch.tensor([sum(ns[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    M = sum(ns)
    q = (0.1 * torch.randn(M, kv_heads * G, dim, device="cuda", generator=gen)).to(DT[dtype])
    cache = lib8.KV8Cache(k, v, ks, vs)
    step = lib8.KV8Step(row0, torch.tensor(lens, dtype=torch.int32, device="cuda"), table, M, n)
    ws = lib8.alloc_workspace(lib8.kv8_workspace_bytes(kv_heads * G, kv_heads, dim))
    lse = torch.empty(M, kv_heads * G, device="cuda")
    scale = dim ** -0.5

    # Probabilities in 64 bits, once.
    probs, logs, weigh = [], [], []
    for b, L in enumerate(lens):
        pg = table[b, :used[b]].long()
        kk = (k[pg].double() - 128) * ks[pg].double()[:, :, None, None]
        kk = kk.transpose(0, 1).reshape(kv_heads, -1, dim)[:, :L]
        qq = q[row0[b]:row0[b + 1]].double().unflatten(1, (kv_heads, G)).permute(1, 2, 0, 3)
        s = torch.einsum("hgnd,hld->hgnl", qq, kk) * scale
        at, j = torch.arange(L - ns[b], L, device="cuda")[:, None], torch.arange(L, device="cuda")
        s = s.masked_fill((j > at) | ((j <= at - window) if window else torch.zeros_like(j > at)), -math.inf)
        d = scale * qq.abs().sum(-1) * 256 * (dim + 32) * 2.0 ** -24 * ks.max() + s.masked_fill(s.isinf(), 0).abs().amax(-1) * 2.0 ** -21 + 2.0 ** -20
        sums = (L / 16 + 64) * 2.0 ** -23
        probs.append(torch.softmax(s, -1))
        logs.append((torch.logsumexp(s, -1), 2 * d + sums + 2.0 ** -22 * 12))
        weigh.append(2 * d + 2.0 ** -11 + sums)

    for trial in range(10):
        v.fill_(128)
        where = []
        for b, L in enumerate(lens):
            grans = -(-L // 16)
            first = max(0, L - ns[b] - window + 1) // 16 if window else 0
            # Heads side by side, the last granule and the first among them.
            start = int(torch.randint(first, grans, (1,), device="cuda", generator=gen)) if trial else grans - 1
            where.append([first + (start - first + h) % (grans - first) for h in range(kv_heads)])
            for h, gr in enumerate(where[b]):
                slot = 16 * gr % page
                v[table[b, 16 * gr // page].long(), h, slot:slot + 16] = torch.randint(
                    150, 256, (16, dim), device="cuda", generator=gen, dtype=torch.uint8)
        out = lib8.kv8_attention(cache, step, q, ws, lse=lse, scale=scale, window=window)
        assert lib8.w8a8_workspace_status(ws) == 0
        for b, L in enumerate(lens):
            r = slice(int(row0[b]), int(row0[b + 1]))
            got = out[r].double().unflatten(1, (kv_heads, G)).permute(1, 2, 0, 3)
            z, (want_z, ez) = lse[r].double().unflatten(1, (kv_heads, G)).permute(1, 2, 0), logs[b]
            assert ((z - want_z).abs() <= ez).all(), (b, trial)
            for h, gr in enumerate(where[b]):
                t0, t1 = 16 * gr, min(16 * gr + 16, L)
                page_id = table[b, t0 // page].long()
                vv = (v[page_id, h, t0 % page:t0 % page + t1 - t0].double() - 128) * vs[page_id, h].double()
                ref = probs[b][h, :, :, t0:t1] @ vv
                e = weigh[b][h][..., None] * ref                 # (the values are above zero)
                assert ((got[h] - ref).abs() <= e + UNIT[dtype] * (ref + e) + TINY[dtype]).all(), (b, h, gr, trial)
