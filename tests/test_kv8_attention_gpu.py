"""kv8_attention on the GPU against the plain 64-bit form, over the shapes and masks where it can go wrong.  The
bounds are derived in kv8_util.Case.attention."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import UNIT, Case

pytestmark = pytest.mark.gpu


def _run(c, scale=None, window=0, flags=0, pad_out=0):
    scale = c.D ** -0.5 if scale is None else scale
    c.tensors()
    out = torch.full((c.M, c.Hq * c.D + pad_out), float("nan"), dtype=c.q.dtype, device="cuda")
    view = out[:, :c.Hq * c.D].unflatten(1, (c.Hq, c.D))
    lse = torch.full((c.M, c.Hq), float("nan"), device="cuda")
    lib8.kv8_attention(c.cache, c.step, c.q, c.ws, out=view, lse=lse, scale=scale, window=window, flags=flags)
    torch.cuda.synchronize()
    assert c.status() == 0
    if pad_out:
        assert torch.isnan(out[:, c.Hq * c.D:].float()).all()     # nothing past the heads is written
    return view, lse, scale


EDGES = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 200, 257]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_single_tokens_at_edge_lengths(dtype, dim, page):
    c = Case([1] * len(EDGES), EDGES, 8, 2, dim, page, dtype, seed=dim + page)
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 1), (7, 1), (5, 5), (12, 4), (16, 1), (17, 1), (40, 2), (64, 2),
                                              (96, 1), (130, 1)])
def test_head_layouts(q_heads, kv_heads):
    c = Case([1, 1, 1], [70, 1, 300], q_heads, kv_heads, 128, 64, seed=q_heads)
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ns,lens", [
    ([6, 6, 6], [6, 100, 64]),
    ([1, 8, 0, 5, 3], [40, 8, 25, 130, 67]),       # a sequence without rows
    ([2, 3, 1], [0, 1, 0]),                        # lengths of zero, more rows than tokens: rows that see nothing
    ([4, 9], [2, 5]),
    ([33, 17], [33, 200]),
    ([70], [70]),
    ([129, 1, 2], [300, 500, 2]),
])
def test_windows_and_prompts(ns, lens, dim):
    c = Case(ns, lens, 8, 2, dim, 32, "bf16", seed=sum(ns) + dim, pad=8)
    out, lse, scale = _run(c, pad_out=16)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("ns,lens,heads,window,causal", [
    ([29, 1, 0, 28], [29, 64, 9, 200], (8, 2), 0, True),
    ([130, 33], [130, 65], (1, 1), 0, True),                 # more than a tile of 128
    ([129, 2], [300, 77], (8, 1), 0, True),                  # 1032 rows of a kv head
    ([97, 300], [97, 1003], (16, 2), 130, True),
    ([100], [1503], (8, 1), 0, False),
    ([60, 2], [1000, 1], (4, 2), 100, True),
    ([60, 200], [63, 200], (3, 1), 17, True),
    ([40, 64], [0, 161], (4, 1), 0, False),
    ([150], [4001], (2, 1), 0, True),                        # one sequence over many CTAs
])
@pytest.mark.parametrize("page", [16, 128])
def test_prompts_of_wide_heads(ns, lens, heads, window, causal, page):
    c = Case(ns, lens, *heads, 256, page, "bf16" if page == 16 else "f16", seed=sum(ns) + page, pad=8)
    out, lse, scale = _run(c, window=window, flags=0 if causal else lib8.KV8_FLAG_NOT_CAUSAL, pad_out=16)
    c.check_attention(out, lse, scale, window, causal)


@pytest.mark.parametrize("dim,longest", [(64, 9), (64, 32), (128, 9), (128, 32), (128, 60), (256, 32), (256, 60)])
@pytest.mark.parametrize("window,causal,dtype", [(0, True, "bf16"), (37, True, "f16"), (0, False, "bf16")])
def test_many_sequences_of_many_rows(dim, longest, window, causal, dtype):
    # Tiles enough for the kernel of many rows with 36 to 240 rows of a kv head; sequences without rows or tokens,
    # single rows, fewer tokens than rows, and a few long ones whose tiles are cut.
    rng = np.random.default_rng(dim + longest)
    ns = [0, 1, longest, longest] + rng.integers(1, longest + 1, 31).tolist()
    lens = [9, 1, 0, longest // 2] + [int(n + rng.integers(0, 300)) for n in ns[4:]]
    lens[7], lens[20] = 3001, 1100
    c = Case(ns, lens, 8, 2, dim, 16, dtype, seed=longest, pad=8)
    out, lse, scale = _run(c, window=window, flags=0 if causal else lib8.KV8_FLAG_NOT_CAUSAL, pad_out=16)
    c.check_attention(out, lse, scale, window, causal)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 10**6])
@pytest.mark.parametrize("ns,lens", [([1, 1, 1, 1], [1, 16, 130, 400]), ([5, 3, 40], [5, 90, 333]), ([150], [420])])
def test_sliding_windows(ns, lens, window):
    c = Case(ns, lens, 8, 2, 64, 16, "f16", seed=window % 97)
    out, lse, scale = _run(c, window=window)
    c.check_attention(out, lse, scale, window)


@pytest.mark.parametrize("ns,lens", [([1, 4, 2], [0, 77, 160]), ([50, 20], [33, 129]), ([3, 130], [1, 260])])
def test_not_causal(ns, lens):
    c = Case(ns, lens, 4, 2, 128, 64, "bf16", seed=5)
    out, lse, scale = _run(c, flags=lib8.KV8_FLAG_NOT_CAUSAL)
    c.check_attention(out, lse, scale, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ns,lens,heads", [([1], [40001], (4, 1)), ([1, 1, 1], [9000, 17, 5003], (8, 2)), ([5], [7001], (8, 1)),
                                           ([70], [6007], (4, 1))])
def test_long_caches_split_over_many_ctas(ns, lens, heads, dtype):
    c = Case(ns, lens, *heads, 128, 64, dtype, seed=9, amp=2.0)
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


def test_many_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 90, 700).tolist()
    ns = [int(min(1 + (b % 3 == 0), max(l, 1))) if b % 11 else 0 for b, l in enumerate(lens)]
    c = Case(ns, lens, 4, 1, 64, 16, "f16", seed=4)
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("ns,lens", [([1, 1], [150, 333]), ([20], [222]), ([80], [300])])
def test_page_scales_of_every_size(ns, lens):
    # Pages of zero scale, and value scales over sixty orders of magnitude: the largest logits stand beside the
    # smallest values and the other way round.
    c = Case(ns, lens, 8, 2, 128, 16, "bf16", seed=8)
    used = c.table[c.table >= 0]
    c.vs[used[::3]] *= 1e-20
    c.vs[used[1::5]] = 0.0
    c.vs[used[2::7]] *= 1e12
    c.ks[used[::4]] = 0.0
    c.ks[used[1::4]] *= 30.0
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("ns,lens", [([1, 2], [150, 333]), ([20], [222]), ([80], [300])])
@pytest.mark.parametrize("small,large", [(0.0, 1e12), (1e-30, 1e8), (0.0, 1.0)])
def test_values_far_from_the_largest_score(ns, lens, small, large):
    # The pages with the largest scores (by up to 2^150) hold values of no or next to no size: what the output
    # is made of has probabilities that leave fp32's range long before the sums do.
    c = Case(ns, lens, 8, 2, 128, 16, "bf16", seed=18)
    used = c.table[c.table >= 0]
    c.ks[used[::3]] *= 25.0
    c.vs[used[::3]] *= small
    c.vs[used[1::3]] *= large
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("ns,lens", [([3, 2], [180, 67]), ([70], [150])])
def test_query_magnitudes(ns, lens):
    # Rows of very large, very small, zero and one-sided queries.
    c = Case(ns, lens, 4, 2, 128, 32, "bf16", seed=2)
    rows = c.qkv
    rows[0] *= 3.0e4
    rows[1] *= 1e-30
    rows[2] = 0.0
    rows[3] = rows[3].abs() + 2.0
    out, lse, scale = _run(c)
    c.check_attention(out, lse, scale)


@pytest.mark.parametrize("ns,lens", [([3, 1], [100, 30]), ([70, 1], [150, 30])])
def test_nan_stays_in_its_row(ns, lens):
    c = Case(ns, lens, 4, 2, 128, 32, "bf16", seed=2)
    c.qkv[1, 5] = float("nan")          # row 1, head 0
    out, lse, scale = _run(c)
    assert torch.isnan(out[1, 0].float()).all() and torch.isnan(lse[1, 0])
    got = out.clone()
    got[1, 0] = 0
    ref, _, e, _ = c.attention(scale)
    keep = np.ones((c.M, c.Hq), bool)
    keep[1, 0] = False
    err = np.abs(got.double().cpu().numpy() - ref)[keep]
    assert (err <= (e + UNIT[c.dtype] * (np.abs(ref) + e))[keep]).all()


@pytest.mark.parametrize("n,rows", [(1, [0]), (40, list(range(40)))])
def test_bad_indices_are_recorded_and_left_out(n, rows):
    c = Case([n, 1, 1], [120, 90, 40], 4, 2, 128, 32, "bf16", seed=6)
    c.tensors()
    table = c.step.page_table.clone()
    table[1, 1] = c.pages + 7           # a page that does not exist
    table[1, 2] = -5
    step = lib8.KV8Step(c.step.row0, c.step.kv_len, table, c.M, c.max_n)
    out = torch.zeros_like(c.q.contiguous())
    lib8.kv8_attention(c.cache, step, c.q, c.ws, out=out)
    assert c.status() == lib8.W8A8_DEV_BAD_INDEX and c.status() == 0
    c.check_attention(out, None, c.D ** -0.5, rows=rows + [n + 1])
    # What is left of sequence 1: its first page alone.
    d = Case([n, 1, 1], [120, 32, 40], 4, 2, 128, 32, "bf16", seed=6)
    d.table, d.kq, d.vq, d.ks, d.vs, d.qkv = c.table, c.kq, c.vq, c.ks, c.vs, c.qkv
    d.check_attention(out, None, c.D ** -0.5, rows=[n])
    # A length past the table, rows past the call's, a negative length: left out, the others stay right.
    for bad in (dict(kv_len=[120, 10**6, 40]), dict(kv_len=[120, -3, 40]), dict(row0=[0, n, n + 9, n + 2]),
                dict(row0=[0, n, n - 1, n + 2])):
        kv = torch.tensor(bad.get("kv_len", c.lens), dtype=torch.int32, device="cuda")
        r0 = torch.tensor(bad.get("row0", c.row0.tolist()), dtype=torch.int32, device="cuda")
        out.zero_()
        lib8.kv8_attention(c.cache, lib8.KV8Step(r0, kv, c.step.page_table, c.M, c.max_n), c.q, c.ws, out=out)
        assert c.status() == lib8.W8A8_DEV_BAD_INDEX
        if "kv_len" in bad:
            c.check_attention(out, None, c.D ** -0.5, rows=rows + [n + 1])


def test_replays_and_a_graph_with_other_lengths():
    c = Case([1, 3, 1, 40], [700, 2500, 90, 800], 8, 2, 128, 64, "bf16", seed=12)
    out, lse, scale = _run(c)
    first = out.clone()
    for _ in range(3):
        lib8.kv8_attention(c.cache, c.step, c.q, c.ws, out=out, lse=lse, scale=scale)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            lib8.kv8_attention(c.cache, c.step, c.q, c.ws, out=out, lse=lse, scale=scale)
    torch.cuda.synchronize()
    for lens in ([700, 2500, 90, 800], [1, 30, 64, 41], [650, 2499, 0, 40]):
        c.lens = lens
        c.step.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        c.check_attention(out, lse, scale)
    assert c.status() == 0


def test_on_another_stream():
    c = Case([1, 1], [513, 64], 8, 2, 128, 64, "bf16", seed=1).tensors()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(c.q.contiguous())
    lib8.kv8_attention(c.cache, c.step, c.q, c.ws, out=out, stream=s)
    s.synchronize()
    c.check_attention(out, None, c.D ** -0.5)


def test_cache_offsets_past_32_bits():
    # Five GB a side; the sequence's pages lie at both ends.
    D, P, H, pages = 128, 128, 8, 40000
    k, v = (torch.empty((pages, H, P, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty((pages, H), device="cuda") for _ in range(2))
    c = Case([1], [300], 8, H, D, P, "bf16", seed=3, spare=0).tensors()
    where = [0, 39999, 20001]
    for i, w in enumerate(where):
        src = int(c.table[0, i])
        k[w], v[w], ks[w], vs[w] = c.kc[src], c.vc[src], c.ksd[src], c.vsd[src]
    cache = lib8.KV8Cache(k, v, ks, vs)
    table = torch.tensor([where + [-1]], dtype=torch.int32, device="cuda")
    step = lib8.KV8Step(c.step.row0, c.step.kv_len, table, 1, 1)
    out = lib8.kv8_attention(cache, step, c.q, c.ws)
    c.check_attention(out, None, D ** -0.5)
    assert c.status() == 0


@pytest.mark.parametrize("dim,n,kv_heads,page", [(64, 1, 8, 64), (128, 1, 8, 64), (128, 3, 8, 32), (128, 6, 4, 128), (256, 1, 4, 16)])
def test_long_contexts_under_load(dim, n, kv_heads, page):
    # Every SM streams for long: runs of 32 granules of a warp and more, slots refilled while others still read
    # theirs.  Every row of the first pass against 64 bits, and every bit of the others against the first.
    gen = torch.Generator(device="cuda").manual_seed(dim + n)
    B, G, width = 64, 4, 7936 // page
    lens = torch.randint(5000, width * page + 1, (B,), device="cuda", generator=gen, dtype=torch.int32)
    shape = (B * width, kv_heads, page, dim)
    k, v = (torch.randint(1, 256, shape, device="cuda", generator=gen, dtype=torch.uint8) for _ in range(2))
    ks, vs = (0.01 * torch.exp(0.2 * torch.randn(shape[:2], device="cuda", generator=gen)) for _ in range(2))
    table = torch.randperm(B * width, device="cuda", generator=gen).to(torch.int32).view(B, width)
    row0 = torch.arange(B + 1, device="cuda", dtype=torch.int32) * n
    q = torch.randn(B * n, kv_heads * G, dim, device="cuda", generator=gen).bfloat16()
    cache, step = lib8.KV8Cache(k, v, ks, vs), lib8.KV8Step(row0, lens, table, B * n, n)
    ws = lib8.alloc_workspace(lib8.kv8_workspace_bytes(kv_heads * G, kv_heads, dim))
    first = lib8.kv8_attention(cache, step, q, ws).clone()
    for _ in range(20):
        assert torch.equal(lib8.kv8_attention(cache, step, q, ws), first)
    assert lib8.w8a8_workspace_status(ws) == 0
    scale = dim ** -0.5
    for b in range(B):
        L = int(lens[b])
        pages = table[b].long()
        per_token = [s[pages].double().repeat_interleave(page, 0)[:L].T for s in (ks, vs)]              # [heads, L]
        kk, vv = ((x[pages].double().sub_(128).transpose(0, 1).reshape(kv_heads, -1, dim)[:, :L] * s[:, :, None])
                  for x, s in zip((k, v), per_token))
        qq = q[b * n:(b + 1) * n].double().unflatten(1, (kv_heads, G)).permute(1, 2, 0, 3)              # [heads, G, n, dim]
        s = torch.einsum("hgnd,hld->hgnl", qq, kk) * scale
        seen = torch.arange(L, device="cuda")[None] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        w = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
        ref = torch.einsum("hgnl,hld->hgnd", w, vv)
        d = (scale * qq.abs().sum(-1) * 256 * (dim + 32) * 2.0 ** -24 * per_token[0].amax(1)[:, None, None]
             + s.abs().amax(-1) * 2.0 ** -21 + 2.0 ** -20)
        e = (2 * d + 2.0 ** -11 + (L / 16 + 64) * 2.0 ** -23)[..., None] * torch.einsum("hgnl,hld->hgnd", w, vv.abs())
        e = e + (L * 2.0 ** -25 * (w * per_token[1][:, None, None]).amax(-1) * 127)[..., None]
        got = first[b * n:(b + 1) * n].double().unflatten(1, (kv_heads, G)).permute(1, 2, 0, 3)
        assert ((got - ref).abs() <= e + UNIT["bf16"] * (ref.abs() + e)).all(), b


def test_no_rows_is_a_no_op():
    c = Case([1], [5], 4, 2, 64, 16).tensors()
    step = lib8.KV8Step(torch.zeros_like(c.step.row0), c.step.kv_len, c.step.page_table, 0, 1)
    q = c.q[:0]
    assert lib8.kv8_attention(c.cache, step, q, c.ws).shape == (0, 4, 64)
