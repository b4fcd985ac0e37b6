"""kv8_attention_shared on the GPU against the plain 64-bit form over each sequence's own tokens (bounds: kv8_util), with
groups, prefixes and rows where it can go wrong."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import Case

pytestmark = pytest.mark.gpu
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731


class Shared(Case):
    """A Case whose groups (first sequences seq0, tokens in common prefix) hold the same pages."""

    def __init__(self, ns, lens, seq0, prefix, *heads, wide=True, **kw):
        super().__init__(ns, lens, *heads, **kw)
        if wide:
            # Room for so many tokens that the step is worth sharing.
            width = 700000 // (len(ns) * self.P * self.Hkv) + 1
            self.table = np.pad(self.table, ((0, 0), (0, max(0, width - self.table.shape[1]))), constant_values=-1)
            self.width = self.table.shape[1]
        self.seq0, self.prefix = seq0, prefix
        self.max_rows = 1
        self.share()
        for a, b in zip(seq0, seq0[1:]):
            self.max_rows = max(self.max_rows, sum(ns[a:b]))

    def share(self):
        for g, length in enumerate(self.prefix):
            a, b = self.seq0[g], self.seq0[g + 1]
            for s in range(a + 1, b):
                k = min(length // self.P, -(-self.lens[s] // self.P), -(-self.lens[a] // self.P))    # (pages that both have)
                self.table[s, :k] = self.table[a, :k]

    def tensors(self):
        super().tensors()
        self.groups = lib8.KV8Groups(i32(self.seq0), i32(self.prefix), self.max_rows)
        self.ws = lib8.alloc_workspace(lib8.kv8_shared_workspace_bytes(self.M, len(self.prefix), self.Hq, self.Hkv, self.D))
        return self

    def run(self, pad_out=0, status=0):
        self.tensors()
        out = torch.full((self.M, self.Hq * self.D + pad_out), float("nan"), dtype=self.q.dtype, device="cuda")
        view = out[:, :self.Hq * self.D].unflatten(1, (self.Hq, self.D))
        lse = torch.full((self.M, self.Hq), float("nan"), device="cuda")
        lib8.kv8_attention_shared(self.cache, self.step, self.groups, self.q, self.ws, out=view, lse=lse)
        torch.cuda.synchronize()
        assert self.status() == status
        if pad_out:
            assert torch.isnan(out[:, self.Hq * self.D:].float()).all()     # nothing past the heads is written
        return view, lse

    def check(self, **kw):
        out, lse = self.run(**kw)
        self.check_attention(out, lse, self.D ** -0.5)
        return out, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_single_tokens(dtype, dim, page):
    # Prefixes of whole pages, of a page and a bit, of less than a page, of none; a group of one.
    prefix = [2 * page, page + 5, page - 1, 0, 3 * page]
    seq0 = [0, 3, 5, 7, 9, 10]
    lens = [2 * page + 1, 2 * page + 130, 2 * page + 17, page + 40, page + 6, 40 + page, 90 + page, 33, 5, 3 * page + 1]
    Shared([1] * 10, lens, seq0, prefix, 8, 2, dim, page, dtype=dtype, seed=dim + page, pad=8).check(pad_out=16)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 1), (5, 5), (12, 4), (17, 1), (40, 2), (130, 1)])
def test_head_layouts(q_heads, kv_heads):
    Shared([1, 2, 1, 1], [150, 200, 129, 300], [0, 3, 4], [128, 200], q_heads, kv_heads, 128, 64, seed=q_heads).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ns,lens,seq0,prefix", [
    ([6, 3, 6, 1], [70, 100, 71, 90], [0, 4], [64]),                     # verify windows
    ([5, 0, 2], [70, 80, 66], [0, 3], [64]),                             # a sequence without rows
    ([8, 1, 3], [66, 100, 70], [0, 3], [64]),                            # rows that stand inside the prefix
    ([1, 2, 1], [40, 100, 90], [0, 3], [64]),                            # the first sequence does not hold it
    ([1, 2, 1], [0, 100, 90], [0, 3], [64]),
    ([2, 3, 1], [70, 0, 1], [0, 3], [64]),                               # others that hold nothing, or less
    ([64, 3], [64, 67], [0, 2], [64]),                                   # a prompt of the prefix itself
    ([70, 40, 25], [70 + 128, 168, 153], [0, 3], [128]),                 # prompts behind it: some hundred rows
    ([1, 1, 1, 1, 1], [100, 130, 90, 110, 300], [1, 4], [64]),           # sequences of no group
    ([2, 2, 2, 2], [100, 130, 90, 110], [0, 2, 2, 4], [96, 64, 32]),     # a group of none
])
def test_windows_and_prompts(ns, lens, seq0, prefix, dim):
    Shared(ns, lens, seq0, prefix, 8, 2, dim, 32, seed=sum(lens) + dim, pad=8).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ns,own,prefix,heads", [
    ([1] * 40, 200, [4096], (16, 2)),               # two tiles of rows; parts of a cut prefix
    ([1] * 70, 90, [6016], (8, 2)),                 # a part tile
    ([1, 3, 2], 60, [9024], (4, 1)),                # few rows, many parts
    ([130, 200], 250, [1024], (8, 2)),              # prompts: many tiles
    ([33] * 6, 40, [512], (8, 8)),                  # a kv head for each query head
])
def test_long_prefixes(ns, own, prefix, heads, dim):
    rng = np.random.default_rng(own)
    lens = [prefix[0] + n + int(rng.integers(0, own)) for n in ns]
    Shared(ns, lens, [0, len(ns)], prefix, *heads, dim, 64, seed=own + dim, amp=2.0).check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_groups(dim):
    # More items than SMs: prefixes that are not cut beside ones that are.
    rng = np.random.default_rng(dim)
    sizes = rng.integers(1, 5, 60)
    seq0 = np.concatenate([[0], np.cumsum(sizes)]).tolist()
    prefix = (rng.integers(0, 30, 60) * 16 + rng.integers(0, 16, 60)).tolist()
    prefix[7], prefix[30] = 2000, 1500
    ns = rng.integers(0, 4, seq0[-1]).tolist()
    lens = [prefix[g] + n + int(rng.integers(0, 50)) for g in range(60) for n in ns[seq0[g]:seq0[g + 1]]]
    Shared(ns, lens, seq0, prefix, 8, 4, dim, 16, seed=dim).check()


def test_many_sequences_and_groups():
    rng = np.random.default_rng(1)
    B = 1500
    seq0 = list(range(0, B + 1, 3))
    prefix = [32 + 16 * (g % 4) for g in range(len(seq0) - 1)]
    lens = [prefix[b // 3] + int(rng.integers(1, 40)) for b in range(B)]
    Shared([1] * B, lens, seq0, prefix, 2, 1, 64, 16, seed=4).check()


def test_values_of_very_different_sizes():
    # A prefix of large scores or values beside small ones of the sequences' own, and the reverse.
    for big in (0, 1):
        c = Shared([2, 1, 1], [600, 700, 530], [0, 3], [512], 8, 2, 128, 64, seed=big, amp=3.0)
        pre = c.table[0, :8]
        rest = np.setdiff1d(np.arange(c.pages), pre)
        c.ks[pre if big else rest] *= 8
        c.vs[rest if big else pre] *= 1e-3
        c.check()


def test_rows_behind_the_last_sequence_stay():
    c = Shared([1, 2, 1], [150, 200, 140], [0, 3], [128], 8, 2, 128, 64, seed=2)
    c.tensors()
    room = 9
    q = torch.randn(room, 8, 128, device="cuda").to(c.q.dtype)
    q[:c.M] = c.q
    step = lib8.KV8Step(c.step.row0, c.step.kv_len, c.step.page_table, room, 2)
    ws = lib8.alloc_workspace(lib8.kv8_shared_workspace_bytes(room, 1, 8, 2, 128))
    out, lse = torch.full_like(q, 7.0), torch.full((room, 8), 7.0, device="cuda")
    lib8.kv8_attention_shared(c.cache, step, c.groups, q, ws, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[c.M:] == 7).all() and (lse[c.M:] == 7).all()
    c.check_attention(out[:c.M], lse[:c.M], 128 ** -0.5)


@pytest.mark.parametrize("seq0,prefix,status", [([0, 9], [128], 4), ([-1, 3], [128], 4), ([2, 1], [128], 4), ([0, 3], [-64], 0),
                                                ([0, 3], [1 << 30], 0), ([5, 9], [64], 4), ([0, 3], [2**31 - 1], 0)])
def test_groups_without_sense_share_nothing(seq0, prefix, status):
    c = Shared([1, 2, 1], [150, 200, 140], [0, 3], [128], 8, 2, 128, 64, seed=2)
    c.seq0, c.prefix = seq0, prefix
    out, lse = c.run(status=status)
    c.check_attention(out, lse, 128 ** -0.5)


def test_bad_pages_and_rows_are_left_out():
    c = Shared([1, 2, 1, 1], [150, 200, 140, 90], [0, 3, 4], [128, 64], 8, 2, 128, 64, seed=2)
    good, _ = c.check()
    c.table[0, 1] = c.pages + 3                       # of the shared prefix
    out, _ = c.run(status=lib8.W8A8_DEV_BAD_INDEX)
    assert torch.equal(out[4:], good[4:]) and torch.isfinite(out.float()).all()
    c = Shared([1, 2, 1, 1], [150, 200, 140, 90], [0, 3, 4], [128, 64], 8, 2, 128, 64, seed=2)
    c.row0[1] = 77                                    # rows that are not there
    out, _ = c.run(status=lib8.W8A8_DEV_BAD_INDEX)
    assert torch.equal(out[3:], good[3:])


def test_a_graph_follows_lengths_and_prefixes():
    c = Shared([1] * 6, [300, 310, 330, 200, 222, 270], [0, 3, 6], [256, 128], 8, 2, 128, 64, seed=3)
    c.tensors()
    out, lse = torch.empty_like(c.q.contiguous()), torch.empty(c.M, c.Hq, device="cuda")
    call = lambda: lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws, out=out, lse=lse)   # noqa: E731
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for seq0, prefix, lens in ([0, 3, 6], [256, 128], None), ([0, 3, 6], [64, 192], [290, 257, 299, 200, 210, 193]), ([0, 2, 4], [128, 64], None):
        c.seq0, c.prefix = seq0, prefix
        if lens:
            c.lens = lens
        c.groups.seq0.copy_(i32(seq0))
        c.groups.prefix.copy_(i32(prefix))
        c.step.kv_len.copy_(i32(c.lens))
        c.share()                                     # what is now read as shared has to be the same
        c.step.page_table.copy_(torch.from_numpy(c.table))
        g.replay()
        torch.cuda.synchronize()
        assert c.status() == 0
        c.check_attention(out, lse, 128 ** -0.5)
        first = out.clone(), lse.clone()
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)


def test_lengths_that_change_between_two_calls():
    # Device work between two calls of one graph rewrites what the second and third launches read early.
    c = Shared([1] * 6, [300, 310, 330, 420, 322, 370], [0, 6], [256], 8, 2, 128, 64, seed=3)
    c.tensors()
    lens = [i32([300, 310, 330, 420, 322, 370]), i32([257, 290, 258, 270, 300, 310])]
    prefix = [i32([256]), i32([192])]
    outs = [torch.empty_like(c.q.contiguous()) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        for i in range(2):
            c.step.kv_len.copy_(lens[i])
            c.groups.prefix.copy_(prefix[i])
            lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws, out=outs[i])
    for _ in range(50):
        g.replay()
    torch.cuda.synchronize()
    assert c.status() == 0
    for i in range(2):
        c.lens = lens[i].tolist()
        c.check_attention(outs[i], None, 128 ** -0.5)


def test_the_workspace_serves_plain_attention_too():
    c = Shared([1] * 5, [700, 650, 680, 900, 640], [0, 5], [640], 8, 2, 128, 64, seed=5)
    c.tensors()
    for _ in range(2):
        a = lib8.kv8_attention(c.cache, c.step, c.q, c.ws)
        b = lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws)
        torch.cuda.synchronize()
        c.check_attention(a, None, 128 ** -0.5)
        c.check_attention(b, None, 128 ** -0.5)
    assert c.status() == 0


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_small_reads(dim):
    # (The launch of kv8_attention: every sequence reads its own pages.)
    Shared([1, 3, 1, 2], [150, 200, 140, 90], [0, 3, 4], [128, 64], 8, 2, dim, 64, seed=2, wide=False, pad=8).check(pad_out=16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("longest", [9, 16, 19, 20])
def test_windows_of_some_tens_of_rows(dim, longest):
    # Rows of a kv head in one tile of the sequences' own launch, and in several.
    rng = np.random.default_rng(longest)
    ns = [longest, 1, 0] + rng.integers(1, longest + 1, 9).tolist()
    lens = [512 + n + int(rng.integers(0, 300)) for n in ns]
    Shared(ns, lens, [0, 12], [512], 8, 2, dim, 32, seed=longest, pad=8).check(pad_out=16)


def test_another_stream():
    c = Shared([1] * 5, [700, 650, 680, 900, 640], [0, 5], [640], 8, 2, 128, 64, seed=5)
    c.tensors()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for how in (lambda: lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws, stream=s),):
        out = how()
        s.synchronize()
        c.check_attention(out, None, 128 ** -0.5)


def test_two_streams_at_once():
    # Two steps with workspaces of their own, under each other's load: the bits of each alone.
    cs = [Shared([1] * 40, [2048 + 17 * b + 1 for b in range(40)], [0, 40], [2048], 8, 2, 128, 64, seed=1),
          Shared([3] * 12, [1024 + 33 * b + 3 for b in range(12)], [0, 5, 12], [1024, 1000], 16, 4, 128, 32, seed=2)]
    alone, outs, graphs = [], [], []
    for c in cs:
        c.tensors()
        out = torch.empty_like(c.q.contiguous())
        lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws, out=out)
        torch.cuda.synchronize()
        alone.append(out.clone())
        outs.append(out)
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            for _ in range(20):
                lib8.kv8_attention_shared(c.cache, c.step, c.groups, c.q, c.ws, out=out)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, a, o in zip(cs, alone, outs):
        assert c.status() == 0 and torch.equal(a, o)
