"""spec_verify and spec_probs on the GPU: drawn tokens against exact whole numbers (equal), probabilities against 64 bits
(bounds: spec_util.probs)."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
import spec_util

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")   # noqa: E731


def _dist(rng, rows, V, dtype, sharp=3.0):
    x = rng.standard_normal((rows, V)) * sharp
    e = np.exp(x - x.max(1, keepdims=True))
    return torch.tensor((e / e.sum(1, keepdims=True)).astype(np.float32)).to(DT[dtype])


class Windows:
    def __init__(self, ns, V, dtype="f32", drafted=True, seed=0, behind=0, sharp=3.0):
        rng = np.random.default_rng(seed)
        self.ns, self.V, self.dtype = ns, V, dtype
        self.row0 = np.concatenate([[0], np.cumsum(ns)])
        R = int(self.row0[-1]) + behind
        self.R = R
        self.p = _dist(rng, R, V, dtype, sharp)
        self.q = _dist(rng, R, V, dtype, sharp) if drafted else None
        near = rng.random(R) < 0.5          # drafts that are like the target are accepted more often
        if drafted:
            self.q[near] = self.p[near].clone()
        # Tokens drawn from the draft.
        src = (self.q if drafted else self.p).double().numpy()
        cum = src.cumsum(1)
        drawn = np.minimum((cum <= rng.random(R)[:, None] * cum[:, -1:]).sum(1), V - 1)
        self.tokens = np.concatenate([[0], drawn[:-1]]) if R else drawn
        self.accept, self.sample = rng.random(R).astype(np.float32), rng.random(R).astype(np.float32)

    def run(self, strided=0, ws=None):
        d = "cuda"
        def rows(t):   # noqa: E306
            if t is None:
                return None
            wide = torch.full((self.R, self.V + strided), 0.5, dtype=t.dtype, device=d)
            wide[:, :self.V] = t.to(d)
            return wide[:, :self.V]
        self.ws = lib8.alloc_workspace(lib8.spec_workspace_bytes(len(self.ns), self.V)) if ws is None else ws
        nxt, take = torch.full((self.R,), -9, dtype=torch.int32, device=d), torch.full((len(self.ns),), -9, dtype=torch.int32, device=d)
        f = lambda x: torch.tensor(x, device=d)   # noqa: E731
        self.args = (rows(self.p), i32(self.tokens), i32(self.row0), f(self.accept), f(self.sample), self.ws)
        self.kw = dict(q=rows(self.q), next=nxt, take=take)
        lib8.spec_verify(*self.args, **self.kw)
        torch.cuda.synchronize()
        return nxt.tolist(), take.tolist()

    def expect(self):
        n = lambda t: None if t is None else t.float().numpy()   # noqa: E731
        nxt, take = spec_util.verify(n(self.p), n(self.q), self.tokens, self.row0.tolist(), self.accept, self.sample)
        return [-9 if x is None else x for x in nxt], take

    def check(self, status=0, **kw):
        got, want = self.run(**kw), self.expect()
        assert got[1] == want[1]
        assert got[0] == want[0]
        assert lib8.w8a8_workspace_status(self.ws) == status
        return got


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 128, 511, 513, 1000, 4097, 32000, 100003])
def test_windows(V, dtype, drafted):
    c = Windows([6, 1, 0, 8, 3, 2], V, dtype, drafted, seed=V)
    c.check()


@pytest.mark.parametrize("strided", [0, 1, 3, 4, 61])
@pytest.mark.parametrize("V", [64, 1003])
def test_strides_and_rows_of_no_sequence(V, strided):
    for dtype in ("f32", "bf16"):
        Windows([3, 5, 1], V, dtype, True, seed=strided, behind=4).check(strided=strided)


@pytest.mark.parametrize("seqs,V", [(64, 5003), (200, 777), (700, 130), (5000, 20)])
def test_many_sequences(seqs, V):
    rng = np.random.default_rng(seqs)
    Windows(rng.integers(0, 6, seqs).tolist(), V, "f32", True, seed=seqs).check()


@pytest.mark.parametrize("drafted", [True, False])
def test_large_vocabularies(drafted):
    Windows([2, 1], 1 << 18, "f32", drafted, seed=1).check()
    Windows([1, 3], 262143, "bf16", drafted, seed=2).check()


def test_long_windows():
    # Windows of more than a warp's tests, accepted to the end, and rejected past the first 32.
    for seed in range(4):
        c = Windows([70, 33, 34, 100], 40, "f32", True, seed=seed)
        c.q = c.p.clone()
        c.accept[:] = 0.999
        c.accept[[40, 70 + 31, 70 + 33 + 32]] = 0.0
        if seed % 2:
            c.q[45] = torch.roll(c.p[45], 1)
            c.accept[45] = 1 - 2.0 ** -24
        _, take = c.check()
        assert max(take) > 32


@pytest.mark.parametrize("u", [0.0, 2.0 ** -149, 1e-30, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 1.5, -0.5, float("nan"), float("inf")])
def test_random_numbers_at_their_ends(u):
    for V in (7, 3001):
        c = Windows([3, 2, 1, 4], V, "f32", True, seed=5)
        c.sample[:] = u
        c.check()
        c.sample[:] = 0.3
        c.accept[:] = u
        c.check()


def test_flat_rows():
    # Equal weights: the draw lies at a border for many random numbers.
    V = 4096
    c = Windows([1] * 64, V, "f32", False, seed=0)
    c.p[:] = 1.0 / V
    c.sample = (np.arange(64) / 64).astype(np.float32)
    got, _ = c.check()
    assert got == [64 * i for i in range(64)]


def test_rows_with_nothing_to_draw_from():
    # The residual empty: the target itself; the target empty too: none.
    c = Windows([2, 2, 2, 1, 2], 50, "f32", True, seed=3)
    c.accept[:] = 1.0
    c.q[:] = c.p.clone()
    c.p[4], c.p[6] = 0.0, 0.0
    got, take = c.check(status=lib8.W8A8_DEV_BAD_INDEX)
    assert got[4] == -1 and got[6] == -1 and take == [1, 1, 1, 1, 1] and got[0] >= 0
    c = Windows([2, 2], 50, "f32", False, seed=3)
    c.p[:] = 0.0
    c.p[0, c.tokens[1]], c.p[2, c.tokens[3]] = 0.5, 1.0
    c.accept[:] = [0.7, 0.0, 0.7, 0.0]
    c.p[3, 9] = 1e-30                  # below half a unit: no weight
    got, take = c.check(status=lib8.W8A8_DEV_BAD_INDEX)
    assert got == [c.tokens[1], -1, c.tokens[3], -1] and take == [1, 2]


def test_values_outside_the_unit_interval():
    c = Windows([3, 2, 4], 300, "f32", True, seed=9)
    flat = c.p.view(-1)
    flat[::7], flat[3::11], flat[5::13], flat[6::17] = float("nan"), -0.5, 2.0, float("inf")
    c.q.view(-1)[::5] = float("nan")
    c.check()


@pytest.mark.parametrize("token", [-1, 300, 2**31 - 1, -2**31])
@pytest.mark.parametrize("drafted", [True, False])
def test_tokens_outside_the_vocabulary(token, drafted):
    c = Windows([4, 3], 300, "f32", drafted, seed=9)
    c.accept[:] = 0.0
    c.tokens[[2, 5]] = token
    got, take = c.check(status=lib8.W8A8_DEV_BAD_INDEX)
    assert take == [2, 1]


@pytest.mark.parametrize("row0,want", [([0, 3, 2, 7], [3, 0, None]), ([-1, 3, 5, 7], [0, None, None]), ([0, 3, 5, 99], [None, None, 0])])
def test_rows_without_sense_are_left_out(row0, want):
    c = Windows([3, 2, 2], 300, "f32", True, seed=9)
    c.accept[:] = 0.0
    c.row0 = np.array(row0)
    _, take = c.run()
    assert lib8.w8a8_workspace_status(c.ws) == lib8.W8A8_DEV_BAD_INDEX
    assert all(w is None or w == t for w, t in zip(want, take))


def test_no_rows():
    ws = lib8.alloc_workspace(lib8.spec_workspace_bytes(3, 100))
    e = torch.empty(0, device="cuda")
    nxt, take = lib8.spec_verify(torch.empty(0, 100, device="cuda"), i32([]), i32([0, 0, 0, 0]), e, e, ws)
    assert nxt.shape == (0,) and take.tolist() == [0, 0, 0]
    assert lib8.spec_probs(torch.empty(0, 100, device="cuda")).shape == (0, 100)


def test_a_workspace_serves_calls_of_other_sizes_and_graphs():
    ws = lib8.alloc_workspace(max(lib8.spec_workspace_bytes(s, v) for s, v in ((1, 1 << 18), (700, 200), (6, 32000))))
    cs = [Windows([2], 1 << 18, seed=1), Windows([2] * 700, 200, seed=2), Windows([6] * 6, 32000, seed=3)]
    for c in cs * 2:
        c.check(ws=ws)
    c = cs[2]
    want = c.expect()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        lib8.spec_verify(*c.args, **c.kw)
    for turn in range(3):
        c.sample[:] = 0.1 + 0.3 * turn
        c.args[4].copy_(torch.tensor(c.sample))
        want = c.expect()
        g.replay()
        torch.cuda.synchronize()
        assert (c.kw["next"].tolist(), c.kw["take"].tolist()) == want
    assert lib8.w8a8_workspace_status(ws) == 0


def test_the_draws_follow_the_target():
    # What comes out of a window, accepted or drawn, is distributed as the target's first row, whatever the draft is.
    V, n = 12, 20000
    rng = np.random.default_rng(0)
    p, q = _dist(rng, 1, V, "f32", 1.0), _dist(rng, 1, V, "f32", 1.0)
    first = rng.choice(V, n, p=q[0].double().numpy() / q[0].double().sum().item())
    c = Windows([2] * n, V, "f32", True, seed=1)
    c.p[::2], c.q[::2] = p, q
    c.tokens[1::2] = first
    nxt, _ = c.run()
    count = np.bincount(np.array(nxt)[::2], minlength=V)
    want = p[0].double().numpy() * n
    # Six standard deviations of a count.
    assert (np.abs(count - want) <= 6 * np.sqrt(want) + 1).all()


# ------------------------------------------------------------------------------------------- probabilities
def _probs(x, inv=None, strided=0, out_strided=0):
    R, V = x.shape
    wide = torch.full((R, V + strided), float("inf"), dtype=x.dtype, device="cuda")
    wide[:, :V] = x.cuda()
    out = torch.full((R, V + out_strided), -3.0, device="cuda")
    lib8.spec_probs(wide[:, :V], None if inv is None else torch.tensor(inv, device="cuda"), out=out[:, :V])
    torch.cuda.synchronize()
    assert (out[:, V:] == -3.0).all()
    want, bound = spec_util.probs(x.double().numpy(), np.ones(R) if inv is None else np.asarray(inv, np.float64))
    got = out[:, :V].cpu().double().numpy()
    worst = (np.abs(got - want) / bound).max()
    assert worst <= 1.0, worst
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (2, 3), (5, 31), (4, 128), (3, 2047), (7, 4100), (2, 32000), (16, 32000), (3, 65537),
                                    (2, 100003), (40, 16384), (90, 16388), (160, 1001)])
def test_probabilities(rows, V, dtype):
    rng = np.random.default_rng(V)
    inv = (0.5 + rng.random(rows)).astype(np.float32)
    inv[rows // 2] = np.inf
    _probs(torch.tensor(rng.standard_normal((rows, V)).astype(np.float32) * 3).to(DT[dtype]), inv)


@pytest.mark.parametrize("rows,V", [(1, 131072), (320, 131072), (2, 1 << 18), (1, 262143), (1, 131073), (200, 140000), (160, 100003)])
def test_large_probabilities(rows, V):
    g = torch.Generator().manual_seed(V)
    x = torch.randn(rows, V, generator=g).mul_(3).to(torch.bfloat16)
    inv = np.linspace(0.6, 1.4, rows).astype(np.float32)
    if rows < 100:
        _probs(x, inv)
        return
    out = lib8.spec_probs(x.cuda(), torch.tensor(inv, device="cuda")).cpu()
    for r in range(0, rows, 13):
        want, bound = spec_util.probs(x[r:r + 1].double().numpy(), inv[r:r + 1].astype(np.float64))
        assert (np.abs(out[r].double().numpy() - want[0]) <= bound[0]).all()
    assert (out.double().sum(1) - 1).abs().max() < 1e-5


@pytest.mark.parametrize("strided,out_strided", [(0, 0), (4, 8), (1, 0), (0, 3), (5, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_probabilities(dtype, strided, out_strided):
    rng = np.random.default_rng(2)
    for V in (1000, 1001):
        _probs(torch.tensor(rng.standard_normal((5, V)).astype(np.float32)).to(DT[dtype]), None, strided, out_strided)


@pytest.mark.parametrize("inv", [1.0, 0.0, 1e-3, 50.0, 1e30, float("inf"), -1.0, float("nan")])
def test_masks_infinities_and_temperatures(inv):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rng = np.random.default_rng(1)
    for V in (9, 5000):
        x = torch.tensor(rng.standard_normal((9, V)).astype(np.float32) * 20)
        x[0] = -inf
        x[1, :] = -inf
        x[1, V // 2] = -3.0
        x[2, ::2] = low
        x[3] = low
        x[4, [1, V - 1]] = inf
        x[5, 3] = nan
        x[6] = nan
        x[7, :] = 2.5                    # all equal: the first for temperature 0
        x[8, : V - 1] = -inf
        got = _probs(x, np.full(9, inv, np.float32))
        assert (got[0] == 0).all() and (got[6] == 0).all() and got[1, V // 2] == 1


def test_the_first_of_the_largest():
    x = torch.zeros(6, 20000, dtype=torch.bfloat16)
    at = [0, 1, 777, 9999, 10000, 19998]
    for r, a in enumerate(at):
        x[r, a:] = 1.0
    got = lib8.spec_probs(x.cuda(), torch.full((6,), float("inf"), device="cuda"))
    assert got.argmax(1).tolist() == at and (got.sum(1) == 1).all() and (got.max(1).values == 1).all()


def test_probabilities_in_place_and_in_a_graph():
    x = torch.randn(20, 40000, device="cuda")
    want = lib8.spec_probs(x)
    y = x.clone()
    assert lib8.spec_probs(y, out=y) is y and torch.equal(y, want)
    out = torch.zeros_like(x)
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        lib8.spec_probs(x, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_probabilities_back_to_back():
    # Launches that begin while the one before ends, several rows a cluster.
    x = [torch.randn(160, 32768, device="cuda").to(torch.bfloat16) for _ in range(3)]
    want = [lib8.spec_probs(t) for t in x]
    outs = [torch.empty_like(w) for w in want]
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        for i in range(12):
            lib8.spec_probs(x[i % 3], out=outs[i % 3])
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
