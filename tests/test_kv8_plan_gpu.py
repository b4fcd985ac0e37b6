"""kv8_plan on the GPU against the plain form in whole numbers: every output is equal."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
import spec_util

pytestmark = pytest.mark.gpu
OUT = ("row0", "kv_len", "held", "granted", "state", "positions", "slots", "seq_of")


class Plan:
    def __init__(self, seqs, P, seed, max_tokens=8, rows=None, spare=None, ended=0.1, idle=0.1, longest=700, ahead=3):
        rng = np.random.default_rng(seed)
        self.P, self.max_tokens = P, max_tokens
        self.lens = rng.integers(0, longest, seqs)
        self.ns = np.minimum(rng.integers(0, max_tokens + 1, seqs), self.lens)
        self.take = rng.integers(0, self.ns + 1)
        self.grow = np.where(rng.random(seqs) < idle, 0, rng.integers(0, max_tokens + 1, seqs))
        self.take[rng.random(seqs) < ended] = -1
        self.held = -(-self.lens // P) + rng.integers(0, ahead, seqs)
        self.pinned = np.minimum(rng.integers(0, 4, seqs), self.held)
        self.row0 = np.concatenate([[0], np.cumsum(self.ns)])
        width = int(self.held.max() + max_tokens // P + 2)
        used = int(self.held.sum())
        free = int(rng.integers(0, seqs * (max_tokens // P + 1) + 3)) if spare is None else spare
        pages = used + free
        ids = rng.permutation(pages)
        self.table = np.full((seqs, width), -7)
        self.table[np.arange(width)[None] < self.held[:, None]] = ids[:used]
        capacity = max(1, pages + int(rng.integers(0, 3)))
        self.ring = np.full(capacity, -5)
        head = int(rng.integers(0, capacity))
        self.ring[(head + np.arange(free)) % capacity] = ids[used:]
        self.state = [head, free]
        self.rows = seqs * max_tokens if rows is None else rows

    def gpu(self):
        i = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")   # noqa: E731
        self.d = {k: i(getattr(self, k)) for k in ("row0", "kv_len", "table", "held", "pinned", "take", "grow", "ring", "state")}
        self.step = lib8.KV8Step(self.d["row0"], self.d["kv_len"], self.d["table"], self.rows, self.max_tokens)
        self.pool = lib8.KV8Pool(self.d["ring"], self.d["state"])
        self.ws = lib8.alloc_workspace(256)
        return self

    @property
    def kv_len(self):
        return self.lens

    def expect(self, pinned=True):
        t, r = self.table.copy(), self.ring.copy()
        got = spec_util.plan(self.P, self.row0.tolist(), self.lens.tolist(), t, self.held.tolist(),
                             self.pinned.tolist() if pinned else [0] * len(self.lens), self.take.tolist(), self.grow.tolist(), r,
                             self.state, self.rows, self.max_tokens)
        return dict(zip(OUT, got), table=t, ring=r)

    def run(self, in_place=False, pinned=True, some=True):
        self.gpu()
        B, full = len(self.lens), lambda n: torch.full((n,), -9, dtype=torch.int32, device="cuda")   # noqa: E731
        per_row = {k: full(self.rows) for k in ("positions", "slots", "seq_of")} if some else {}
        granted = full(B) if some else None
        out = {} if in_place else dict(row0_out=full(B + 1), kv_len_out=full(B), held_out=full(B), pool_out=full(2))
        lib8.kv8_plan(self.step, self.P, self.pool, self.d["held"], self.d["take"], self.d["grow"], self.ws,
                      pinned=self.d["pinned"] if pinned else None, granted=granted, **per_row, **out)
        torch.cuda.synchronize()
        if in_place:
            out = dict(row0_out=self.d["row0"], kv_len_out=self.d["kv_len"], held_out=self.d["held"], pool_out=self.d["state"])
        else:
            for k in ("row0", "held", "state"):
                assert self.d[k].tolist() == np.asarray(getattr(self, k)).tolist()    # inputs are left alone
        got = dict(row0=out["row0_out"], kv_len=out["kv_len_out"], held=out["held_out"], state=out["pool_out"], table=self.d["table"],
                   ring=self.d["ring"], **per_row)
        if some:
            got["granted"] = granted
        return got

    def check(self, got, want=None):
        want = want or self.expect()
        for k, v in got.items():
            w = np.asarray(want[k])
            if k in ("positions", "slots", "seq_of"):
                w = np.concatenate([w, np.full(self.rows - len(w), -9)])      # behind the last row: as it was
            assert np.array_equal(v.cpu().numpy(), w), k


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("seqs", [1, 2, 31, 33, 64, 256, 257, 700, 1024, 1025, 2500])
def test_steps(seqs, P, in_place):
    for seed in range(2):
        c = Plan(seqs, P, seed * 1000 + seqs + P)
        c.check(c.run(in_place))
        assert lib8.w8a8_workspace_status(c.ws) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("seqs,longest", [(1, 900), (5, 300), (40, 5000), (300, 70), (1500, 40)])
def test_prompts_of_many_pages(seqs, longest, in_place):
    # Many rows: several CTAs, found by search; many new pages of one sequence.
    c = Plan(seqs, 16, seqs, max_tokens=2000 if seqs < 100 else 60, longest=longest, spare=seqs * 130)
    c.check(c.run(in_place))
    assert lib8.w8a8_workspace_status(c.ws) == 0


@pytest.mark.parametrize("seqs", [3, 60, 300, 1300])
@pytest.mark.parametrize("what", ["pages", "rows", "no pages", "no rows"])
def test_what_does_not_fit_is_not_granted(seqs, what):
    for seed in range(3):
        kw = {"pages": dict(spare=seqs // 3), "rows": dict(rows=2 * seqs + seed, spare=3 * seqs), "no pages": dict(spare=0),
              "no rows": dict(rows=0)}[what]
        c = Plan(seqs, 16, seed + seqs, max_tokens=20 if what != "rows" else 8, ahead=1, **kw)
        want = c.expect()
        got = c.run(in_place=seed == 1)
        c.check(got, want)
        assert lib8.w8a8_workspace_status(c.ws) == 0
        if what != "no pages" and seqs > 3:
            assert 0 < sum(g > 0 for g in want["granted"]) < (c.grow > 0).sum() or what == "no rows"


@pytest.mark.parametrize("rows", [1000, 1 << 22])
def test_sums_that_pass_31_bits(rows):
    c = Plan(6000, 128, 6, max_tokens=1 << 20, rows=rows, spare=9000, longest=300, ahead=1)
    assert c.grow.astype(np.int64).sum() > 2**31 - 1
    c.check(c.run(some=rows < 10**4))
    assert lib8.w8a8_workspace_status(c.ws) == 0


def test_optional_arguments():
    c = Plan(50, 32, 5)
    c.check(c.run(pinned=False, some=False), c.expect(pinned=False))


@pytest.mark.parametrize("field,value", [("take", 9999), ("grow", -1), ("grow", 9), ("kv_len", -3), ("kv_len", 0), ("held", -1), ("held", 10**6),
                                         ("pinned", -2)])
def test_numbers_without_sense_are_left_out(field, value):
    c = Plan(40, 16, 8, ended=0.0, idle=0.0)
    c.lens = np.maximum(c.lens, c.max_tokens)
    c.held = np.maximum(c.held, -(-c.lens // 16))
    if field == "kv_len":
        c.ns[7] = 4
        c.row0 = np.concatenate([[0], np.cumsum(c.ns)])
        c.lens[7] = value
    else:
        getattr(c, field)[7] = value
    want = c.expect()
    got = c.run()
    assert lib8.w8a8_workspace_status(c.ws) == lib8.W8A8_DEV_BAD_INDEX
    assert want["granted"][7] == 0
    c.check(got, want)


def test_a_pool_without_sense_hands_nothing_out():
    for state in ([-1, 3], [0, 10**6], [10**6, 1]):
        c = Plan(20, 16, 4, max_tokens=40, ended=0.0, ahead=1)
        c.gpu()
        real, c.state = c.state, state
        got = c.run()
        assert lib8.w8a8_workspace_status(c.ws) == lib8.W8A8_DEV_BAD_INDEX
        assert (c.held == got["held"].cpu().numpy()).all() and got["state"].tolist() == [0, 0]


def test_steps_in_a_graph_keep_every_page():
    # In place, captured once: windows grow and are taken back, sequences end and begin; no page is lost or given twice.
    c = Plan(70, 16, 3, ended=0.0, spare=400, longest=100)
    c.pinned[:] = 0
    c.gpu()
    d = c.d
    rows = {k: torch.full((c.rows,), -9, dtype=torch.int32, device="cuda") for k in ("positions", "slots", "seq_of")}
    call = lambda: lib8.kv8_plan(c.step, c.P, c.pool, d["held"], d["take"], d["grow"], c.ws, pinned=d["pinned"], **rows)   # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    rng = np.random.default_rng(5)
    pages = set(c.table[np.arange(c.table.shape[1])[None] < c.held[:, None]]) | {c.ring[(c.state[0] + i) % len(c.ring)] for i in range(c.state[1])}
    narrow = False          # whether a sequence has outgrown its row of the table: it gets nothing, and that is recorded
    for turn in range(60):
        n = np.diff(d["row0"].cpu().numpy())
        c.take, c.grow = rng.integers(0, n + 1), rng.integers(0, 9, 70)
        c.take[rng.random(70) < 0.05] = -1
        d["take"].copy_(torch.tensor(c.take, dtype=torch.int32))
        d["grow"].copy_(torch.tensor(c.grow, dtype=torch.int32))
        c.row0, c.lens, c.held, c.table, c.ring = (d[k].cpu().numpy() for k in ("row0", "kv_len", "held", "table", "ring"))
        c.state = d["state"].tolist()
        want = c.expect()
        narrow |= bool(((c.take >= 0) & (-(-(c.lens - n + c.take + c.grow) // c.P) > c.table.shape[1])).any())
        g.replay()
        torch.cuda.synchronize()
        for k in ("row0", "kv_len", "held", "state", "table", "ring"):
            assert np.array_equal(d[k].cpu().numpy(), np.asarray(want[k])), (turn, k)
        live = len(want["slots"])
        assert rows["slots"][:live].tolist() == list(want["slots"])
        t, h, ring, (head, free) = d["table"].cpu().numpy(), d["held"].cpu().numpy(), d["ring"].cpu().numpy(), d["state"].tolist()
        now = t[np.arange(t.shape[1])[None] < h[:, None]].tolist() + [ring[(head + i) % len(ring)] for i in range(free)]
        assert len(now) == len(set(now)) and set(now) == pages, turn
    assert lib8.w8a8_workspace_status(c.ws) == (lib8.W8A8_DEV_BAD_INDEX if narrow else 0)
