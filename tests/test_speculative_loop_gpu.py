"""The example loop end to end, its step in a captured graph: at every replay the plan, the attention, the probabilities
and the verification against the plain forms over what the step was given."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
import spec_util
from kv8_util import UNIT, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("speculative_loop", os.path.join(ROOT, "examples", "speculative_loop.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _context64(m, loop, b, rows, q):
    """q [rows, heads, dim] of sequence b's last tokens over its cached ones, in 64 bits: (out, sum of weighted magnitudes)."""
    L, P = int(loop.kv_len[b]), loop.page
    pages = loop.table[b, :-(-L // P)].long().cpu()
    val = lambda c, s: ((c.cpu()[pages].double() - 128) * s.cpu()[pages].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:L].numpy()   # noqa: E731
    k, v = val(loop.cache.k, loop.cache.k_scale), val(loop.cache.v, loop.cache.v_scale)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    G = m.Q_HEADS // m.KV_HEADS
    for i in range(rows):
        for h in range(m.Q_HEADS):
            n = L - rows + i + 1
            s = k[:n, h // G] @ q[i, h] * m.DIM ** -0.5
            w = np.exp(s - s.max())
            w /= w.sum()
            out[i, h], mag[i, h] = w @ v[:n, h // G], w @ np.abs(v[:n, h // G])
    return out, mag


@pytest.mark.parametrize("page", [16, 64])
def test_a_loop_of_captured_steps(page):
    m = _example()
    batch, window = 7, 4
    loop = m.SpeculativeLoop(batch, 330, window, 330 + 40, page_tokens=page, seed=3)
    ring, table = loop.pool.ring, loop.table
    own = batch * (table.shape[1] - loop.prefix // page)
    longest, turns = 0, 0
    for turn in range(60):
        before = {k: getattr(loop, k).cpu().numpy().copy() for k in ("row0", "kv_len", "table", "held", "pinned", "take", "grow")}
        ring0, state0 = ring.cpu().numpy().copy(), loop.pool.state.tolist()
        # Every third step accepts all drafts that the target can say at all.
        loop.run(torch.zeros(loop.rows, device="cuda") if turn % 3 == 2 else None)
        torch.cuda.synchronize()
        assert lib8.w8a8_workspace_status(loop.ws) == 0 and lib8.w8a8_workspace_status(loop.spec_ws) == 0
        want = spec_util.plan(page, *(before[k].tolist() if before[k].ndim == 1 else before[k] for k in ("row0", "kv_len", "table", "held",
                              "pinned", "take", "grow")), ring0, state0, loop.rows, window)
        row0, kv_len, held, granted, state, positions, _, seq_of = want
        for got, w in ((loop.row0, row0), (loop.kv_len, kv_len), (loop.held, held), (loop.granted, granted), (loop.pool.state, state),
                       (loop.table, before["table"]), (ring, ring0)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(w))
        M = row0[-1]
        assert loop.positions[:M].tolist() == positions and loop.seq_of[:M].tolist() == seq_of
        # No page is lost: what the requests hold beside the prompt's, and what is free.
        assert sum(max(0, h - p) for h, p in zip(held, before["pinned"].tolist())) + state[1] == own
        if turn % 9 == 0:
            for b in range(batch):
                n = granted[b]
                if n == 0:
                    continue
                r = slice(row0[b], row0[b] + n)
                out, mag = _context64(m, loop, b, n, f64(loop.q[r]))
                # weights are fp16 (2^-11), scores and sums fp32 (far less at these lengths), the output bf16
                e = 2.0 ** -10 * mag
                assert (np.abs(f64(loop.context[r]) - out) <= e + UNIT["bf16"] * (np.abs(out) + e)).all()
        p, bound = spec_util.probs(f64(loop.logits[:M]), f64(loop.inv_temp[:M]))
        assert (np.abs(f64(loop.p[:M]) - p) <= bound).all()
        nxt, take = spec_util.verify(loop.p[:M].cpu().numpy(), None, loop.tokens.tolist(), row0, loop.accept.tolist(), loop.sample.tolist())
        assert loop.next[:M].tolist() == nxt
        got = loop.take.tolist()
        assert all(g == t or (g == -1 and kv_len[b] - granted[b] + t + window > loop.max_len) for b, (g, t) in enumerate(zip(got, take)))
        longest, turns = max(longest, *take), turns + (M > 0)
        if M == 0:
            break
    # Every request ran to its end, drafts were accepted, and every page of theirs is free again.
    assert M == 0 and turns >= 40 // window and longest == window
    assert loop.pool.state[1].item() == own and (loop.kv_len == 0).all()
