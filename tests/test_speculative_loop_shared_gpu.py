"""The example loop with a page table as wide as a serving loop's (of the longest sequences it allows), so that its captured
step attends by the launches that share the prompt, which read some of the step's words before the work that they wait for by
themselves: behind the plan and the append of the same step, at every replay."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import UNIT, f64
from test_speculative_loop_gpu import _context64, _example

pytestmark = pytest.mark.gpu


def _wide(m, batch, prompt, window, max_len, page, seed):
    loop = m.SpeculativeLoop(batch, prompt, window, max_len, page_tokens=page, seed=seed)
    # Room for so many tokens (times kv heads) that a step is worth sharing whatever its rows.
    width = 700000 // (batch * page * m.KV_HEADS) + 1
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    table[:, :loop.table.shape[1]] = loop.table
    loop.table = table
    loop.step = lib8.KV8Step(loop.row0, loop.kv_len, table, loop.rows, window)
    assert batch * width * page * m.KV_HEADS > 700000 and window * m.Q_HEADS // m.KV_HEADS < 80
    return loop


@pytest.mark.parametrize("page", [16, 64])
def test_every_replay_attends_as_a_call_by_itself(page):
    m = _example()
    batch, window = 7, 4
    loop = _wide(m, batch, 330, window, 330 + 40, page, seed=3)
    turns = 0
    for turn in range(60):
        loop.run(torch.zeros(loop.rows, device="cuda") if turn % 3 == 2 else None)
        torch.cuda.synchronize()
        assert lib8.w8a8_workspace_status(loop.ws) == 0 and lib8.w8a8_workspace_status(loop.spec_ws) == 0
        M = int(loop.row0[-1])
        if M == 0:
            break
        turns += 1
        # The same call behind nothing that is still under way: the same bits.
        again = lib8.kv8_attention_shared(loop.cache, loop.step, loop.groups, loop.q, loop.ws)
        torch.cuda.synchronize()
        assert torch.equal(loop.context[:M], again[:M])
        row0, granted = loop.row0.tolist(), loop.granted.tolist()
        for b in range(batch):
            n = granted[b]
            if n == 0:
                continue
            r = slice(row0[b], row0[b] + n)
            out, mag = _context64(m, loop, b, n, f64(loop.q[r]))
            # weights are fp16 (2^-11), scores and sums fp32 (far less at these lengths), the output bf16
            e = 2.0 ** -10 * mag
            assert (np.abs(f64(loop.context[r]) - out) <= e + UNIT["bf16"] * (np.abs(out) + e)).all()
    assert M == 0 and turns >= 40 // window


def test_long_loops_of_many_requests():
    m = _example()
    loop = _wide(m, 24, 2048, 5, 2048 + 400, 64, seed=5)
    for turn in range(40):
        loop.run(torch.zeros(loop.rows, device="cuda") if turn % 2 else None)
        torch.cuda.synchronize()
        M = int(loop.row0[-1])
        again = lib8.kv8_attention_shared(loop.cache, loop.step, loop.groups, loop.q, loop.ws)
        alone = lib8.kv8_attention(loop.cache, loop.step, loop.q, loop.ws)
        torch.cuda.synchronize()
        assert M > 0 and torch.equal(loop.context[:M], again[:M])
        # Both are off by fp16 weights (2^-11 of what a row's largest value is, at most) and the outputs' rounding.
        a, b = loop.context[:M].float(), alone[:M].float()
        top = a.abs().amax() + b.abs().amax()
        assert (a - b).abs().max() <= 2 * (2.0 ** -10 + 2.0 ** -8) * top
    assert lib8.w8a8_workspace_status(loop.ws) == 0 and lib8.w8a8_workspace_status(loop.spec_ws) == 0
