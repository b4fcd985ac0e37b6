"""kv8_attention_shared beside sequences whose offsets make no sense: they are left out, and the others' rows are those of
kv8_attention (bounds: kv8_util)."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from test_kv8_shared_gpu import Shared

pytestmark = pytest.mark.gpu


def _case():
    lens = [128 + 1 + 7 * b % 90 for b in range(70)]
    return Shared([1] * 70, lens, [0, 35, 70], [128, 128], 8, 2, 128, 64, seed=6)


@pytest.mark.parametrize("at,value", [(20, -5), (36, -2**31), (65, 0), (70, -1), (70, 3), (1, 2**31 - 1), (0, -1), (40, 5), (35, -1)])
def test_rows_of_the_others_are_written(at, value):
    c = _case()
    good, good_lse = c.run()
    c.check_attention(good, good_lse, 128 ** -0.5)
    # The sequence that ends and the one that begins there: without sense (no rows, or not in the step), or longer than
    # max_tokens.  Nobody else's rows are theirs.
    left_out = [r for r in (at - 1, at) if 0 <= r < 70]
    real, c.row0[at] = c.row0[at], value
    out, lse = c.run(status=lib8.W8A8_DEV_BAD_INDEX)
    plain = torch.full_like(good, float("nan"))
    lib8.kv8_attention(c.cache, c.step, c.q, c.ws, out=plain)
    torch.cuda.synchronize()
    rest = np.setdiff1d(np.arange(70), left_out)
    assert torch.isfinite(plain[rest].float()).all()
    assert torch.isfinite(out[rest].float()).all()
    c.row0[at] = real
    out[left_out], lse[left_out] = good[left_out], good_lse[left_out]
    c.check_attention(out, lse, 128 ** -0.5)
