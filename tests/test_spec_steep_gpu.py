"""spec_probs at finite temperatures next to 0: inv_temp whose product with log2 e passes the fp32 range, as
torch.nan_to_num(1 / temperature) makes of temperature 0 (bounds: spec_util.probs; there a product of a difference with
inv_temp and log2 e counts four roundings, of which the ones here take three: 4 and 1 / 4 are exact)."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
import spec_util

pytestmark = pytest.mark.gpu
MAX = torch.finfo(torch.float32).max
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inv", [2.0 ** 126, 2.0 ** 126 * 1.5, 2.0 ** 127, 2.35e38, 2.37e38, 3e38, MAX])
@pytest.mark.parametrize("V", [9, 4099, 5000, 140000])
def test_the_largest_finite_factors(V, inv, dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    rng = np.random.default_rng(V)
    x = torch.tensor(rng.standard_normal((8, V)).astype(np.float32) * 20)
    x[1] = -inf
    x[1, V // 2] = -3.0
    x[2, ::2] = low
    x[3, [1, V - 1]] = inf
    x[4, 3] = nan
    x[5] = 2.5                                        # all equal
    x[6] = -inf
    x[7] = torch.tensor(rng.random(V).astype(np.float32)) * 2e-38     # logits whose differences this factor resolves
    x = x.to(DT[dtype])
    got = lib8.spec_probs(x.cuda(), torch.full((8,), inv, device="cuda")).cpu().double().numpy()
    want, bound = spec_util.probs(x.double().numpy(), np.full(8, np.float32(inv), np.float64))
    assert (np.abs(got - want) <= bound).all()
    assert np.abs(got[[0, 1, 2, 3, 4, 5, 7]].sum(1) - 1).max() < 1e-5 and (got[6] == 0).all()


def test_temperature_zero_by_way_of_the_largest_number_draws_the_largest_logit():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 32000, generator=g)
    inv = torch.nan_to_num(1 / torch.zeros(3, device="cuda"))
    p = lib8.spec_probs(x.cuda(), inv)
    row0, half = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda"), torch.full((3,), 0.5, device="cuda")
    ws = lib8.alloc_workspace(lib8.spec_workspace_bytes(3, 32000))
    nxt, take = lib8.spec_verify(p, torch.zeros(3, dtype=torch.int32, device="cuda"), row0, half, half, ws)
    assert nxt.tolist() == x.argmax(1).tolist() and take.tolist() == [1, 1, 1] and lib8.w8a8_workspace_status(ws) == 0
