"""A workspace of spec_verify made for the largest batch and vocabulary serves every smaller one."""
import pytest
import torch

import int8_weight_gemm_gb300 as lib8


@pytest.mark.parametrize("vocab", [1, 4096, 4097, 20000, 131072, 1 << 18])
def test_bytes_never_fall_with_the_sequences(vocab):
    sizes = [lib8.spec_workspace_bytes(s, vocab) for s in [*range(1, 1300), 5000, 65534, 65535]]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("seqs", [1, 2, 38, 64, 152, 300, 305, 608, 609, 4000])
def test_bytes_never_fall_with_the_vocabulary(seqs):
    sizes = [lib8.spec_workspace_bytes(seqs, v) for v in [*range(1, 1 << 18, 1021), 1 << 18]]
    assert sizes == sorted(sizes)


@pytest.mark.gpu
def test_a_workspace_of_many_sequences_serves_fewer():
    V, most = 20000, 305
    ws = lib8.alloc_workspace(lib8.spec_workspace_bytes(most, V))
    g = torch.Generator(device="cuda").manual_seed(2)
    p = lib8.spec_probs(torch.randn(most, V, device="cuda", generator=g))
    u = torch.rand(most, device="cuda", generator=g)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")   # noqa: E731
    def draw(n, ws):   # noqa: E306
        row0 = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        nxt, take = lib8.spec_verify(p[:n], i32(n), row0, u[:n], u[:n], ws)
        assert (take == 1).all() and lib8.w8a8_workspace_status(ws) == 0
        return nxt.tolist()
    all_of = draw(most, ws)
    for n in (304, 300, 203, 152, 90, 60, 38, 7, 1, most):
        own = lib8.alloc_workspace(lib8.spec_workspace_bytes(n, V))
        assert draw(n, ws) == draw(n, own) == all_of[:n]
