"""The example layer end to end: prompts, then decode steps through its graph; the attention's output against the
plain form over what the cache holds, and the appended tokens against the layer's own keys and values."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import UNIT, f64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _attention64(m, layer, b, q):
    """q [heads, dim] of sequence b's last token over its cached tokens, in 64 bits: (out, sum of weighted magnitudes)."""
    n = int(layer.kv_len[b])
    P = layer.cache.page_tokens
    pages = layer.table[b, :-(-n // P)].long().cpu()
    val = lambda c, s: ((c.cpu()[pages].double() - 128) * s.cpu()[pages].double()[..., None, None]).transpose(1, 2).flatten(0, 1)[:n].numpy()   # noqa: E731
    k, v = val(layer.cache.k, layer.cache.k_scale), val(layer.cache.v, layer.cache.v_scale)
    out, mag = np.zeros_like(q), np.zeros_like(q)
    for h in range(m.Q_HEADS):
        s = k[:, h // (m.Q_HEADS // m.KV_HEADS)] @ q[h] * m.DIM ** -0.5
        w = np.exp(s - s.max())
        w /= w.sum()
        vv = v[:, h // (m.Q_HEADS // m.KV_HEADS)]
        out[h], mag[h] = w @ vv, w @ np.abs(vv)
    return out, mag


def test_prompts_then_decode_steps():
    m = _example()
    layer = m.AttentionLayer(3, 400, page_tokens=32, seed=5)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = lambda *s: torch.randn(*s, m.HIDDEN, device="cuda", generator=g).to(torch.bfloat16)   # noqa: E731
    for b, n in enumerate((1, 200, 131)):
        y = layer.prompt(b, x(n))
        assert y.shape == (n, m.HIDDEN) and torch.isfinite(y.float()).all()
    lens = [1, 200, 131]
    assert layer.kv_len.tolist() == lens
    for step in range(20):
        y = layer.decode(x(3))
        torch.cuda.synchronize()
        lens = [n + 1 for n in lens]
        assert layer.kv_len.tolist() == lens
        if step % 6 == 0:
            for b in range(3):
                out, mag = _attention64(m, layer, b, f64(layer.q[b]))
                # weights are fp16 (2^-11), scores and sums fp32 (far less at these lengths), the output bf16
                e = 2.0 ** -10 * mag
                assert (np.abs(f64(layer.context[b]) - out) <= e + UNIT["bf16"] * (np.abs(out) + e)).all()
        assert torch.isfinite(y.float()).all()
    assert lib8.w8a8_workspace_status(layer.ws) == 0
    assert lib8.w8a8_workspace_status(layer.qkv.ws) == 0
