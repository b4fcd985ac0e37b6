"""The Python side of the attention-side entry points, on the CPU."""
import pytest
import torch

import int8_weight_gemm_gb300 as lib8


def test_workspace_bytes_follow_the_device(monkeypatch):
    # The library sizes a workspace by the current device's SMs: a value of one device does not stand for the next.
    class OfDevice:
        sms = 152

        def kv8_workspace_bytes(self, q_heads, kv_heads, head_dim):
            return 256 + self.sms * head_dim

    device = OfDevice()
    monkeypatch.setattr(lib8, "lib", lambda: device)
    assert lib8.kv8_workspace_bytes(6, 3, 64) == 256 + 152 * 64
    device.sms = 148
    assert lib8.kv8_workspace_bytes(6, 3, 64) == 256 + 148 * 64


def _raises(fragment, fn, *args, **kw):
    with pytest.raises(ValueError, match=fragment):
        fn(*args, **kw)


@pytest.mark.parametrize("other", [torch.int8, torch.bool, torch.float8_e4m3fn])
def test_the_cache_is_of_unsigned_bytes(other):
    k, s = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2))
    _raises("k: expected uint8", lib8.KV8Cache, k.view(other), k, s, s)
    _raises("v: expected uint8", lib8.KV8Cache, k, k.view(other), s, s)


def test_scales_rotations_and_sums_are_fp32():
    k, s = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2))
    _raises("k_scale: expected float32", lib8.KV8Cache, k, k, s.int(), s)
    _raises("v_scale: expected float32", lib8.KV8Cache, k, k, s, s.int())
    _raises("cos_sin: expected float32", lib8.QKPrep, torch.zeros((9, 64), dtype=torch.int32), 64)

    class Stub:          # what the call reads of the handles
        tokens, head_dim = 4, 64

    x, ws = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.uint8)
    _raises("lse: expected float32", lib8.kv8_attention, Stub, Stub, x, ws, lse=torch.zeros((4, 2), dtype=torch.int32))
