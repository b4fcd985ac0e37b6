"""The Python side of the attention-side entry points, on the CPU."""
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
