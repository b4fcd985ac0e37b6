"""Argument checks of the attention-side entry points, on the CPU: at the C entry (fake addresses, never used) and in
the Python binding."""
import ctypes

import pytest
import torch

import int8_weight_gemm_gb300 as lib8

A = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
WS = 1 << 30


def _cache(**kw):
    d = dict(k=1 << 20, v=1 << 20, k_scale=1 << 20, v_scale=1 << 20, pages=10, kv_heads=2, page_tokens=64, head_dim=128)
    d.update(kw)
    return ctypes.byref(lib8.KV8CacheT(**d))


def _step(**kw):
    d = dict(row0=1 << 20, kv_len=1 << 20, page_table=1 << 20, seqs=2, tokens=2, max_tokens=1, table_width=4)
    d.update(kw)
    return ctypes.byref(lib8.KV8StepT(**d))


def _prep(**kw):
    d = dict(gamma_q=1 << 20, gamma_k=1 << 20, cos_sin=1 << 20, eps=1e-6, rot_dim=128, max_pos=64, interleaved=0)
    d.update(kw)
    return ctypes.byref(lib8.QKPrepT(**d))


def _attention(cache=None, step=None, q=A, qs=1024, heads=8, out=A, os=1024, lse=A, scale=0.1, window=0, flags=0, dtype=0, ws=A, n=WS):
    return lib8.lib().kv8_attention(cache or _cache(), step or _step(), q, qs, heads, out, os, lse, ctypes.c_float(scale), window,
                                    flags, dtype, ws, n, None)


def _append(cache=None, step=None, prep=None, k=A, ks=256, v=A, vs=256, q=A, qs=1024, heads=8, qo=A, qos=1024, pos=A, dtype=0, ws=A, n=WS):
    return lib8.lib().kv8_append(cache or _cache(), step or _step(), prep or _prep(), k, ks, v, vs, q, qs, heads, qo, qos, pos,
                                 dtype, ws, n, None)


def _read(cache=None, step=None, k=A, ks=256, v=A, vs=256, dtype=0, ws=A, n=WS):
    return lib8.lib().kv8_read(cache or _cache(), step or _step(), k, ks, v, vs, dtype, ws, n, None)


def _qk(prep=None, q=A, qs=1024, heads=8, k=A, ks=256, kv=2, dim=128, pos=A, tokens=4, qo=A, qos=1024, ko=A, kos=256, dtype=0, ws=A, n=WS):
    return lib8.lib().qk_norm_rope(prep or _prep(), q, qs, heads, k, ks, kv, dim, pos, tokens, qo, qos, ko, kos, dtype, ws, n, None)


BAD_CACHES = [(dict(k=None), 1), (dict(v_scale=None), 1), (dict(pages=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=1025), 1),
              (dict(page_tokens=48), 2), (dict(page_tokens=8), 2), (dict(head_dim=96), 2), (dict(pages=2**25), 1),
              (dict(k=(1 << 20) + 8), 3), (dict(k_scale=(1 << 20) + 2), 3)]
BAD_STEPS = [(dict(row0=None), 1), (dict(kv_len=None), 1), (dict(page_table=None), 1), (dict(seqs=0), 1), (dict(seqs=70000), 1),
             (dict(tokens=-1), 1), (dict(max_tokens=0), 1), (dict(table_width=0), 1), (dict(table_width=2**25), 1),
             (dict(kv_len=(1 << 20) + 2), 3)]


@pytest.mark.parametrize("call", [_attention, _append, _read])
def test_cache_and_step_are_checked(call):
    for kw, code in BAD_CACHES:
        assert call(cache=_cache(**kw)) == code, kw
    for kw, code in BAD_STEPS:
        assert call(step=_step(**kw)) == code, kw
    assert call(ws=None) == 1 and call(ws=ODD) == 3 and call(n=0) == 4
    assert call(dtype=2) == 1
    assert call(step=_step(tokens=0)) == 0          # nothing to do, nothing launched


def test_attention_arguments():
    for kw, code in [(dict(q=None), 1), (dict(out=None), 1), (dict(q=ODD), 3), (dict(out=ODD), 3), (dict(qs=1023), 1), (dict(qs=1028), 3),
                     (dict(os=1000), 1), (dict(heads=7), 1), (dict(heads=0), 1), (dict(lse=ctypes.c_void_p((1 << 20) + 2)), 3),
                     (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
                     (dict(window=-1), 1), (dict(flags=2), 1), (dict(window=5, flags=lib8.KV8_FLAG_NOT_CAUSAL), 1),
                     (dict(n=lib8.kv8_workspace_bytes(8, 2, 128) - 1), 4)]:
        assert _attention(**kw) == code, kw


def test_append_and_read_arguments():
    for kw, code in [(dict(k=None), 1), (dict(v=None), 1), (dict(k=ODD), 3), (dict(ks=200), 1), (dict(vs=260), 3), (dict(q=None), 1),
                     (dict(qo=None), 1), (dict(qo=ODD), 3), (dict(heads=-1), 1), (dict(pos=ctypes.c_void_p((1 << 20) + 2)), 3)]:
        assert _append(**kw) == code, kw
    for kw, code in [(dict(k=None), 1), (dict(v=None), 1), (dict(k=ODD), 3), (dict(ks=200), 1), (dict(vs=260), 3)]:
        assert _read(**kw) == code, kw


@pytest.mark.parametrize("call", [_append, _qk])
def test_prep_is_checked(call):
    for kw, code in [(dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(rot_dim=-16), 1), (dict(rot_dim=144), 1), (dict(rot_dim=24), 2),
                     (dict(cos_sin=None), 1), (dict(max_pos=0), 1), (dict(gamma_k=(1 << 20) + 8), 3), (dict(cos_sin=(1 << 20) + 4), 3)]:
        assert call(prep=_prep(**kw)) == code, kw


def test_qk_arguments():
    for kw, code in [(dict(heads=-1), 1), (dict(heads=0, kv=0), 1), (dict(dim=80), 2), (dict(tokens=-1), 1), (dict(pos=None), 1),
                     (dict(q=None), 1), (dict(ko=None), 1), (dict(k=ODD), 3), (dict(qos=1020), 1), (dict(kos=260), 3), (dict(dtype=3), 1),
                     (dict(n=255), 4), (dict(tokens=0), 0)]:
        assert _qk(**kw) == code, kw


def test_workspace_bytes():
    assert lib8.kv8_workspace_bytes(8, 2, 128) >= 256
    assert lib8.lib().kv8_workspace_bytes(8, 0, 128) == 0
    assert lib8.lib().kv8_workspace_bytes(8, 2, 100) == 0
    assert lib8.lib().kv8_workspace_bytes(-1, 2, 128) == 0


def _raises(fragment, fn, *args, **kw):
    with pytest.raises(ValueError, match=fragment):
        fn(*args, **kw)


def test_handles_check_their_tensors():
    k = torch.zeros((3, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((3, 2))
    _raises("k: expected a CUDA tensor", lib8.KV8Cache, k, k, s, s)
    _raises("k: expected .pages", lib8.KV8Cache, k[0], k, s, s)
    _raises("v: expected shape", lib8.KV8Cache, k, k[:2], s, s)
    _raises("v: expected 1-byte", lib8.KV8Cache, k, k.short(), s, s)
    _raises("k_scale: expected shape", lib8.KV8Cache, k, k, s[:2], s)
    _raises("v_scale: expected 4-byte", lib8.KV8Cache, k, k, s, s.half())
    _raises("k: expected a contiguous", lib8.KV8Cache, k.transpose(1, 2), k.transpose(1, 2), s[:, :1].expand(3, 16), s)
    r, n, t = (torch.zeros(x, dtype=torch.int32) for x in ((3,), (2,), (2, 5)))
    _raises("row0: expected a CUDA tensor", lib8.KV8Step, r, n, t, 2, 1)
    _raises("row0: expected shape", lib8.KV8Step, n, n, t, 2, 1)
    _raises("kv_len: expected 4-byte", lib8.KV8Step, r, n.long(), t, 2, 1)
    _raises("kv_len: expected int32", lib8.KV8Step, r, n.float(), t, 2, 1)
    _raises("page_table: expected .seqs", lib8.KV8Step, r, n, t[0], 2, 1)
    tab, g = torch.zeros((9, 64)), torch.zeros(64, dtype=torch.bfloat16)
    _raises("cos_sin: expected a CUDA tensor", lib8.QKPrep, tab, 64)
    _raises("cos_sin: expected .max_pos, 32.", lib8.QKPrep, tab, 32)
    _raises("gamma_q: expected 2-byte", lib8.QKPrep, None, 0, tab[0])
    _raises("gamma_q: expected a CUDA tensor", lib8.QKPrep, None, 0, g)


def test_call_checks_come_before_the_library():
    class Stub:          # what the calls read of the handles
        tokens, kv_heads, head_dim = 4, 2, 64

        def check(self, dtype, dim):
            pass

    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    ws = torch.zeros(1024, dtype=torch.uint8)
    s = Stub()
    _raises("k: expected a CUDA tensor", lib8.kv8_append, s, s, s, x, x, ws)
    _raises("k: expected bfloat16 or float16", lib8.kv8_append, s, s, s, x.float(), x, ws)
    _raises("k: expected shape", lib8.kv8_append, s, s, s, x[:3], x, ws)
    _raises("q: expected shape", lib8.kv8_attention, s, s, x[:, :, :32], ws)
    _raises("q: expected contiguous heads", lib8.kv8_attention, s, s, x.transpose(0, 2).contiguous().transpose(0, 2), ws)
    _raises("q: expected a CUDA tensor", lib8.kv8_attention, s, s, x, ws)
    _raises("k: expected torch.bfloat16", lib8.qk_norm_rope, s, x, x.half(), None, ws)
    _raises("k_out: expected bfloat16 or float16", lib8.kv8_read, s, s, ws, k_out=x.float(), v_out=x)
