"""Argument checks of the speculative loop's entry points, on the CPU: at the C entry (fake addresses, never used) and in
the Python binding."""
import ctypes

import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from test_kv8_checks import A, BAD_CACHES, BAD_STEPS, ODD, WS, _cache, _raises, _step

BASE = 1 << 20
OFF = ctypes.c_void_p(BASE + 2)


def _groups(**kw):
    d = dict(seq0=BASE, prefix=BASE, groups=2, max_rows=4)
    d.update(kw)
    return ctypes.byref(lib8.KV8GroupsT(**d))


def _pool(**kw):
    d = dict(ring=BASE, state=BASE, capacity=10)
    d.update(kw)
    return ctypes.byref(lib8.KV8PoolT(**d))


def _out(**kw):
    d = {n: BASE for n, _ in lib8.KV8PlanT._fields_}
    d.update(kw)
    return ctypes.byref(lib8.KV8PlanT(**d))


def _shared(cache=None, step=None, groups=None, q=A, qs=1024, heads=8, out=A, os=1024, lse=A, scale=0.1, dtype=0, ws=A, n=WS):
    return lib8.lib().kv8_attention_shared(cache or _cache(), step or _step(), groups or _groups(), q, qs, heads, out, os, lse,
                                           ctypes.c_float(scale), dtype, ws, n, None)


def _plan(step=None, page=64, pool=None, held=A, pinned=A, take=A, grow=A, out=None, ws=A, n=WS):
    return lib8.lib().kv8_plan(step or _step(), page, pool or _pool(), held, pinned, take, grow, out or _out(), ws, n, None)


def _probs(x=A, xs=100, inv=A, out=A, os=100, rows=4, vocab=100, dtype=2):
    return lib8.lib().spec_probs(x, xs, inv, out, os, rows, vocab, dtype, None)


def _verify(p=A, ps=100, q=A, qs=100, tokens=A, row0=A, seqs=2, rows=4, vocab=100, accept=A, sample=A, next=A, take=A, dtype=2, ws=A, n=WS):
    return lib8.lib().spec_verify(p, ps, q, qs, tokens, row0, seqs, rows, vocab, accept, sample, next, take, dtype, ws, n, None)


def test_shared_attention_arguments():
    for kw, code in BAD_CACHES:
        assert _shared(cache=_cache(**kw)) == code, kw
    for kw, code in BAD_STEPS:
        assert _shared(step=_step(**kw)) == code, kw
    for kw, code in [(dict(seq0=None), 1), (dict(prefix=None), 1), (dict(groups=0), 1), (dict(groups=65536), 1), (dict(max_rows=0), 1),
                     (dict(max_rows=(1 << 22) + 1), 1), (dict(seq0=BASE + 2), 3), (dict(prefix=BASE + 1), 3)]:
        assert _shared(groups=_groups(**kw)) == code, kw
    for kw, code in [(dict(q=None), 1), (dict(out=None), 1), (dict(q=ODD), 3), (dict(out=ODD), 3), (dict(qs=1023), 1), (dict(qs=1028), 3),
                     (dict(os=1000), 1), (dict(heads=7), 1), (dict(heads=0), 1), (dict(lse=OFF), 3), (dict(scale=0.0), 1),
                     (dict(scale=float("nan")), 1), (dict(dtype=2), 1), (dict(ws=None), 1), (dict(ws=ODD), 3),
                     (dict(n=lib8.kv8_shared_workspace_bytes(2, 2, 8, 2, 128) - 1), 4), (dict(step=_step(tokens=0)), 0)]:
        assert _shared(**kw) == code, kw


def test_plan_arguments():
    for kw, code in BAD_STEPS:
        assert _plan(step=_step(**kw)) == code, kw
    for kw, code in [(dict(page=48), 2), (dict(page=0), 2), (dict(held=None), 1), (dict(take=None), 1), (dict(grow=None), 1), (dict(take=OFF), 3),
                     (dict(pinned=OFF), 3), (dict(ws=None), 1), (dict(ws=ODD), 3), (dict(n=255), 4)]:
        assert _plan(**kw) == code, kw
    for kw, code in [(dict(ring=None), 1), (dict(state=None), 1), (dict(capacity=0), 1), (dict(capacity=(1 << 30) + 1), 1), (dict(ring=BASE + 2), 3)]:
        assert _plan(pool=_pool(**kw)) == code, kw
    for kw, code in [(dict(row0=None), 1), (dict(kv_len=None), 1), (dict(held=None), 1), (dict(pool_state=None), 1), (dict(slots=BASE + 2), 3),
                     (dict(granted=BASE + 1), 3)]:
        assert _plan(out=_out(**kw)) == code, kw


def test_probability_arguments():
    for kw, code in [(dict(x=None), 1), (dict(out=None), 1), (dict(xs=99), 1), (dict(os=99), 1), (dict(rows=-1), 1), (dict(vocab=0), 1),
                     (dict(vocab=(1 << 18) + 1, xs=1 << 20, os=1 << 20), 1), (dict(dtype=3), 1), (dict(x=OFF), 3), (dict(out=OFF), 3),
                     (dict(inv=OFF), 3), (dict(x=ctypes.c_void_p(BASE + 1), dtype=0), 3), (dict(rows=0, x=None, out=None), 0)]:
        assert _probs(**kw) == code, kw


def test_verification_arguments():
    for kw, code in [(dict(p=None), 1), (dict(ps=99), 1), (dict(qs=99), 1), (dict(tokens=None), 1), (dict(row0=None), 1), (dict(accept=None), 1),
                     (dict(sample=None), 1), (dict(next=None), 1), (dict(take=None), 1), (dict(seqs=0), 1), (dict(seqs=65536), 1),
                     (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(vocab=(1 << 18) + 1, ps=1 << 20, qs=1 << 20), 1), (dict(dtype=5), 1),
                     (dict(p=OFF), 3), (dict(q=OFF), 3), (dict(tokens=OFF), 3), (dict(accept=OFF), 3), (dict(take=OFF), 3), (dict(ws=None), 1),
                     (dict(ws=ODD), 3), (dict(n=lib8.spec_workspace_bytes(2, 100) - 1), 4)]:
        assert _verify(**kw) == code, kw


def test_workspace_bytes():
    assert lib8.kv8_shared_workspace_bytes(64, 1, 32, 8, 128) > lib8.kv8_workspace_bytes(32, 8, 128)
    more = [lib8.kv8_shared_workspace_bytes(t, 3, 8, 2, 64) for t in (0, 1, 100, 5000)]
    assert more == sorted(more) and more[0] > 0
    L = lib8.lib()
    for bad in [(-1, 1, 8, 2, 64), (4, 0, 8, 2, 64), (4, 1, 7, 2, 64), (4, 1, 8, 2, 96), (4, 1, 0, 2, 64), (4, 70000, 8, 2, 64)]:
        assert L.kv8_shared_workspace_bytes(*bad) == 0
    assert lib8.spec_workspace_bytes(1, 1) > 256 and L.spec_workspace_bytes(0, 5) == 0 and L.spec_workspace_bytes(5, 0) == 0


def test_handles_check_their_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)   # noqa: E731
    _raises("seq0: expected a CUDA tensor", lib8.KV8Groups, i(3), i(2), 4)
    _raises("seq0: expected shape", lib8.KV8Groups, i(2), i(2), 4)
    _raises("prefix: expected 4-byte", lib8.KV8Groups, i(3), i(2).long(), 4)
    _raises("prefix: expected int32", lib8.KV8Groups, i(3), i(2).float(), 4)
    _raises("ring: expected a CUDA tensor", lib8.KV8Pool, i(9), i(2))
    _raises("state: expected shape", lib8.KV8Pool, i(9), i(3))
    _raises("ring: expected a contiguous", lib8.KV8Pool, i(18)[::2], i(2))


def test_call_checks_come_before_the_library():
    class Stub:          # what the calls read of the handles
        tokens, kv_heads, head_dim = 4, 2, 64

        class c:
            seqs, row0, kv_len, state = 2, 0, 0, 0

    s = Stub()
    x, ws = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(1024, dtype=torch.uint8)
    i = lambda *n: torch.zeros(n, dtype=torch.int32)   # noqa: E731
    _raises("q: expected a CUDA tensor", lib8.kv8_attention_shared, s, s, s, x, ws)
    _raises("q: expected shape", lib8.kv8_attention_shared, s, s, s, x[:3], ws)
    _raises("lse: expected float32", lib8.kv8_attention_shared, s, s, s, x, ws, lse=i(4, 2))
    _raises("held: expected a CUDA tensor", lib8.kv8_plan, s, 64, s, i(2), i(2), i(2), ws)
    _raises("take: expected shape", lib8.kv8_plan, s, 64, s, i(2), i(3), i(2), ws)
    _raises("grow: expected 4-byte", lib8.kv8_plan, s, 64, s, i(2), i(2), i(2).long(), ws)
    _raises("slots: expected shape", lib8.kv8_plan, s, 64, s, i(2), i(2), i(2), ws, slots=i(3))
    _raises("row0_out: expected shape", lib8.kv8_plan, s, 64, s, i(2), i(2), i(2), ws, row0_out=i(2))
    p = torch.zeros(4, 10)
    _raises("logits: expected a CUDA tensor", lib8.spec_probs, p)
    _raises("logits: expected .rows, vocab", lib8.spec_probs, p[0])
    _raises("logits: expected bfloat16, float16 or float32", lib8.spec_probs, p.double())
    _raises("logits: expected contiguous rows", lib8.spec_probs, p.t())
    _raises("inv_temp: expected shape", lib8.spec_probs, p, torch.zeros(3))
    _raises("out: expected torch.float32", lib8.spec_probs, p, out=p.half())
    f = torch.zeros(4)
    _raises("p: expected a CUDA tensor", lib8.spec_verify, p, i(4), i(3), f, f, ws)
    _raises("q: expected torch.float32", lib8.spec_verify, p, i(4), i(3), f, f, ws, q=p.half())
    _raises("q: expected shape", lib8.spec_verify, p, i(4), i(3), f, f, ws, q=p[:3])
    _raises("tokens: expected shape", lib8.spec_verify, p, i(5), i(3), f, f, ws)
    _raises("accept: expected shape", lib8.spec_verify, p, i(4), i(3), f[:3], f, ws)
    _raises("sample: expected float32", lib8.spec_verify, p, i(4), i(3), f, i(4), ws)
    _raises("take: expected shape", lib8.spec_verify, p, i(4), i(3), f, f, ws, take=i(3))


@pytest.mark.parametrize("u", [0.0, 2.0 ** -149, 2.0 ** -30, 0.3, 1 - 2.0 ** -24])
def test_the_host_form_draws_by_the_definition(u):
    import numpy as np

    import spec_util

    rng = np.random.default_rng(3)
    p = rng.random((1, 9)).astype(np.float32)
    p /= p.sum() * 1.01
    nxt, take = spec_util.verify(p, None, [0], [0, 1], [0.0], [np.float32(u)])
    cum = np.cumsum(p[0].astype(np.float64))
    assert take == [1] and nxt[0] == int((cum <= float(np.float32(u)) * cum[-1]).sum())
