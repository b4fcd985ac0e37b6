"""kv8_append and kv8_attention at the ends of their ranges, against plain 64-bit forms: values of the largest size, the
longest windows, the smallest weights, negative scales, positions out of the table.  The bounds are those of
kv8_util.Case.attention unless a test says otherwise."""
import copy

import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import DT, UNIT, Case, f64
from test_kv8_append_gpu import REL, _check16, _check_append, _prep, _turned

pytestmark = pytest.mark.gpu
LOG2E = 1.4426950408889634


def _last(c, n):
    """The last n rows of a case of one sequence, over the same cache."""
    d = copy.copy(c)
    d.ns, d.row0, d.M, d.max_n, d.qkv = [n], np.array([0, n], np.int32), n, n, c.qkv[c.M - n:]
    return d


def _take_cache(c):
    """The case's host copy of the cache = what the device holds of the pages in use."""
    used = c.table[c.table >= 0]
    for host, scales, dev, sdev in ((c.kq, c.ks, c.kc, c.ksd), (c.vq, c.vs, c.vc, c.vsd)):
        host[used] = dev.cpu().numpy().astype(np.int32)[used] - 128
        scales[used] = sdev.cpu().numpy()[used]


def _check(c, window=0, flags=0):
    c.tensors()
    lse = torch.full((c.M, c.Hq), float("nan"), device="cuda")
    out = lib8.kv8_attention(c.cache, c.step, c.q, c.ws, lse=lse, window=window, flags=flags)
    assert c.status() == 0
    c.check_attention(out, lse, c.D ** -0.5, window, not flags & lib8.KV8_FLAG_NOT_CAUSAL)
    return out, lse


def _ladder(c, length):
    """Queries a e_0 and keys y e_0: a page's logits are 0 (two pages out of three, the first two among them) or, in
    powers of two, one of 0 ... 16 that differs from row to row."""
    rows = np.arange(c.M * c.Hq) % 131 * (16 / 131) / LOG2E * c.D ** 0.5
    x = torch.zeros((c.M, c.Hq + 2 * c.Hkv, c.D))
    x[:, :c.Hq, 0] = torch.from_numpy(rows.reshape(c.M, c.Hq).astype(np.float32))
    high = (np.arange(length) // c.P) % 3 == 2
    return x, high


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 200])
def test_appended_infinities(dim, rows):
    # An infinity is held at the largest scale that an append makes (2^121).  Rows whose score on such a page passes
    # their reference by less than what moves it, beside rows that it moves, in both kernels.
    L = 200
    c = Case([L], [L], 8, 1, dim, 16, "bf16", seed=dim)
    x, high = _ladder(c, L)
    x[:, 8, 0] = torch.from_numpy(high.astype(np.float32))
    x[:, 9] = torch.from_numpy(c.rng.standard_normal((L, dim)).astype(np.float32))
    at = np.flatnonzero(high)[3::16]                 # one token of a page
    x[at[0::2], 9, 5] = float("inf")
    x[at[1::2], 9, 7] = float("-inf")
    c.qkv = x.flatten(1).to(DT["bf16"])
    c.tensors()
    lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
    _take_cache(c)
    assert (c.vs[c.table[c.table >= 0]] > 2.0 ** 121).any()
    _check(_last(c, rows))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 3, 200])
def test_the_largest_value_scales(dim, rows):
    # Scales next to fp32's largest number, which a cache filled by another program may have.
    L = 200
    c = Case([L], [L], 8, 1, dim, 16, "bf16", seed=dim)
    x, high = _ladder(c, L)
    c.qkv = x.flatten(1).to(DT["bf16"])
    pages = c.table[0, :-(-L // 16)]
    c.kq[pages] = 0
    c.kq[pages[2::3], :, :, 0] = 127
    c.ks[pages] = np.float32(1 / 127)
    c.vq[pages] = np.sign(c.vq[pages])
    c.vs[pages[0::3]] = 1e-30
    c.vs[pages[1::3]] = 1.0
    c.vs[pages[2::3]] = 3.4028234e38
    c.vq[pages[2::3], :, :8] = 0                     # (a page's tokens weigh the same: no weight of a large value is near 1)
    _check(_last(c, rows))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rows", [3, 193])
def test_an_appended_infinite_key_stays_with_the_rows_that_see_it(dim, rows):
    # The last token, alone on its page, has it: every row before it, and the other sequence, keep their results.
    c = Case([193, 40], [193, 90], 8, 1, dim, 16, "bf16", seed=dim)
    c.qkv[192, 8 * dim + 3] = float("inf")
    c.tensors()
    lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
    assert c.status() == 0
    _take_cache(c)
    assert c.ks[c.table[0, 12], 0] > 2.0 ** 121
    d = copy.copy(c)
    d.ns = [rows, 40]
    d.row0, d.M, d.max_n = np.array([0, rows, rows + 40], np.int32), rows + 40, max(rows, 40)
    d.qkv = c.qkv[193 - rows:]
    d.tensors()
    out = lib8.kv8_attention(d.cache, d.step, d.q, d.ws)
    assert d.status() == 0
    out[rows - 1] = 0
    d.check_attention(out, None, dim ** -0.5, rows=[r for r in range(d.M) if r != rows - 1])


@pytest.mark.parametrize("window", [2**30 - 1, 2**30, 2**31 - 2, 2**31 - 1])
@pytest.mark.parametrize("ns,lens", [([5, 1, 4], [2, 3, 0]), ([70, 3], [5, 90]), ([300], [40])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_longer_than_any_cache(ns, lens, window, dim):
    # With more rows than tokens the first row's position is below zero.
    c = Case(ns, lens, 4, 1, dim, 16, "bf16", seed=dim + len(ns))
    out, lse = _check(c, window=window)
    whole = lib8.kv8_attention(c.cache, c.step, c.q, c.ws)
    assert torch.equal(out, whole)


@pytest.mark.parametrize("far", [17.5, 21.5, 24.5])
@pytest.mark.parametrize("rows", [1, 3, 200])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_strong_tokens_without_values_over_a_flat_rest(dim, rows, far):
    # Every sixteenth token holds nearly all of the probability and no value; the output is made of the others, which
    # weigh 2^-far of it.  As Case.attention's bound, but that a weight is off by at most 2^-32 of the largest (fp16's
    # half spacing, 2^-25, where the largest is at least 2^7), not by 2^-25.
    L = 300
    c = Case([rows], [L], 8, 1, dim, 16, "f16", seed=dim)
    x = torch.zeros((rows, 10, dim))
    x[:, :8, 0] = far / LOG2E * dim ** 0.5
    c.qkv = x.flatten(1).to(DT["f16"])
    pages = c.table[0, :-(-L // 16)]
    c.kq[pages] = 0
    c.kq[pages, :, 0, 0] = 127
    c.ks[pages] = np.float32(1 / 127)
    c.vq[pages] = np.abs(c.vq[pages]) // 2 + 60
    c.vq[pages, :, 0] = 0
    c.vs[pages] = 1.0
    out, _ = _check(c)
    ref, _, e, _ = c.attention(dim ** -0.5)
    seen = np.arange(L - rows, L) + 1                # of a row
    w0 = 1 / (-(-seen // 16) + (seen - -(-seen // 16)) * 2.0 ** -far)
    slack = (seen * 127 * w0)[:, None, None]         # tokens times the largest weighted scale
    e = e - slack * 2.0 ** -25 * (1 - 2.0 ** -6) + slack * 2.0 ** -32
    assert (np.abs(f64(out) - ref) <= e + UNIT["f16"] * (np.abs(ref) + e)).all()


def _turn_signs(c):
    """Negative scales for two pages out of three: of the keys, of the values, of both in turn."""
    used = c.table[c.table >= 0]
    c.ks[used[0::3]] *= -1
    c.vs[used[0::3]] *= -1
    c.vs[used[1::3]] *= -1
    c.ks[used[2::5]] *= -1


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("ns,lens,window,flags", [([1, 1, 3], [150, 17, 333], 0, 0), ([20], [222], 0, 0), ([300], [333], 0, 0),
                                                  ([2, 40], [200, 100], 70, 0), ([5, 260], [90, 300], 0, lib8.KV8_FLAG_NOT_CAUSAL)])
def test_negative_scales(ns, lens, window, flags, dim):
    c = Case(ns, lens, 8, 2, dim, 16, "bf16", seed=dim + len(ns))
    _turn_signs(c)
    _check(c, window, flags)


@pytest.mark.parametrize("rows", [2, 100])
def test_negative_scales_far_from_the_largest_score(rows):
    # The largest scores stand on pages of no value size, so that weights come from their own exponents.
    c = Case([rows], [222], 8, 2, 128, 16, "bf16", seed=18)
    used = c.table[c.table >= 0]
    c.ks[used[::3]] *= 25.0
    c.vs[used[::3]] = 0.0
    c.vs[used[1::3]] *= -1e12
    _check(c)


@pytest.mark.parametrize("amp", [0.05, 1.0, 8.0])
@pytest.mark.parametrize("ns,lens", [([1, 8, 0, 5], [40, 8, 25, 130]), ([33, 3], [66, 30])])
def test_append_onto_pages_of_negative_scale(ns, lens, amp):
    # The page's tokens keep their values: its scale is the larger of its magnitude and the new tokens', and positive.
    c = Case(ns, lens, 4, 2, 64, 32, "bf16", seed=6, amp=amp)
    used = c.table[c.table >= 0]
    c.ks[used] *= -1
    c.vs[used[::2]] *= -1
    c.kq[used, :, 0, :4], c.vq[used, :, 0, 4:8] = -128, -128        # (byte 0, which no append writes)
    c.tensors()
    lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
    assert c.status() == 0
    for x, q, s, qd, sd in ((c.k, c.kq, c.ks, c.kc, c.ksd), (c.v, c.vq, c.vs, c.vc, c.vsd)):
        now_q, now_s = qd.cpu().numpy().astype(np.float64) - 128, sd.cpu().numpy().astype(np.float64)
        x = f64(x)
        for b, (n, L) in enumerate(zip(ns, lens)):
            for t in range(L - n - (L - n) % c.P if n else L, L, c.P):
                page, lo, hi = int(c.table[b, t // c.P]), max(L - n - t, 0), min(L - t, c.P)
                new = x[c.row0[b] + t + lo - (L - n):c.row0[b] + t + hi - (L - n)]
                fresh = np.abs(new).max((0, 2)) / 127
                want = np.maximum(fresh, np.abs(s[page]) if lo else 0)
                assert np.abs(now_s[page] - want).max() <= 2.0 ** -22 * want.max()
                step = now_s[page][:, None, None]
                got = now_q[page] * step
                # half a step and the fp32 roundings of 127 steps; -128 steps are held as -127 or 127
                e = step * (0.5 + 2.0 ** -15)
                assert (np.abs(got[:, lo:hi] - new.transpose(1, 0, 2)) <= e).all()
                was = q[page] * s[page].astype(np.float64)[:, None, None]
                assert (np.abs(got[:, :lo] - was[:, :lo]) <= e + step * 0.5 * (np.abs(q[page][:, :lo]) == 128)).all()


@pytest.mark.parametrize("dim,rot,interleaved", [(64, 64, False), (128, 128, False), (128, 64, True), (256, 256, False), (256, 96, False)])
@pytest.mark.parametrize("bad", [-1, 60, 2**31 - 1])
def test_rows_of_positions_out_of_the_table_are_left_out(dim, rot, interleaved, bad):
    # Rows 1, 4 and 8 stand at positions that the table does not have: their rows of the outputs are not written, their
    # keys enter the cache as zeros and do not count in a page's scale; their values, which do not rotate, are appended.
    n, L, P = 10, 40, 16
    out = np.zeros(n, bool)
    out[[1, 4, 8]] = True
    pos = np.where(out, bad, np.arange(n) + 3).astype(np.int32)
    good = np.where(out, 0, pos)
    c = Case([n], [L], 4, 2, dim, P, "bf16", seed=dim).tensors()
    prep = _prep(c, rot, interleaved, True, 60)
    c.k[torch.from_numpy(out).cuda()] *= 1000.0
    posd = torch.from_numpy(pos).cuda()
    qo, ko = torch.full_like(c.q.contiguous(), 7.0), torch.full_like(c.k.contiguous(), 7.0)
    lib8.qk_norm_rope(prep, c.q, c.k, posd, c.ws, q_out=qo, k_out=ko)
    assert c.status() == lib8.W8A8_DEV_BAD_INDEX and c.status() == 0
    for got, x, g in ((qo, c.q, c.gq), (ko, c.k, c.gk)):
        assert (got[torch.from_numpy(out).cuda()] == 7.0).all()
        _check16(c, got[torch.from_numpy(~out).cuda()], x[torch.from_numpy(~out).cuda()], g, good[~out])
    qo.fill_(7.0)
    lib8.kv8_append(c.cache, c.step, prep, c.k, c.v, c.ws, q=c.q, q_out=qo, positions=posd)
    assert c.status() == lib8.W8A8_DEV_BAD_INDEX
    assert (qo[torch.from_numpy(out).cuda()] == 7.0).all()
    _check16(c, qo[torch.from_numpy(~out).cuda()], c.q[torch.from_numpy(~out).cuda()], c.gq, good[~out])
    y, mag = _turned(c, c.k, c.gk, good)
    after_q, after_s = c.kc.cpu().numpy().astype(np.int32) - 128, c.ksd.cpu().numpy()
    for t in range((L - n) // P * P, L, P):
        page, lo, hi = int(c.table[0, t // P]), max(L - n - t, 0), min(L - t, P)
        rows = np.arange(t + lo - (L - n), t + hi - (L - n))
        for h in range(2):
            keep = rows[~out[rows]]
            old = float(c.ks[page, h]) if lo else 0.0
            s = max(old, np.abs(y[keep, h]).max() / 127)
            got_s = float(after_s[page, h])
            assert abs(got_s - s) <= 2 * REL * (mag[keep, h].max() / 127 + s)
            slack = REL * mag[keep, h] / got_s + 127 * 2.0 ** -20
            assert (np.abs(after_q[page, h, lo:hi][~out[rows]] - (y[keep, h] / got_s).clip(-127, 127)) <= 0.5 + slack).all()
            assert (after_q[page, h, lo:hi][out[rows]] == 0).all()
    v = f64(c.v)
    _check_append(c, v, np.abs(v), c.vq, c.vs, c.vc.cpu().numpy().astype(np.int32) - 128, c.vsd.cpu().numpy(), True)
