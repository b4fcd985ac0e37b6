"""qk_norm_rope, kv8_append and kv8_read on the GPU against plain forms.

Values that only pass through the quantisation are held to the bit (single IEEE steps).  Where a norm or a rotation
comes first, a value is an fp32 result of at most D / 8 + 8 additions, a division, a square root and three products
each rounded once, so it is within 2^-18 of its magnitude (the sum of the rotation's two products); a byte is then
within half a step plus 127 * 2^-17 (value and scale) of the exact quotient."""
import numpy as np
import pytest
import torch

import int8_weight_gemm_gb300 as lib8
from kv8_util import DT, TINY, UNIT, Case, away, f64, norm_turn, rotation

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18


def _prep(c, rot, interleaved, norm, max_pos, eps=1e-6):
    rng = np.random.default_rng(77)
    c.eps, c.rot, c.inter = eps, rot, interleaved
    c.tab = rotation(max_pos, rot) if rot else None
    c.gq, c.gk = (torch.tensor(rng.uniform(0.5, 1.5, c.D).astype(np.float32)).to(DT[c.dtype]) for _ in range(2)) if norm else (None, None)
    dev = lambda t: None if t is None else t.cuda()   # noqa: E731
    return lib8.QKPrep(None if c.tab is None else torch.from_numpy(c.tab).cuda(), rot, dev(c.gq), dev(c.gk), eps, interleaved)


def _turned(c, x, gamma, pos):
    return norm_turn(f64(x), None if gamma is None else f64(gamma), c.eps, c.tab, c.rot, c.inter, pos)


def _check16(c, got, x, gamma, pos):
    y, mag = _turned(c, x, gamma, pos)
    e = REL * mag
    assert (np.abs(f64(got) - y) <= e + UNIT[c.dtype] * (np.abs(y) + e) + TINY[c.dtype]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,rot,interleaved,norm", [(128, 128, False, True), (128, 64, True, False), (64, 64, False, False),
                                                      (64, 16, True, True), (64, 48, False, True), (256, 256, True, True),
                                                      (256, 96, False, False), (128, 0, False, True), (128, 0, False, False)])
@pytest.mark.parametrize("rows,q_heads,kv_heads", [(1, 8, 2), (13, 5, 1), (100, 3, 3)])
def test_qk_norm_rope(rows, q_heads, kv_heads, dim, rot, interleaved, norm, dtype):
    c = Case([rows], [rows], q_heads, kv_heads, dim, 16, dtype, seed=rows + dim, pad=8).tensors()
    prep = _prep(c, rot, interleaved, norm, 500)
    pos = c.rng.integers(0, 500, rows).astype(np.int32)
    c.qkv[0, :4] = 0.0
    c.tensors()
    posd = torch.from_numpy(pos).cuda()
    q, k = lib8.qk_norm_rope(prep, c.q, c.k, posd, c.ws)
    _check16(c, q, c.q, c.gq, pos)
    _check16(c, k, c.k, c.gk, pos)
    # In place, and into strided rows: the same bits.
    qi, ki = c.q.clone(), c.k.clone()
    lib8.qk_norm_rope(prep, qi, ki, posd, c.ws, q_out=qi, k_out=ki)
    wide = torch.full((rows, (q_heads + kv_heads) * dim + 8), float("nan"), dtype=DT[dtype], device="cuda")
    qs = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    ks = wide[:, q_heads * dim:-8].unflatten(1, (kv_heads, dim))
    lib8.qk_norm_rope(prep, c.q, c.k, posd, c.ws, q_out=qs, k_out=ks)
    for a in (qi, qs):
        assert torch.equal(a, q)
    for a in (ki, ks):
        assert torch.equal(a, k)
    assert torch.isnan(wide[:, -8:].float()).all()
    assert c.status() == 0


def test_zero_rows_and_zero_heads():
    c = Case([3], [3], 4, 2, 64, 16).tensors()
    prep = _prep(c, 64, False, True, 10)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    q, k = lib8.qk_norm_rope(prep, c.q[:0], c.k[:0], pos[:0], c.ws)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    c.q.zero_()          # a zero head: 0 / sqrt(eps)
    q, _ = lib8.qk_norm_rope(prep, c.q, c.k, pos, c.ws)
    assert (q == 0).all()
    step = lib8.KV8Step(torch.zeros_like(c.step.row0), c.step.kv_len, c.step.page_table, 0, 1)
    lib8.kv8_append(c.cache, step, prep, c.k[:0], c.v[:0], c.ws)
    k, v = lib8.kv8_read(c.cache, step, c.ws)
    assert k.shape == (0, 2, 64)


def test_positions_out_of_the_table_are_recorded():
    c = Case([2], [2], 4, 2, 64, 16).tensors()
    prep = _prep(c, 64, False, False, 10)
    q, _ = lib8.qk_norm_rope(prep, c.q, c.k, torch.tensor([3, 10], dtype=torch.int32, device="cuda"), c.ws)
    assert c.status() == lib8.W8A8_DEV_BAD_INDEX
    _check16(c, q[:1], c.q[:1], None, np.array([3]))


def _expect(c, x64, mag, cache_q, scales, exact32):
    """Bytes and scales that an append leaves, page by page; `exact32`: x64 holds fp32 values and every step is
    evaluated in fp32, so the result is exact.  Yields (page, head, slots kept, new slots, expected...)."""
    for b, (n, L) in enumerate(zip(c.ns, c.lens)):
        a, r = L - n, int(c.row0[b])
        for t in range(a - a % c.P, L, c.P):
            page = int(c.table[b, t // c.P])
            lo, hi = max(a - t, 0), min(L - t, c.P)
            for h in range(c.Hkv):
                x = x64[r + t + lo - a:r + t + hi - a, h]
                mg = mag[r + t + lo - a:r + t + hi - a, h]
                if n:
                    yield page, h, lo, hi, x, mg


def _check_append(c, x64, mag, before_q, before_s, after_q, after_s, exact32):
    touched = np.zeros(before_s.shape, bool)
    for page, h, lo, hi, x, mg in _expect(c, x64, mag, before_q, before_s, exact32):
        touched[page, h] = True
        got_q, got_s = after_q[page, h], float(after_s[page, h])
        old = before_s[page, h] if lo else np.float32(0)
        if exact32:
            fresh = np.float32(np.abs(x).max()) / np.float32(127)
            s = max(old, fresh) if lo else fresh
            assert np.float32(got_s) == s
            want = away((x.astype(np.float32) / s).astype(np.float64)).clip(-127, 127) if s else np.zeros_like(x)
            assert np.array_equal(got_q[lo:hi], want)
        else:
            fresh = np.abs(x).max() / 127
            s = max(float(old), fresh)
            assert abs(got_s - s) <= 2 * REL * (mg.max() / 127 + s)
            real = x / got_s if got_s else np.zeros_like(x)
            slack = (REL * mg / got_s if got_s else 0.0) + 127 * 2.0 ** -20
            assert (np.abs(got_q[lo:hi] - real.clip(-127, 127)) <= 0.5 + slack).all()
        if lo:      # the earlier tokens: at the new scale where it grew, else untouched
            was = before_q[page, h, :lo]
            if np.float32(got_s) > old:
                held = (was.astype(np.float32) * old).astype(np.float32) / np.float32(got_s)
                was = away(held.astype(np.float64)).clip(-127, 127)
            assert np.array_equal(got_q[:lo], was)
        assert np.array_equal(got_q[hi:], before_q[page, h, hi:])          # later slots are not written
    assert np.array_equal(after_q[~touched], before_q[~touched])
    assert np.array_equal(after_s[~touched].view(np.uint32), before_s[~touched].view(np.uint32))


CASES = [([1, 1, 1, 1], [1, 16, 17, 100]), ([1, 8, 0, 5, 3], [40, 8, 25, 130, 67]), ([70, 129], [70, 200]), ([300], [301]),
         ([16, 33], [32, 33])]


@pytest.mark.parametrize("ns,lens", CASES)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 128), (128, 32), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_without_rotation_is_exact(ns, lens, dim, page, dtype):
    for amp in (0.3, 1.0, 8.0):          # the page's scale stays, or grows for some pages, or for all
        c = Case(ns, lens, 4, 2, dim, page, dtype, seed=dim + page, pad=8, amp=amp).tensors()
        lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
        torch.cuda.synchronize()
        for x, q, s, qd, sd in ((c.k, c.kq, c.ks, c.kc, c.ksd), (c.v, c.vq, c.vs, c.vc, c.vsd)):
            x = f64(x)
            _check_append(c, x, np.abs(x), q, s, qd.cpu().numpy().astype(np.int32) - 128, sd.cpu().numpy(), True)
        assert c.status() == 0


@pytest.mark.parametrize("ns,lens", CASES)
@pytest.mark.parametrize("dim,page,rot,interleaved,norm,dtype", [(128, 64, 128, False, True, "bf16"), (64, 16, 32, True, False, "f16"),
                                                                 (256, 128, 256, False, True, "f16"), (128, 32, 64, True, True, "bf16"),
                                                                 (64, 128, 64, False, False, "bf16")])
@pytest.mark.parametrize("slots", [True, False])
def test_append_with_norm_and_rotation(ns, lens, dim, page, rot, interleaved, norm, dtype, slots):
    c = Case(ns, lens, 5, 1, dim, page, dtype, seed=dim + page + rot, amp=1.2).tensors()
    prep = _prep(c, rot, interleaved, norm, 700)
    pos = np.concatenate([np.arange(l - n, l) for n, l in zip(ns, lens)]).astype(np.int32)
    if not slots:
        pos = (pos * 2 + 1).astype(np.int32)
    q = lib8.kv8_append(c.cache, c.step, prep, c.k, c.v, c.ws, q=c.q, positions=None if slots else torch.from_numpy(pos).cuda())
    torch.cuda.synchronize()
    assert c.status() == 0
    _check16(c, q, c.q, c.gq, pos)
    y, mag = _turned(c, c.k, c.gk, pos)
    _check_append(c, y, mag, c.kq, c.ks, c.kc.cpu().numpy().astype(np.int32) - 128, c.ksd.cpu().numpy(), False)
    v = f64(c.v)
    _check_append(c, v, np.abs(v), c.vq, c.vs, c.vc.cpu().numpy().astype(np.int32) - 128, c.vsd.cpu().numpy(), True)


def test_zero_values_infinities_and_nan():
    c = Case([3], [3], 2, 1, 64, 16, "bf16").tensors()
    c.k.zero_()
    c.v[:] = 1.0
    c.v[0, 0, 3] = float("inf")
    c.v[1, 0, 4] = float("-inf")
    c.v[2, 0, 5] = float("nan")
    lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
    page = int(c.table[0, 0])
    assert float(c.ksd[page, 0]) == 0.0 and (c.kc[page, 0, :3] == 128).all()
    s = float(c.vsd[page, 0])
    assert np.isfinite(s) and s == float(np.float32(3.4028234e38) / np.float32(127))
    v = c.vc[page, 0, :3].cpu().numpy().astype(int) - 128
    assert v[0, 3] == 127 and v[1, 4] == -127 and v[2, 5] == 0 and np.count_nonzero(v) == 2


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 128)])
def test_read(dim, page, dtype):
    c = Case([1, 0, 70, 33], [40, 9, 90, 33], 2, 3, dim, page, dtype, seed=1).tensors()
    k, v = lib8.kv8_read(c.cache, c.step, c.ws, dtype=DT[dtype])
    for b, (n, L) in enumerate(zip(c.ns, c.lens)):
        for t in range(L - n, L):
            page_id, off, r = int(c.table[b, t // c.P]), t % c.P, int(c.row0[b]) + t - (L - n)
            for got, q, s in ((k, c.kq, c.ks), (v, c.vq, c.vs)):
                want = torch.from_numpy(q[page_id, :, off].astype(np.float32) * s[page_id][:, None]).to(DT[dtype])
                assert torch.equal(got[r].cpu(), want)
    wide = torch.full((c.M, 3 * dim + 8), float("nan"), dtype=DT[dtype], device="cuda")
    lib8.kv8_read(c.cache, c.step, c.ws, k_out=wide[:, :-8].unflatten(1, (3, dim)), v_out=v)
    assert torch.equal(wide[:, :-8].unflatten(1, (3, dim)), k) and torch.isnan(wide[:, -8:].float()).all()
    assert c.status() == 0


def test_bad_indices_write_nothing():
    c = Case([2, 2], [40, 20], 2, 1, 64, 16, "bf16").tensors()
    prep = _prep(c, 64, False, False, 100)
    table = c.step.page_table.clone()
    table[0, 2] = c.pages            # the page of both new tokens of sequence 0
    step = lib8.KV8Step(c.step.row0, c.step.kv_len, table, c.M, 2)
    before = c.kc.clone(), c.vc.clone()
    lib8.kv8_append(c.cache, step, prep, c.k, c.v, c.ws)
    assert c.status() == lib8.W8A8_DEV_BAD_INDEX
    own = int(c.table[1, 1])
    for now, was in ((c.kc, before[0]), (c.vc, before[1])):
        keep = [i for i in range(c.pages) if i != own]
        assert torch.equal(now[keep], was[keep]) and not torch.equal(now[own], was[own])
    for bad in (dict(kv_len=[1, 20]), dict(kv_len=[10**6, 20]), dict(row0=[0, 3, 2])):      # n > kv_len; past the table; rows past the call
        c.tensors()
        kv = torch.tensor(bad.get("kv_len", c.lens), dtype=torch.int32, device="cuda")
        r0 = torch.tensor(bad.get("row0", c.row0.tolist()), dtype=torch.int32, device="cuda")
        step = lib8.KV8Step(r0, kv, c.step.page_table, c.M, 2)
        lib8.kv8_append(c.cache, step, None, c.k, c.v, c.ws)
        lib8.kv8_read(c.cache, step, c.ws)
        assert c.status() == lib8.W8A8_DEV_BAD_INDEX
        first = [int(p) for p in c.table[0] if p >= 0]
        assert torch.equal(c.kc[first].cpu(), torch.from_numpy((c.kq[first] + 128).astype(np.uint8)))


def test_tokens_taken_back_are_written_over():
    # A verify window of 5 tokens, 3 of them rejected, then the next window over the same slots: the page's scale
    # stays large enough, and what is read back is the new tokens within half a step.
    c = Case([5], [37], 2, 2, 64, 32, "bf16", seed=3, amp=2.0).tensors()
    lib8.kv8_append(c.cache, c.step, None, c.k, c.v, c.ws)
    c.step.kv_len.fill_(39)                      # 34 kept, 5 new
    k2, v2 = c.k * 0.5, c.v * 3.0
    lib8.kv8_append(c.cache, c.step, None, k2.contiguous(), v2.contiguous(), c.ws)
    k, v = lib8.kv8_read(c.cache, c.step, c.ws)
    page = int(c.table[0, 1])
    for got, want, s in ((k, k2, c.ksd), (v, v2, c.vsd)):
        step = f64(s[page])[None, :, None]
        assert (np.abs(f64(got) - f64(want)) <= 0.5 * step + 2.0 ** -8 * np.abs(f64(want)) + 2.0 ** -8 * step).all()
    assert c.status() == 0


def test_append_then_attention_in_one_graph():
    """A decode loop as a captured graph: append (norm, rotation, quantisation) and attention over what was appended,
    replayed for successive tokens with the lengths advanced on the device."""
    c = Case([1, 1], [1, 1], 4, 2, 128, 16, "bf16", seed=21)
    width, pages = 4, 8
    kc, vc = (torch.zeros((pages, 2, 16, 128), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, 2), float("nan"), device="cuda") for _ in range(2))
    cache = lib8.KV8Cache(kc, vc, ks, vs)
    table = torch.tensor([[5, 2, 7, -1], [1, 0, 3, -1]], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    step = lib8.KV8Step(torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), kv_len, table, 2, 1)
    prep = _prep(c, 128, False, True, 64)
    ws = lib8.alloc_workspace(lib8.kv8_workspace_bytes(4, 2, 128))
    qkv = torch.zeros((2, 8 * 128), dtype=torch.bfloat16, device="cuda")
    q, k, v = (qkv[:, a:b].unflatten(1, (-1, 128)) for a, b in ((0, 512), (512, 768), (768, 1024)))
    qo, out = (torch.empty((2, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # Sequence 1 begins with a prompt of 9 tokens.
    prompt = torch.randn((9, 4, 128), device="cuda").to(torch.bfloat16)
    first = lib8.KV8Step(torch.tensor([0, 0, 9], dtype=torch.int32, device="cuda"), kv_len, table, 9, 9)
    lib8.kv8_append(cache, first, prep, prompt[:, :2], prompt[:, 2:], ws)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        kv_len.add_(1)
        lib8.kv8_append(cache, step, prep, k, v, ws, q=q, q_out=qo)
        lib8.kv8_attention(cache, step, qo, ws, out=out)
    for t in range(30):
        qkv.copy_(torch.randn((2, 8 * 128), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        c.ns, c.lens, c.P, c.table, c.M = [1, 1], [t + 1, t + 10], 16, table.cpu().numpy(), 2
        c.row0 = np.array([0, 1, 2], np.int32)
        c.kq, c.vq = (x.cpu().numpy().astype(np.int32) - 128 for x in (kc, vc))
        c.ks, c.vs = ks.cpu().numpy(), vs.cpu().numpy()
        _check16(c, qo, q, c.gq, np.array([t, t + 9]))
        c.qkv = torch.cat([qo.flatten(1).cpu(), torch.zeros(2, 512, dtype=torch.bfloat16)], 1)
        c.check_attention(out, None, 128 ** -0.5)
    assert lib8.w8a8_workspace_status(ws) == 0
