"""Plain 64-bit forms of the attention-side operators (numpy, from their definitions) and the case builder their GPU
tests share."""
import numpy as np
import torch

import int8_weight_gemm_gb300 as lib8

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}    # half a unit in the last place, relative: 2^-p of a p-bit significand
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}  # half the spacing of the smallest values


def f64(t):
    return t.detach().cpu().double().numpy()


def rotation(max_pos, rot):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(max_pos)[:, None] * inv[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def norm_turn(x, gamma, eps, table, rot, interleaved, pos):
    """x [rows, heads, D] in 64 bits; also the magnitude that bounds each value's rounding errors."""
    x = x.astype(np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * gamma
    y, mag = x.copy(), np.abs(x)
    if rot:
        ev = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        od = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        c, s = (table[pos][:, None, i].astype(np.float64) for i in (slice(0, rot // 2), slice(rot // 2, rot)))
        a, b = x[..., ev], x[..., od]
        y[..., ev], y[..., od] = a * c - b * s, b * c + a * s
        mag[..., ev], mag[..., od] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, mag


def away(x):
    return np.where(x < 0, -np.floor(0.5 - x), np.floor(x + 0.5))


class Case:
    """A cache with random contents, a step over it and its 16-bit tensors, on the GPU with host copies.

    Unused page-table entries are -1, unallocated pages hold NaN scales and the slots past a sequence's end hold
    arbitrary bytes, so a read that a kernel should not make shows."""

    def __init__(self, ns, lens, q_heads, kv_heads, dim, page, dtype="bf16", seed=0, spare=2, kscale=0.03, vscale=0.03,
                 pad=0, amp=1.0):
        rng = np.random.default_rng(seed)
        self.ns, self.lens, self.Hq, self.Hkv, self.D, self.P, self.dtype = ns, lens, q_heads, kv_heads, dim, page, dtype
        B = len(ns)
        used = [-(-l // page) for l in lens]
        self.width = max(1, max(used) + 1)
        self.pages = sum(used) + spare
        ids = rng.permutation(self.pages)
        self.table = np.full((B, self.width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u]
            at += u
        shape = (self.pages, kv_heads, page, dim)
        self.kq = np.clip(np.rint(rng.standard_normal(shape) * 34), -127, 127).astype(np.int32)
        self.vq = np.clip(np.rint(rng.standard_normal(shape) * 34), -127, 127).astype(np.int32)
        self.ks = (kscale * np.exp(0.2 * rng.standard_normal(shape[:2]))).astype(np.float32)
        self.vs = (vscale * np.exp(0.2 * rng.standard_normal(shape[:2]))).astype(np.float32)
        free = ids[at:]
        self.ks[free] = np.nan
        self.vs[free] = np.nan
        self.row0 = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.M = int(self.row0[-1])
        self.max_n = max(1, max(ns))
        self.rng = rng
        wide = (q_heads + 2 * kv_heads) * dim + pad
        self.qkv = torch.tensor(rng.standard_normal((self.M, wide)).astype(np.float32) * amp).to(DT[dtype])

    def tensors(self):
        d = "cuda"
        self.kc = torch.from_numpy((self.kq + 128).astype(np.uint8)).to(d)
        self.vc = torch.from_numpy((self.vq + 128).astype(np.uint8)).to(d)
        self.ksd, self.vsd = torch.from_numpy(self.ks).to(d), torch.from_numpy(self.vs).to(d)
        self.cache = lib8.KV8Cache(self.kc, self.vc, self.ksd, self.vsd)
        self.step = lib8.KV8Step(torch.from_numpy(self.row0).to(d), torch.tensor(self.lens, dtype=torch.int32, device=d),
                                 torch.from_numpy(self.table).to(d), self.M, self.max_n)
        self.ws = lib8.alloc_workspace(lib8.kv8_workspace_bytes(self.Hq, self.Hkv, self.D))
        dev = self.qkv.to(d)
        a, b = self.Hq * self.D, self.Hkv * self.D
        self.q = dev[:, :a].unflatten(1, (self.Hq, self.D))
        self.k = dev[:, a:a + b].unflatten(1, (self.Hkv, self.D))
        self.v = dev[:, a + b:a + 2 * b].unflatten(1, (self.Hkv, self.D))
        return self

    def status(self):
        return lib8.w8a8_workspace_status(self.ws)

    def values(self, b, h):
        """The cached keys and values of sequence b, kv head h, in 64 bits [len, D], and their scales per token."""
        pages = self.table[b, :-(-self.lens[b] // self.P)]
        out = []
        for q, s in ((self.kq, self.ks), (self.vq, self.vs)):
            sc = np.repeat(s[pages, h].astype(np.float64), self.P)[:self.lens[b]]
            out += [q[pages, h].reshape(-1, self.D)[:self.lens[b]].astype(np.float64) * sc[:, None], sc]
        return out

    def attention(self, scale, window=0, causal=True):
        """(out, lse) in 64 bits and the bounds of |gpu - out| before its last rounding, and of lse.

        The bounds follow the arithmetic: a logit is an fp32 dot product of D terms over (byte * query) products
        whose magnitudes are at most 255 |q|, times two scales, so its error is at most `d`; a weight is off by
        2 d relatively (numerator and denominator), by the rounding of the weights to fp16 (2^-11, or 2^-25 of the
        row's largest), and the sums of n tokens by n / 16 + 64 fp32 roundings (sixteen tokens to a matrix
        instruction)."""
        G = self.Hq // self.Hkv
        q = f64(self.qkv[:, :self.Hq * self.D]).reshape(self.M, self.Hq, self.D)
        out, lse = np.zeros_like(q), np.full((self.M, self.Hq), -np.inf)
        e_out, e_lse = np.zeros_like(q), np.zeros((self.M, self.Hq))
        for b, (n, L) in enumerate(zip(self.ns, self.lens)):
            if n == 0 or L == 0:
                continue
            j = np.arange(L)[None]
            p = (L - n + np.arange(n))[:, None]
            seen = np.ones((n, L), bool) if not causal else j <= p
            if window:
                seen &= j > p - window
            r = slice(self.row0[b], self.row0[b + 1])
            for h in range(self.Hkv):
                k, ks, v, vs = self.values(b, h)
                for hq in range(h * G, (h + 1) * G):
                    s = (q[r, hq] @ k.T) * scale
                    s = np.where(seen, s, -np.inf)
                    live = seen.any(1)
                    m = np.where(live, s.max(1, initial=-np.inf), 0.0)
                    w = np.exp(s - m[:, None])
                    l = w.sum(1)
                    w = w / np.where(live, l, 1.0)[:, None]
                    count = seen.sum(1)
                    out[r, hq] = w @ v
                    with np.errstate(divide="ignore"):
                        lse[r, hq] = np.where(live, m + np.log(l), -np.inf)
                    top = np.abs(np.where(seen, s, 0.0)).max(1)
                    d = (scale * np.abs(q[r, hq]).sum(1) * 256 * (self.D + 32) * 2.0 ** -24
                         * np.where(seen, ks[None], 0.0).max(1) + top * 2.0 ** -21 + 2.0 ** -20)
                    sums = (count / 16 + 64) * 2.0 ** -23
                    big = (w * vs[None]).max(1) * 127
                    e_out[r, hq] = ((2 * d + 2.0 ** -11 + sums)[:, None] * (w @ np.abs(v))
                                    + (count * 2.0 ** -25 * big)[:, None])
                    e_lse[r, hq] = 2 * d + sums + np.abs(np.where(live, lse[r, hq], 0.0)) * 2.0 ** -22
        return out, lse, e_out, e_lse

    def check_attention(self, got, lse, scale, window=0, causal=True, rows=slice(None)):
        ref, ref_lse, e, el = self.attention(scale, window, causal)
        got = f64(got)
        bound = e + UNIT[self.dtype] * (np.abs(ref) + e) + TINY[self.dtype]
        assert np.isfinite(got[rows]).all()
        worst = (np.abs(got - ref) / bound)[rows]
        assert worst.max(initial=0.0) <= 1.0, f"out: {worst.max():.3g} of the bound"
        if lse is not None:
            z = f64(lse)
            empty = np.isneginf(ref_lse)
            assert np.array_equal(np.isneginf(z)[rows], empty[rows])
            ok = np.abs(np.where(empty, 0.0, z) - np.where(empty, 0.0, ref_lse)) <= el
            assert ok[rows].all()
