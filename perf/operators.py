"""The attention-side operators of the library as measured cases: the rotation of queries and keys with their
norms (qk_norm_rope), the 8-bit paged key-value cache (kv8_append, kv8_read) and the attention over it
(kv8_attention).

`own` picks the side: False runs the operators' plain form (elementary torch operations in 32 bits, rounded once
at the end), True the library's entry points.  `exact` evaluates the definitions in 64 bits.

The cache: uint8 [pages, kv_heads, page_tokens, head_dim], a byte standing for (byte - 128) * scale with one fp32
scale for each (page, kv head).  A step names its rows: sequence b owns rows row0[b] ... row0[b + 1] - 1, whose
cache slots are the last ones below kv_len[b]."""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------------------- cases
def _attn(name, dtype, batch, n_min, n_max, len_min, len_max, q_heads, kv_heads, dim, page, window=0):
    return dict(name=name, op="attention", dtype=dtype, batch=batch, n_min=n_min, n_max=n_max, len_min=len_min,
                len_max=len_max, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, window=window)


def _append(name, dtype, batch, n_min, n_max, len_min, len_max, q_heads, kv_heads, dim, page, rot, interleaved, norm):
    return dict(name=name, op="append", dtype=dtype, batch=batch, n_min=n_min, n_max=n_max, len_min=len_min,
                len_max=len_max, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page, rot=rot,
                interleaved=interleaved, norm=norm)


def _rope(name, dtype, rows, q_heads, kv_heads, dim, rot, interleaved, norm):
    return dict(name=name, op="qk", dtype=dtype, rows=rows, q_heads=q_heads, kv_heads=kv_heads, dim=dim, rot=rot,
                interleaved=interleaved, norm=norm)


def listed():
    return [
        # One user's next token on one of four tensor-parallel ranks: the fused QKV product of N = 1536 columns is
        # 8 query heads and 2 key-value heads of 128.  Latency counts.
        _attn("attn one sequence", "bf16", 1, 1, 1, 517, 517, 8, 2, 128, 64),
        # A decode batch of 16 requests (the library's M = 16) of uneven lengths on a whole model's heads.
        _attn("attn batch 16", "bf16", 16, 1, 1, 257, 4099, 32, 8, 128, 64),
        # A full serving batch on long contexts: the cache read is what the step costs.
        _attn("attn batch 64 long", "bf16", 64, 1, 1, 6001, 8191, 32, 8, 128, 64),
        # One very long document, one token at a time: all the parallelism is along the cache.
        _attn("attn one long", "f16", 1, 1, 1, 131071, 131071, 32, 8, 128, 128),
        # A speculative-verify window of 6 tokens a request (T = 6 of the verify reads).
        _attn("attn verify window", "bf16", 16, 6, 6, 1001, 5003, 32, 8, 128, 32),
        # Sliding-window layers with a key-value head for each query head, short heads and small pages.
        _attn("attn sliding window", "f16", 32, 1, 4, 700, 4090, 16, 16, 64, 16, 1024),
        # A chunk of two prompts on top of what the cache holds: compute-bound.
        _attn("attn prompt chunk", "bf16", 2, 1900, 2048, 5800, 6144, 32, 8, 128, 64),
        # The append of a decode batch (with the queries' norm and rotation), then its pages read back.
        _append("append decode", "bf16", 16, 1, 1, 257, 4099, 32, 8, 128, 64, 128, False, True),
        # Verify windows of 1 to 8 tokens, partial interleaved rotation, no norm, small pages.
        _append("append verify", "f16", 32, 1, 8, 100, 2000, 16, 16, 64, 16, 32, True, False),
        # Whole prompts of about 4096 tokens.
        _append("append prompt", "bf16", 4, 3501, 4096, 3501, 4097, 32, 8, 128, 64, 128, False, True),
        # Queries and keys of a decode batch, for a cache of another kind.
        _rope("qk decode", "bf16", 16, 32, 8, 128, 128, False, True),
        # The same over a long prompt.
        _rope("qk prompt", "bf16", 16383, 32, 8, 128, 128, False, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    while kv_heads * group > 64:
        group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    heads = dict(q_heads=kv_heads * group, kv_heads=kv_heads, dim=dim)
    rot = rng.choice([dim, dim, dim // 2])
    tail = dict(rot=rot, interleaved=rng.random() < 0.4, norm=rng.random() < 0.6)
    op = rng.choice(["attention", "attention", "attention", "append", "qk"])
    if op == "qk":
        c = dict(op=op, dtype=dtype, rows=_log(rng, 1, 16000), **heads, **tail)
        while c["rows"] * (c["q_heads"] + kv_heads) * dim > 16383 * 40 * 128:
            c["rows"] = max(1, c["rows"] // 2 - 1)
        return c
    kind = rng.choice(["token", "token", "window", "prompt"])
    batch = _log(rng, 1, 64)
    n_max = 1 if kind == "token" else rng.randint(2, 16) if kind == "window" else _log(rng, 17, 2048)
    n_min = rng.choice([n_max, max(1, n_max // 2)])
    len_max = max(n_max, _log(rng, 16, 131071 if kind == "token" else 16000))
    len_min = rng.choice([len_max, max(1, len_max // 3)])
    if op == "append":
        # Four prompts of 4096 are the most: what is read back and what is appended both count.
        while batch * max(n_max, page) * (heads["q_heads"] + 4 * kv_heads) * dim > 4 * 4096 * 64 * 128 or \
                batch * len_max * kv_heads * dim > 64 * 8191 * 8 * 128:
            batch, len_max = max(1, batch // 2), max(n_max, len_max // 2)
            len_min = min(len_min, len_max)
        return dict(op=op, dtype=dtype, batch=batch, n_min=n_min, n_max=n_max, len_min=len_min, len_max=len_max,
                    page=page, **heads, **tail)
    # No more cache than 64 sequences of 8191 tokens, no more scores than the listed prompt chunk has.
    while batch * len_max * kv_heads * dim > 64 * 7000 * 8 * 128 or \
            batch * n_max * len_max * heads["q_heads"] * max(1, dim // 128) > 2 * 2048 * 5000 * 32:
        if batch > 1:
            batch //= 2
        elif n_max > 1:
            n_max = max(1, n_max // 2)
            n_min = min(n_min, n_max)
        else:
            len_max //= 2
            len_min = min(len_min, len_max)
    window = rng.choice([0, 0, 0, rng.randint(1, max(1, len_max))])
    return dict(op=op, dtype=dtype, batch=batch, n_min=n_min, n_max=n_max, len_min=len_min, len_max=len_max,
                page=page, window=window, **heads)


# ------------------------------------------------------------------------------------------- inputs
def _spread(lo, hi, batch, salt):
    """`batch` whole numbers of [lo, hi], the first one hi: uneven, and the same for every seed."""
    return [hi] + [lo + int(((b + salt) * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for b in range(1, batch)]


def _lengths(case):
    lens = _spread(case["len_min"], case["len_max"], case["batch"], 0)
    ns = [min(n, l) for n, l in zip(_spread(case["n_min"], case["n_max"], case["batch"], 3), lens)]
    return ns, lens


def _rows(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def _table(dim, gen):
    """Rotations: rows of cos, then sin, for `rows` positions."""
    rows, rot = dim
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * inv[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().cuda()


def _gamma(dim, gen, dt):
    return (0.6 + 0.8 * torch.rand(dim, device="cuda", generator=gen)).to(dt)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, D, Hq, Hkv = DT[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"]

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    S = dict(case)
    S["dt"] = dt
    if case["op"] == "qk":
        M = case["rows"]
        qkv = (randn(M, (Hq + 2 * Hkv) * D) * 1.5).to(dt)     # the fused product's output
        S["q"] = qkv[:, :Hq * D].view(M, Hq, D)
        S["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(M, Hkv, D)
        S["positions"] = torch.randint(0, 8192, (M,), device="cuda", generator=gen, dtype=torch.int32)
        S["table"] = _table((8192, case["rot"]), gen)
        S["gq"], S["gk"] = (_gamma(D, gen, dt), _gamma(D, gen, dt)) if case["norm"] else (None, None)
        S["q_out"], S["k_out"] = torch.empty(M, Hq, D, device="cuda", dtype=dt), torch.empty(M, Hkv, D, device="cuda", dtype=dt)
        if own:
            import int8_weight_gemm_gb300 as lib8
            S["prep"] = lib8.QKPrep(S["table"], case["rot"], S["gq"], S["gk"], 1e-6, case["interleaved"])
            S["ws"] = lib8.alloc_workspace(lib8.kv8_workspace_bytes(Hq, Hkv, D))
        return S

    P, B = case["page"], case["batch"]
    ns, lens = _lengths(case)
    M = sum(ns)
    width = -(-max(lens) // P) + 1
    used = [-(-l // P) for l in lens]
    pages = sum(used) + 3
    ids = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    pt = torch.full((B, width), -1, device="cuda", dtype=torch.int32)
    mask = torch.arange(width, device="cuda")[None] < torch.tensor(used, device="cuda")[:, None]
    pt[mask] = ids[:sum(used)]
    S.update(page_table=pt, row0=torch.from_numpy(_rows(ns)).cuda(), kv_len=torch.tensor(lens, device="cuda", dtype=torch.int32),
             tokens=M, max_tokens=max(ns), max_len=max(lens))

    def quants():
        return (randn(pages, Hkv, P, D) * 34).round_().clamp_(-127, 127).add_(128).to(torch.uint8)

    # Pages as appends leave them: the values' scale is the page's largest value over 127, 3 to 4 deviations wide.
    S["kc"], S["vc"] = quants(), quants()
    S["ks"] = 0.026 * torch.exp(0.1 * randn(pages, Hkv))
    S["vs"] = 0.026 * torch.exp(0.1 * randn(pages, Hkv))
    qkv = randn(M, (Hq + 2 * Hkv) * D).to(dt)
    S["q"] = qkv[:, :Hq * D].view(M, Hq, D)
    if case["op"] == "attention":
        S["scale"] = 1.0 / math.sqrt(D)
        S["out"] = torch.empty(M, Hq, D, device="cuda", dtype=dt)
        S["lse"] = torch.empty(M, Hq, device="cuda", dtype=torch.float32)
    else:
        S["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(M, Hkv, D)
        S["v"] = qkv[:, (Hq + Hkv) * D:].view(M, Hkv, D)
        S["table"] = _table((max(lens), case["rot"]), gen)
        S["gq"], S["gk"] = (_gamma(D, gen, dt), _gamma(D, gen, dt)) if case["norm"] else (None, None)
        S["q_out"] = torch.empty(M, Hq, D, device="cuda", dtype=dt)
        # What the append can change of a sequence: its new tokens and the earlier ones of the page they begin in.
        back = [n + (l - n) % P for n, l in zip(ns, lens)]
        S.update(back_row0=torch.from_numpy(_rows(back)).cuda(), back=sum(back), back_max=max(back))
        S["k_back"] = torch.empty(S["back"], Hkv, D, device="cuda", dtype=dt)
        S["v_back"] = torch.empty(S["back"], Hkv, D, device="cuda", dtype=dt)
    if own:
        import int8_weight_gemm_gb300 as lib8
        S["cache"] = lib8.KV8Cache(S["kc"], S["vc"], S["ks"], S["vs"])
        S["step"] = lib8.KV8Step(S["row0"], S["kv_len"], pt, M, max(ns))
        S["ws"] = lib8.alloc_workspace(lib8.kv8_workspace_bytes(Hq, Hkv, D))
        if case["op"] == "append":
            S["prep"] = lib8.QKPrep(S["table"], case["rot"], S["gq"], S["gk"], 1e-6, case["interleaved"])
            S["step_back"] = lib8.KV8Step(S["back_row0"], S["kv_len"], pt, S["back"], S["back_max"])
    return S


# ------------------------------------------------------------------------------------------- one pass
def run(S):
    if own:
        import int8_weight_gemm_gb300 as lib8
        if S["op"] == "qk":
            q, k = lib8.qk_norm_rope(S["prep"], S["q"], S["k"], S["positions"], S["ws"], q_out=S["q_out"], k_out=S["k_out"])
            return {"q": q, "k": k}
        if S["op"] == "append":
            q = lib8.kv8_append(S["cache"], S["step"], S["prep"], S["k"], S["v"], S["ws"], q=S["q"], q_out=S["q_out"])
            k, v = lib8.kv8_read(S["cache"], S["step_back"], S["ws"], k_out=S["k_back"], v_out=S["v_back"])
            return {"q": q, "k": k, "v": v}
        out = lib8.kv8_attention(S["cache"], S["step"], S["q"], S["ws"], scale=S["scale"], window=S["window"],
                                 out=S["out"], lse=S["lse"])
        return {"out": out, "lse": S["lse"]}
    if S["op"] == "qk":
        pos = S["positions"].long()
        return {"q": _norm_rope(S, S["q"], S["gq"], pos).to(S["dt"]), "k": _norm_rope(S, S["k"], S["gk"], pos).to(S["dt"])}
    if S["op"] == "append":
        return _plain_append(S)
    return _plain_attention(S)


def _norm_rope(S, x, gamma, pos):
    x = x.float()
    if gamma is not None:
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * gamma.float()
    R = S["rot"]
    cs = S["table"][pos]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if S["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., R:]], -1) if R < x.shape[-1] else turned


def _slots(row0, kv_len, rows):
    """The sequence and the cache slot of each of a step's rows."""
    r = torch.arange(rows, device=row0.device)
    seq = torch.searchsorted(row0[1:].contiguous(), r.to(row0.dtype), right=True)
    n = row0[1:] - row0[:-1]
    return seq, (kv_len - n)[seq].long() + r - row0[seq].long()


def _quantise(x, cache, scales, page, off, first, kept):
    """New tokens x [rows, heads, D] into their pages; `first`: the pages that hold `kept` earlier tokens each."""
    top = torch.zeros_like(scales).scatter_reduce(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    fresh = top / 127.0
    old = scales[first]
    grown = torch.maximum(old, fresh[first])
    # Earlier tokens of a page whose scale grows are held at the new scale.
    P = cache.shape[2]
    held = torch.arange(P, device=x.device)[None] < kept[:, None]
    ratio_on = (grown > old) & (kept > 0)[:, None]
    was = (cache[first].float() - 128.0) * old[..., None, None]
    again = _round(was / torch.where(grown > 0, grown, 1.0)[..., None, None]).add(128.0).to(torch.uint8)
    cache[first] = torch.where((held[:, None] & ratio_on[..., None])[..., None], again, cache[first])
    s = fresh.clone()
    s[first] = torch.where((kept > 0)[:, None], grown, fresh[first])
    scales[page] = s[page]
    at = s[page][..., None]
    q = _round(x / torch.where(at > 0, at, 1.0)).clamp(-127, 127) * (at > 0)
    cache[page, :, off] = (q + 128.0).to(torch.uint8)


def _round(x):
    """To the nearest whole number, halves away from zero."""
    return torch.trunc(x + torch.copysign(torch.full_like(x, 0.49999997), x))


def _plain_append(S):
    seq, slot = _slots(S["row0"], S["kv_len"], S["tokens"])
    P, pt = S["page"], S["page_table"].long()
    page, off = pt[seq, slot // P], slot % P
    start = (S["kv_len"] - (S["row0"][1:] - S["row0"][:-1])).long()
    first, kept = pt[torch.arange(S["batch"], device=pt.device), start // P], start % P
    _quantise(_norm_rope(S, S["k"], S["gk"], slot), S["kc"], S["ks"], page, off, first, kept)
    _quantise(S["v"].float(), S["vc"], S["vs"], page, off, first, kept)
    seq, slot = _slots(S["back_row0"], S["kv_len"], S["back"])
    page, off = pt[seq, slot // P], slot % P
    back = [((c[page, :, off].float() - 128.0) * s[page][..., None]).to(S["dt"]) for c, s in ((S["kc"], S["ks"]), (S["vc"], S["vs"]))]
    seq, slot = _slots(S["row0"], S["kv_len"], S["tokens"])
    return {"q": _norm_rope(S, S["q"], S["gq"], slot).to(S["dt"]), "k": back[0], "v": back[1]}


def _plain_attention(S):
    B, n, D, Hq, Hkv, P = S["batch"], S["max_tokens"], S["dim"], S["q_heads"], S["kv_heads"], S["page"]
    G, W = Hq // Hkv, -(-S["max_len"] // P)
    pages = S["page_table"][:, :W].clamp(min=0).long()

    def values(cache, scales):
        x = (cache[pages].float() - 128.0) * scales[pages][..., None, None]      # [B, W, Hkv, P, D]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * P, D)

    rows = (S["row0"][1:] - S["row0"][:-1]).long()
    i = torch.arange(n, device=pages.device)
    at = (S["row0"][:-1].long()[:, None] + i).clamp(max=S["tokens"] - 1)          # [B, n]
    q = S["q"][at].float().view(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    s = torch.matmul(q, values(S["kc"], S["ks"]).transpose(-1, -2)).mul_(S["scale"]).view(B, Hkv, n, G, W * P)
    j = torch.arange(W * P, device=pages.device)
    p = (S["kv_len"].long() - rows)[:, None] + i                                  # [B, n]
    seen = j[None, None] <= p[..., None]
    if S["window"]:
        seen &= j[None, None] > p[..., None] - S["window"]
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, n * G, W * P), values(S["vc"], S["vs"])).view(B, Hkv, n, G, D) / total
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, D)
    live = i[None] < rows[:, None]
    return {"out": o[live].to(S["dt"]), "lse": lse.permute(0, 2, 1, 3).reshape(B, n, Hq)[live]}


# ------------------------------------------------------------------------------------------- what a pass costs
def _visible(case):
    """For each sequence the cached tokens that some row sees, and the sum over rows of what each sees."""
    ns, lens = _lengths(case)
    w = case["window"] or (1 << 62)
    held = [l - max(0, l - n - w + 1) for n, l in zip(ns, lens)]
    seen = [sum(min(l - n + i + 1, w) for i in range(n)) for n, l in zip(ns, lens)]
    return ns, held, seen


def work(case):
    D, Hq, Hkv = case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "qk":
        M = case["rows"]
        # the rows in and out, the positions, and each position's row of the rotations (at most the whole table)
        return {"bytes": 4 * M * (Hq + Hkv) * D + 4 * M + 4 * min(M, 8192) * case["rot"], "flops": 8 * M * (Hq + Hkv) * D}
    P = case["page"]
    if case["op"] == "append":
        ns, lens = _lengths(case)
        M, back = sum(ns), sum(n + (l - n) % P for n, l in zip(ns, lens))
        touched = sum(-(-l // P) - (l - n) // P for n, l in zip(ns, lens))
        new = 2 * M * (Hq + 2 * Hkv) * D + 2 * M * Hq * D + 2 * M * Hkv * D + 8 * touched * Hkv + 4 * min(M, max(lens)) * case["rot"]
        read = back * Hkv * D * (2 + 4)
        return {"bytes": new + read, "flops": 8 * M * (Hq + 2 * Hkv) * D}
    ns, held, seen = _visible(case)
    pages = sum(-(-h // P) for h in held)
    return {"bytes": 2 * Hkv * D * sum(held) + 8 * Hkv * pages + 4 * pages + sum(ns) * Hq * (4 * D + 4), "flops": 4 * D * Hq * sum(seen)}


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    S = prepare(case, seed)
    D, Hq, Hkv = case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "qk":
        pos = S["positions"].long()
        return {"q": _turn64(S, S["q"], S["gq"], pos), "k": _turn64(S, S["k"], S["gk"], pos)}
    P, G = case["page"], Hq // Hkv
    ns, lens = _lengths(case)
    starts = _rows(ns)
    if case["op"] == "append":
        got = {"q": [], "k": [], "v": []}
        for b, (n, l) in enumerate(zip(ns, lens)):
            a, r = l - n, int(starts[b])
            pos = torch.arange(a, l, device="cuda")
            got["q"].append(_turn64(S, S["q"][r:r + n], S["gq"], pos))
            new = {"k": _turn64(S, S["k"][r:r + n], S["gk"], pos), "v": S["v"][r:r + n].double()}
            kept = a % P
            for name, cache, scales in (("k", S["kc"], S["ks"]), ("v", S["vc"], S["vs"])):
                for t in range(a - kept, l, P):                    # one page after the other
                    page = int(S["page_table"][b, t // P])
                    x = new[name][max(t, a) - a:min(t + P, l) - a]
                    s = x.abs().amax((0, 2)) / 127.0
                    old = torch.zeros(0, Hkv, D, device="cuda", dtype=torch.float64)
                    if t < a:
                        was = scales[page].double()
                        old = (cache[page, :, :kept].double() - 128.0).transpose(0, 1) * was[:, None]
                        s = torch.maximum(s, was)
                    old, x = (_away(y / s[:, None]).clamp(-127, 127) * s[:, None] for y in (old, x))
                    got[name].append(torch.cat([old, x]))
        return {k: torch.cat(v) for k, v in got.items()}
    if sum(2 * D * Hq * v for v in _visible(case)[2]) > 2.5e12:
        return None
    outs, lses = [], []
    for b, (n, l) in enumerate(zip(ns, lens)):
        pages = S["page_table"][b, :-(-l // P)].long()
        first = max(0, l - n - case["window"] + 1) if case["window"] else 0

        def values(cache, scales, h):
            x = (cache[pages, h].double() - 128.0) * scales[pages, h].double()[:, None, None]
            return x.reshape(-1, D)[first:l]

        r = int(starts[b])
        p = torch.arange(l - n, l, device="cuda")[:, None]
        j = torch.arange(first, l, device="cuda")[None]
        hidden = (j > p) | (j <= p - case["window"]) if case["window"] else j > p
        o = torch.empty(n, Hq, D, device="cuda", dtype=torch.float64)
        z = torch.empty(n, Hq, device="cuda", dtype=torch.float64)
        for h in range(Hkv):
            k, v = values(S["kc"], S["ks"], h), values(S["vc"], S["vs"], h)
            s = torch.einsum("ngd,td->gnt", S["q"][r:r + n, h * G:(h + 1) * G].double(), k) * S["scale"]
            s = s.masked_fill(hidden[None], -math.inf)
            z[:, h * G:(h + 1) * G] = torch.logsumexp(s, -1).T
            o[:, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", torch.softmax(s, -1), v)
        outs.append(o)
        lses.append(z)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _away(x):
    return torch.where(x < 0, -torch.floor(0.5 - x), torch.floor(x + 0.5))


def _turn64(S, x, gamma, pos):
    x = x.double()
    if gamma is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.double()
    R, y = S["rot"], x.clone()
    t = S["table"][pos].double()[:, None]
    even = slice(0, R, 2) if S["interleaved"] else slice(0, R // 2)
    odd = slice(1, R, 2) if S["interleaved"] else slice(R // 2, R)
    z = torch.complex(x[..., even].contiguous(), x[..., odd].contiguous()) * torch.complex(t[..., :R // 2].contiguous(), t[..., R // 2:].contiguous())
    y[..., even], y[..., odd] = z.real, z.imag
    return y
