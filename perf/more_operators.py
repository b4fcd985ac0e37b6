"""The operators of a speculative decoding loop around the 8-bit paged cache as measured cases: attention for sequences
that share a long prefix (kv8_attention_shared), the plan of the next step from the lengths (kv8_plan: page tables, row
offsets, positions, slots), the probabilities of a vocabulary from its logits (spec_probs) and the verification of drafted
tokens against them (spec_verify).

`own` picks the side: False runs the operators' plain form (elementary torch operations in 32 bits, rounded once at the
end; the verification in 64, as a drawn token depends on where a sum of a whole vocabulary lies), True the library's
entry points.  `exact` evaluates the definitions in 64 bits.

A step's rows are those of perf/operators.py: sequence b owns rows row0[b] ... row0[b + 1] - 1, whose cache slots are the
last ones below kv_len[b]; a cached byte stands for (byte - 128) * scale with one fp32 scale for each (page, kv head)."""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases
def _shared(name, dtype, batch, groups, n_min, n_max, prefix_min, prefix_max, tail_min, tail_max, q_heads, kv_heads, dim, page):
    return dict(name=name, op="shared", dtype=dtype, batch=batch, groups=groups, n_min=n_min, n_max=n_max,
                prefix_min=prefix_min, prefix_max=prefix_max, tail_min=tail_min, tail_max=tail_max, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page)


def _plan(name, batch, n_max, prompt_max, prompts, ended, len_min, len_max, page):
    return dict(name=name, op="plan", batch=batch, n_max=n_max, prompt_max=prompt_max, prompts=prompts, ended=ended,
                len_min=len_min, len_max=len_max, page=page)


def _verify(name, dtype, batch, n_min, n_max, vocab, drafted):
    return dict(name=name, op="verify", dtype=dtype, batch=batch, n_min=n_min, n_max=n_max, vocab=vocab, drafted=drafted)


def _probs(name, dtype, rows, vocab, greedy):
    return dict(name=name, op="probs", dtype=dtype, rows=rows, vocab=vocab, greedy=greedy)


def listed():
    return [
        # Four requests behind one short instruction, on one of four tensor-parallel ranks.  Latency counts.
        _shared("shared, four short", "bf16", 4, 1, 1, 1, 512, 512, 5, 188, 8, 2, 128, 64),
        # A full decode batch behind one long document or system prompt.
        _shared("shared, batch 64", "bf16", 64, 1, 1, 1, 6016, 6016, 85, 2175, 32, 8, 128, 64),
        # Speculative-verify windows of 6 tokens, four different prefixes of four requests each.
        _shared("shared, verify windows", "f16", 16, 4, 6, 6, 1001, 4003, 100, 1000, 32, 8, 128, 32),
        # A key-value head for each query head, short heads, small pages.
        _shared("shared, heads of 64", "f16", 32, 1, 1, 4, 2000, 2000, 100, 2090, 16, 16, 64, 16),
        # The requests' own parts of their prompts, behind a prefix that is cached already: compute-bound.
        _shared("shared, prompts", "bf16", 8, 1, 200, 256, 4096, 4096, 200, 256, 32, 8, 128, 64),
        # The bookkeeping of a verify step of 64 requests, a few of which have ended.
        _plan("plan, verify windows", 64, 8, 0, 0, 3, 6001, 8191, 64),
        # A step that mixes many requests with the prompts of new ones, small pages.
        _plan("plan, prompts among 1000", 1000, 4, 2048, 12, 40, 17, 4099, 16),
        # One request's window of 6 (T = 6 of the verify reads) over a small vocabulary.
        _verify("verify, one request", "f32", 1, 6, 6, 32000, True),
        # A full batch of windows of up to 8 over a large vocabulary, with the draft's probabilities.
        _verify("verify, batch 64", "f32", 64, 2, 8, 131072, True),
        # Drafts without probabilities (looked up in the prompt), 16-bit target probabilities, an odd vocabulary.
        _verify("verify, looked up", "bf16", 16, 1, 17, 100003, False),
        # The rows of a decode batch (M = 16), some of them greedy.
        _probs("probs, decode", "bf16", 16, 32000, 4),
        # The rows of a batch of verify windows over a large vocabulary.
        _probs("probs, verify windows", "bf16", 320, 131072, 20),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "plan", "verify", "verify", "probs"])
    if op == "plan":
        batch = _log(rng, 1, 1000)
        page = rng.choice([16, 32, 64, 128])
        prompts = rng.choice([0, rng.randint(0, min(12, batch))])
        lo = _log(rng, 1, 6000)
        return dict(op=op, batch=batch, n_max=rng.randint(1, 8), prompt_max=_log(rng, 9, 2048) if prompts else 0, prompts=prompts,
                    ended=rng.randint(0, batch // 8), len_min=lo, len_max=min(8191, lo + _log(rng, 1, 4099)), page=page)
    if op == "verify":
        n_max = rng.choice([1, 2, 4, 6, 8, 17])
        batch, vocab = _log(rng, 1, 64), _log(rng, 1000, 131072)
        while batch * n_max * vocab > 64 * 5 * 131072:
            batch = max(1, batch // 2)
        return dict(op=op, dtype=rng.choice(["f32", "f32", "bf16", "f16"]), batch=batch, n_min=rng.choice([1, n_max]), n_max=n_max,
                    vocab=vocab, drafted=rng.random() < 0.7)
    if op == "probs":
        rows, vocab = _log(rng, 1, 320), _log(rng, 1000, 131072)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), rows=rows, vocab=vocab, greedy=rng.randint(0, rows // 2))
    dtype = rng.choice(["bf16", "f16"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    batch = _log(rng, 2, 64)
    groups = rng.choice([1, 1, rng.randint(1, max(1, batch // 2))])
    kind = rng.choice(["token", "token", "window", "prompt"])
    n_max = 1 if kind == "token" else rng.randint(2, 8) if kind == "window" else _log(rng, 9, 256)
    n_min = rng.choice([n_max, max(1, n_max // 2)])
    prefix_max = _log(rng, 64, 16000)
    tail_max = n_max + _log(rng, 1, 2175)
    # No more scores than the listed prompts have, no more cache than the listed batch.
    while batch * n_max * (prefix_max + tail_max) * kv_heads * group * dim > 8 * 230 * 4300 * 32 * 128 or \
            (groups * prefix_max + batch * tail_max) * kv_heads * dim > 64 * 1300 * 8 * 128:
        if batch > 2:
            batch //= 2
            groups = min(groups, max(1, batch // 2))
        elif prefix_max > 128:
            prefix_max //= 2
        else:
            n_max = max(1, n_max // 2)
            n_min, tail_max = min(n_min, n_max), max(n_max, tail_max // 2)
    return dict(op=op, dtype=dtype, batch=batch, groups=groups, n_min=n_min, n_max=n_max,
                prefix_min=rng.choice([prefix_max, max(1, prefix_max // 3)]), prefix_max=prefix_max,
                tail_min=rng.choice([tail_max, max(n_max, tail_max // 5)]), tail_max=tail_max, q_heads=kv_heads * group,
                kv_heads=kv_heads, dim=dim, page=page)


# ------------------------------------------------------------------------------------------- inputs
def _spread(lo, hi, count, salt):
    """`count` whole numbers of [lo, hi], the first one hi: uneven, and the same for every seed."""
    return [hi] + [lo + int(((b + salt) * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for b in range(1, count)]


def _starts(ns):
    return np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _layout(case):
    """Of a shared-prefix case: each sequence's rows, prefix (whole pages) and length, each group's first sequence."""
    B, G, P = case["batch"], case["groups"], case["page"]
    seq0 = [g * B // G for g in range(G + 1)]
    prefix = [-(-x // P) * P for x in _spread(case["prefix_min"], case["prefix_max"], G, 2)]
    ns = _spread(case["n_min"], case["n_max"], B, 3)
    tails = [max(n, t) for n, t in zip(ns, _spread(case["tail_min"], case["tail_max"], B, 0))]
    pre = [prefix[g] for g in range(G) for _ in range(seq0[g], seq0[g + 1])]
    return seq0, prefix, ns, [p + t for p, t in zip(pre, tails)], pre


def _prepare_shared(case, S, randn, gen):
    D, Hq, Hkv, P, B = case["dim"], case["q_heads"], case["kv_heads"], case["page"], case["batch"]
    seq0, prefix, ns, lens, pre = _layout(case)
    M, width = sum(ns), -(-max(lens) // P) + 1
    shared = sum(x // P for x in prefix)
    tails = [-(-l // P) - x // P for l, x in zip(lens, pre)]
    pages = shared + sum(tails) + 3
    ids = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32).cpu().numpy()
    table = np.full((B, width), -1, np.int32)
    at, own_at = 0, shared
    for g, x in enumerate(prefix):
        table[seq0[g]:seq0[g + 1], :x // P] = ids[at:at + x // P]
        at += x // P
    for b, t in enumerate(tails):
        table[b, pre[b] // P:pre[b] // P + t] = ids[own_at:own_at + t]
        own_at += t
    S.update(table=torch.from_numpy(table).cuda(), row0=torch.from_numpy(_starts(ns)).cuda(), kv_len=_i32(lens), seq0=_i32(seq0),
             prefix=_i32(prefix), tokens=M, max_tokens=max(ns), seq0_host=seq0, prefix_host=prefix, tail_max=max(l - x for l, x in zip(lens, pre)),
             max_rows=max(sum(ns[a:b]) for a, b in zip(seq0, seq0[1:])))

    def quants():
        return (randn(pages, Hkv, P, D) * 34).round_().clamp_(-127, 127).add_(128).to(torch.uint8)

    # Pages as appends leave them: the values' scale is the page's largest value over 127, 3 to 4 deviations wide.
    S["kc"], S["vc"] = quants(), quants()
    S["ks"] = 0.026 * torch.exp(0.1 * randn(pages, Hkv))
    S["vs"] = 0.026 * torch.exp(0.1 * randn(pages, Hkv))
    S["q"] = randn(M, (Hq + 2 * Hkv) * D).to(DT[case["dtype"]])[:, :Hq * D].view(M, Hq, D)     # of the fused product's output
    S["scale"] = 1.0 / math.sqrt(D)
    S["out"] = torch.empty(M, Hq, D, device="cuda", dtype=DT[case["dtype"]])
    S["lse"] = torch.empty(M, Hq, device="cuda", dtype=torch.float32)
    if own:
        import int8_weight_gemm_gb300 as lib8
        S["cache"] = lib8.KV8Cache(S["kc"], S["vc"], S["ks"], S["vs"])
        S["step"] = lib8.KV8Step(S["row0"], S["kv_len"], S["table"], M, max(ns))
        S["group"] = lib8.KV8Groups(S["seq0"], S["prefix"], S["max_rows"])
        S["ws"] = lib8.alloc_workspace(lib8.kv8_shared_workspace_bytes(M, case["groups"], Hq, Hkv, D))


def _prepare_plan(case, S, seed):
    rng = np.random.default_rng(seed)
    B, P = case["batch"], case["page"]
    lens = rng.integers(case["len_min"], case["len_max"] + 1, B)
    lens[0] = case["len_max"]
    ns = np.minimum(rng.integers(1, case["n_max"] + 1, B), lens)           # the last step's windows
    take = rng.integers(1, ns + 1)                                          # what the verification kept of them
    grow = rng.integers(1, case["n_max"] + 1, B)
    order = rng.permutation(B)
    grow[order[:case["prompts"]]] = rng.integers(max(1, case["prompt_max"] // 2), case["prompt_max"] + 1, case["prompts"]) if case["prompts"] else 0
    take[order[B - case["ended"]:]] = -1
    held = -(-lens // P) + rng.integers(0, 2, B)                            # some sequences hold a page ahead
    pinned = np.minimum(held, rng.integers(0, 3, B))                        # pages of a shared prefix
    longest = case["len_max"] + max(case["n_max"], case["prompt_max"])
    width = longest // P + 2
    used = int(held.sum())
    pages = B * (-(-case["len_max"] // P) + 2) + B * (case["n_max"] // P + 1) + case["prompts"] * (case["prompt_max"] // P + 1)
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    mask = np.arange(width)[None] < held[:, None]
    table[mask] = ids[:used]
    head, free = int(rng.integers(0, pages)), pages - used
    ring = np.full(pages, -1, np.int32)
    ring[(head + np.arange(free)) % pages] = ids[used:]
    rows = B * case["n_max"] + case["prompts"] * case["prompt_max"]          # the step's buffers hold as many
    S.update(row0=_i32(_starts(ns)), kv_len=_i32(lens), table=torch.from_numpy(table).cuda(), held=_i32(held), pinned=_i32(pinned),
             take=_i32(take), grow=_i32(grow), ring=torch.from_numpy(ring).cuda(), pool=_i32([head, free]), rows=rows)
    out = dict(row0=torch.zeros(B + 1, dtype=torch.int32, device="cuda"), pool=torch.zeros(2, dtype=torch.int32, device="cuda"))
    for k in ("kv_len", "held", "granted"):
        out[k] = torch.zeros(B, dtype=torch.int32, device="cuda")
    for k in ("positions", "slots", "seq_of"):
        out[k] = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    S["next"] = out
    if own:
        import int8_weight_gemm_gb300 as lib8
        n = max(1, int(ns.max()), int(grow.max()))
        S["step"] = lib8.KV8Step(S["row0"], S["kv_len"], S["table"], rows, n)
        S["pages"] = lib8.KV8Pool(S["ring"], S["pool"])
        S["ws"] = lib8.alloc_workspace(256)


def _prepare_verify(case, S, gen):
    B, V, dt = case["batch"], case["vocab"], DT[case["dtype"]]
    ns = _spread(case["n_min"], case["n_max"], B, 1)
    R = sum(ns)
    logits = torch.randn(R, V, device="cuda", generator=gen).mul_(3.0)
    p = torch.softmax(logits, -1)
    logits.add_(torch.randn(R, V, device="cuda", generator=gen), alpha=0.7)   # the draft's: near the target's
    q = torch.softmax(logits, -1)
    # Tokens drawn from the draft (row r's is the next row's token): the largest of the logits with Gumbel noise.
    noise = torch.rand(R, V, device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7).log_().neg_().log_()
    drawn = logits.sub_(noise).argmax(-1)
    tokens = torch.roll(drawn, 1).to(torch.int32)
    S.update(p=p.to(dt), q=q.to(dt) if case["drafted"] else None, tokens=tokens, row0=torch.from_numpy(_starts(ns)).cuda(), rows=R,
             accept=torch.rand(R, device="cuda", generator=gen), sample=torch.rand(R, device="cuda", generator=gen),
             next=torch.full((R,), -1, dtype=torch.int32, device="cuda"), take=torch.zeros(B, dtype=torch.int32, device="cuda"))
    if own:
        import int8_weight_gemm_gb300 as lib8
        S["ws"] = lib8.alloc_workspace(lib8.spec_workspace_bytes(B, V))


def _prepare_probs(case, S, randn, gen):
    R, V = case["rows"], case["vocab"]
    S["logits"] = randn(R, V).mul_(3.0).to(DT[case["dtype"]])
    inv = 1.0 / (0.6 + 0.6 * torch.rand(R, device="cuda", generator=gen))
    inv[torch.randperm(R, device="cuda", generator=gen)[:case["greedy"]]] = math.inf     # temperature 0
    S["inv_temp"] = inv
    S["out"] = torch.empty(R, V, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    S = dict(case)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    if case["op"] == "shared":
        _prepare_shared(case, S, randn, gen)
    elif case["op"] == "plan":
        _prepare_plan(case, S, seed)
    elif case["op"] == "verify":
        _prepare_verify(case, S, gen)
    else:
        _prepare_probs(case, S, randn, gen)
    return S


# ------------------------------------------------------------------------------------------- one pass
def run(S):
    op = S["op"]
    if own:
        import int8_weight_gemm_gb300 as lib8
        if op == "shared":
            out = lib8.kv8_attention_shared(S["cache"], S["step"], S["group"], S["q"], S["ws"], out=S["out"], lse=S["lse"], scale=S["scale"])
            return {"out": out, "lse": S["lse"]}
        if op == "plan":
            n = S["next"]
            lib8.kv8_plan(S["step"], S["page"], S["pages"], S["held"], S["take"], S["grow"], S["ws"], pinned=S["pinned"],
                          row0_out=n["row0"], kv_len_out=n["kv_len"], held_out=n["held"], pool_out=n["pool"], granted=n["granted"],
                          positions=n["positions"], slots=n["slots"], seq_of=n["seq_of"])
            return {**n, "table": S["table"], "ring": S["ring"]}
        if op == "verify":
            nxt, take = lib8.spec_verify(S["p"], S["tokens"], S["row0"], S["accept"], S["sample"], S["ws"], q=S["q"], next=S["next"],
                                         take=S["take"])
            return {"next": nxt, "take": take}
        return lib8.spec_probs(S["logits"], S["inv_temp"], out=S["out"])
    return {"shared": _plain_shared, "plan": _plain_plan, "verify": _plain_verify, "probs": _plain_probs}[op](S)


def _part(q, k, v, scale, seen):
    """Scores' maximum, sum of exponentials and weighted values of rows q [..., rows, D] over k, v [..., tokens, D]."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    if seen is not None:
        s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    s = s.sub_(top).exp_()
    return top, s.sum(-1, keepdim=True), torch.matmul(s, v)


def _plain_shared(S):
    B, n, D, Hq, Hkv, P, T = S["batch"], S["max_tokens"], S["dim"], S["q_heads"], S["kv_heads"], S["page"], S["tail_max"]
    G, M = Hq // Hkv, S["tokens"]
    row0, table = S["row0"].long(), S["table"].long()
    dev = row0.device

    def values(cache, scales, pages, at):     # tokens `at` of pages of the same shape -> [..., Hkv, tokens, D]
        x = (cache[pages, :, at].float() - 128.0) * scales[pages][..., None]
        return x.movedim(-2, -3)

    # The prefix of each group once, for all of its rows.
    top, total, acc = (torch.empty(M, Hkv, G, w, device=dev) for w in (1, 1, D))
    q32 = S["q"].float().view(M, Hkv, G, D)
    first = S["seq0_host"]
    for g, length in enumerate(S["prefix_host"]):
        a, b = row0[first[g]], row0[first[g + 1]]
        rows = torch.arange(M, device=dev)
        mine = (rows >= a) & (rows < b)
        j = torch.arange(length, device=dev)
        pages = table[first[g]][j // P]
        k, v = (values(c, s, pages, j % P) for c, s in ((S["kc"], S["ks"]), (S["vc"], S["vs"])))     # [Hkv, tokens, D]
        got = _part(q32[mine].permute(1, 0, 2, 3).reshape(Hkv, -1, D), k, v, S["scale"], None)
        for whole, part in zip((top, total, acc), got):
            whole[mine] = part.view(Hkv, -1, G, part.shape[-1]).transpose(0, 1)
    # Each sequence's own tokens, padded to the longest.
    count = row0[1:] - row0[:-1]
    group = torch.searchsorted(S["seq0"][1:].contiguous(), torch.arange(B, device=dev, dtype=torch.int32), right=True)
    pre = S["prefix"].long()[group]
    own_len = S["kv_len"].long() - pre
    j = torch.arange(T, device=dev)[None].expand(B, T)
    slot = (pre[:, None] + torch.minimum(j, own_len[:, None] - 1))
    pages = table.gather(1, slot // P)
    k, v = (values(c, s, pages, slot % P) for c, s in ((S["kc"], S["ks"]), (S["vc"], S["vs"])))         # [B, Hkv, T, D]
    i = torch.arange(n, device=dev)
    at = (row0[:-1, None] + i).clamp(max=M - 1)
    q = q32[at].permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    seen = j[:, None] <= (own_len - count)[:, None, None] + i[None, :, None]                            # [B, n, T]
    seen = seen[:, None, :, None].expand(B, 1, n, G, T).reshape(B, 1, n * G, T)
    live = i[None] < count[:, None]
    own_top, own_total, own_acc = (x.view(B, Hkv, n, G, -1).transpose(1, 2)[live] for x in _part(q, k, v, S["scale"], seen))
    m = torch.maximum(top, own_top)
    a, b = torch.exp(top - m), torch.exp(own_top - m)
    total = total * a + own_total * b
    out = (acc * a + own_acc * b) / total
    return {"out": out.reshape(M, Hq, D).to(S["q"].dtype), "lse": (m + torch.log(total)).reshape(M, Hq)}


def _plain_plan(S):
    """The next step, all in whole numbers.  A sequence keeps `take` of its last step's rows (-1: it has ended, and its own
    pages go to the end of the ring of free pages), gets `grow` rows, and pages for them from the ring's head, in order;
    from the first sequence on that does not fit, none gets rows."""
    P, R = S["page"], S["rows"]
    dev = S["row0"].device
    row0, kv_len, held, pinned = (S[k].long() for k in ("row0", "kv_len", "held", "pinned"))
    take, grow, ring, table = S["take"].long(), S["grow"].long(), S["ring"], S["table"]
    cap, (head, free) = ring.numel(), S["pool"].long()
    ended = take < 0
    kept = torch.where(ended, 0, kv_len - (row0[1:] - row0[:-1]) + take)
    want = torch.where(ended, 0, grow)
    need = torch.where(want > 0, ((kept + want + P - 1) // P - held).clamp(min=0), 0)
    fits = (torch.cumsum(need, 0) <= free) & (torch.cumsum(want, 0) <= R)
    fits = torch.cumprod(fits.to(torch.int64), 0)
    rows, need = want * fits, need * fits
    first = torch.cumsum(need, 0) - need
    width = torch.arange(table.shape[1], device=dev)[None]
    # Pages go back ...
    back = torch.where(ended, (held - pinned).clamp(min=0), 0)
    gone = ended[:, None] & (width >= pinned[:, None]) & (width < held[:, None])
    ids = table[gone]
    ring[(head + free + torch.arange(ids.numel(), device=dev)) % cap] = ids
    # ... and new ones come.
    fresh = (width >= held[:, None]) & (width < (held + need)[:, None])
    at = (head + first[:, None] + width - held[:, None]) % cap
    table[fresh] = ring[at[fresh]]
    out = S["next"]
    new_len = kept + rows
    ends = torch.cumsum(rows, 0)
    out["row0"].copy_(torch.cat([torch.zeros_like(ends[:1]), ends]))
    out["kv_len"].copy_(new_len)
    out["held"].copy_(torch.where(ended, 0, held + need))
    out["granted"].copy_(rows)
    used = need.sum()
    out["pool"].copy_(torch.stack([(head + used) % cap, free - used + back.sum()]))
    # Each row's sequence, position and slot; rows behind the last sequence stay as they were.
    r = torch.arange(R, device=dev)
    seq = torch.searchsorted(ends, r, right=True)
    live = seq < ends.numel()
    seq = seq.clamp(max=ends.numel() - 1)
    pos = new_len[seq] - ends[seq] + r
    slot = table[seq, (pos // P).clamp(0, table.shape[1] - 1)].long() * P + pos % P
    for k, v in (("positions", pos), ("slots", slot), ("seq_of", seq)):
        out[k].copy_(torch.where(live, v.to(torch.int32), out[k]))
    return {**out, "table": table, "ring": ring}


def _plain_verify(S):
    """Row r of a window holds the target's probabilities after token r; the token of the next row is accepted where
    accept * q < p.  The first row whose successor is not (or the last row) draws the token after it: from p - q where
    that is positive (without q: from p without the rejected token), the last row from p."""
    p, q, row0, R = S["p"], S["q"], S["row0"].long(), S["rows"]
    V, dev = p.shape[1], p.device
    r = torch.arange(R, device=dev)
    seq = torch.searchsorted(row0[1:].contiguous(), r, right=True)
    last = r + 1 == row0[seq + 1]
    t = torch.where(last, 0, S["tokens"].long().roll(-1))
    pt = p[r, t].double()
    qt = q[r, t].double() if q is not None else torch.ones_like(pt)
    stop = last | ~(S["accept"].double() * qt < pt)
    at = torch.full_like(row0[1:], R).scatter_reduce(0, seq[stop], r[stop], "amin")     # the row that draws
    w = p[at].double()
    drawn = ~last[at]
    if q is not None:
        left = (w - q[at].double()).clamp(min=0)
    else:
        left = w.scatter(1, t[at, None], 0.0)
    left = torch.where((drawn & (left.sum(-1) > 0))[:, None], left, w)
    cum = left.cumsum(-1)
    token = (cum <= S["sample"].double()[at, None] * cum[:, -1:]).sum(-1).clamp(max=V - 1)
    out = torch.where(r < at[seq], S["tokens"].long().roll(-1), -1)
    out[at] = token
    S["next"].copy_(out)
    S["take"].copy_(at - row0[:-1] + 1)
    return {"next": S["next"], "take": S["take"]}


def _plain_probs(S):
    x, inv = S["logits"].float(), S["inv_temp"][:, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) * torch.where(torch.isinf(inv), 1.0, inv))
    V = x.shape[1]
    i = torch.arange(V, device=x.device)
    best = torch.where(x == top, i, V).amin(-1, keepdim=True)
    return torch.where(torch.isinf(inv), (i == best).float(), e / e.sum(-1, keepdim=True))


# ------------------------------------------------------------------------------------------- what a pass costs
def work(case):
    if case["op"] == "shared":
        D, Hq, Hkv, P = case["dim"], case["q_heads"], case["kv_heads"], case["page"]
        seq0, prefix, ns, lens, pre = _layout(case)
        held = sum(prefix) + sum(l - x for l, x in zip(lens, pre))
        pages = held // P + len(lens)
        seen = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(ns, lens))
        return {"bytes": 2 * Hkv * D * held + (8 * Hkv + 4) * pages + sum(ns) * Hq * (4 * D + 4), "flops": 4 * D * Hq * seen}
    if case["op"] == "plan":
        B = case["batch"]
        rows = B * (1 + case["n_max"]) // 2 + case["prompts"] * case["prompt_max"] * 3 // 4
        return {"bytes": 4 * (6 * B + 4 * B + 3 * rows + 2 * (rows // case["page"])), "flops": 0}
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "f32" else 2
        # The row that draws, of the draft's too where a window can be rejected.
        sides = 2 if case["drafted"] and case["n_max"] > 1 else 1
        return {"bytes": case["batch"] * (case["vocab"] * size * sides + case["n_max"] * 24), "flops": case["batch"] * case["vocab"] * 2}
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": case["rows"] * case["vocab"] * (size + 4), "flops": 4 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    S = prepare(case, seed)
    return {"shared": _exact_shared, "plan": _exact_plan, "verify": _exact_verify, "probs": _exact_probs}[case["op"]](case, S)


def _exact_shared(case, S):
    D, Hq, Hkv, P = case["dim"], case["q_heads"], case["kv_heads"], case["page"]
    G = Hq // Hkv
    seq0, prefix, ns, lens, pre = _layout(case)
    if sum(2 * D * Hq * n * l for n, l in zip(ns, lens)) > 2.5e12:
        return None
    starts = _starts(ns)
    outs, lses = [], []
    for b, (n, l) in enumerate(zip(ns, lens)):
        pages = S["table"][b, :-(-l // P)].long()
        r = int(starts[b])
        hidden = torch.arange(l, device="cuda")[None] > torch.arange(l - n, l, device="cuda")[:, None]
        o = torch.empty(n, Hq, D, device="cuda", dtype=torch.float64)
        z = torch.empty(n, Hq, device="cuda", dtype=torch.float64)
        for h in range(Hkv):
            k, v = (((c[pages, h].double() - 128.0) * s[pages, h].double()[:, None, None]).reshape(-1, D)[:l]
                    for c, s in ((S["kc"], S["ks"]), (S["vc"], S["vs"])))
            x = torch.einsum("ngd,td->gnt", S["q"][r:r + n, h * G:(h + 1) * G].double(), k) * S["scale"]
            x = x.masked_fill(hidden[None], -math.inf)
            z[:, h * G:(h + 1) * G] = torch.logsumexp(x, -1).T
            o[:, h * G:(h + 1) * G] = torch.einsum("gnt,td->ngd", torch.softmax(x, -1), v)
        outs.append(o)
        lses.append(z)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_plan(case, S):
    """One sequence after the other, on the host."""
    P, R = case["page"], S["rows"]
    get = lambda k: S[k].cpu().tolist()   # noqa: E731
    row0, kv_len, held, pinned, take, grow, ring, table = (get(k) for k in ("row0", "kv_len", "held", "pinned", "take", "grow", "ring", "table"))
    head, free = get("pool")
    cap = len(ring)
    queue = [ring[(head + i) % cap] for i in range(free)]
    back, full, rows = [], False, 0
    new = {k: [] for k in ("row0", "kv_len", "held", "granted", "positions", "slots", "seq_of")}
    new["row0"].append(0)
    used = 0
    for b in range(len(kv_len)):
        if take[b] < 0:
            back += table[b][pinned[b]:held[b]]
            kept, count, pages = 0, 0, 0
        else:
            kept, count, pages = kv_len[b] - (row0[b + 1] - row0[b]) + take[b], grow[b], held[b]
            need = max(0, -(-(kept + count) // P) - pages) if count else 0
            full = full or used + need > free or rows + count > R
            if full:
                count = need = 0
            for _ in range(need):
                table[b][pages] = queue[used]
                pages, used = pages + 1, used + 1
        for t in range(kept, kept + count):
            new["positions"].append(t)
            new["slots"].append(table[b][t // P] * P + t % P)
            new["seq_of"].append(b)
        rows += count
        for k, v in (("row0", rows), ("kv_len", kept + count), ("held", pages), ("granted", count)):
            new[k].append(v)
    for i, x in enumerate(back):
        ring[(head + free + i) % cap] = x
    for k in ("positions", "slots", "seq_of"):
        new[k] += [-1] * (R - rows)
    new["pool"] = [(head + used) % cap, free - used + len(back)]
    order = ("row0", "pool", "kv_len", "held", "granted", "positions", "slots", "seq_of")
    return {**{k: _i32(new[k]) for k in order}, "table": _i32(table), "ring": _i32(ring)}


def _exact_verify(case, S):
    """One request after the other."""
    row0, tokens = S["row0"].tolist(), S["tokens"].tolist()
    accept, sample = S["accept"].double().tolist(), S["sample"].double().tolist()
    out, take = [-1] * S["rows"], []
    for a, b in zip(row0, row0[1:]):
        r = a
        while r + 1 < b:
            t = tokens[r + 1]
            if not accept[r] * (float(S["q"][r, t]) if S["q"] is not None else 1.0) < float(S["p"][r, t]):
                break
            out[r] = t
            r += 1
        w = S["p"][r].double()
        if r + 1 < b:
            left = w.clone()
            if S["q"] is not None:
                left = torch.relu(left - S["q"][r].double())
            else:
                left[tokens[r + 1]] = 0.0
            if float(left.sum()) > 0:
                w = left
        cum = torch.cumsum(w, 0)
        out[r] = int(torch.searchsorted(cum, sample[r] * cum[-1], right=True))
        take.append(r - a + 1)
    return {"next": _i32(out), "take": _i32(take)}


def _exact_probs(case, S):
    out = torch.empty(case["rows"], case["vocab"], device="cuda", dtype=torch.float64)
    for r in range(case["rows"]):
        x, inv = S["logits"][r].double(), float(S["inv_temp"][r])
        if math.isinf(inv):
            out[r] = 0.0
            out[r, int(torch.nonzero(x == x.max())[0, 0])] = 1.0
        else:
            out[r] = torch.softmax(x * inv, 0)
    return out
