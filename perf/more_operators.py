"""Operators of a decode step around the 4-bit K/V cache and the experts as measured calls: K/V append with the
position rotation on the way, attention with capped or biased scores and with prefix and document masks, routing
by softmax or sigmoid scores with groups and a balancing bias.

`run` computes them in elementary torch operations where `own` is false, and through dequant_gemv_moe_gb300 where
it is true.  Both work on the same packed cache, whose layout is:

  cache[page][kv head][page_size / 16] blocks of 16 tokens, 18 * D bytes each (D = head_dim, G = D / 32
  groups of 32 values along D, W = min(G, 4)):
    K codes   [G / W][16 tokens][4 t][W groups] words of 32 bits: values 8t .. 8t+7 of the group, value e
              in nibble (e >> 1) + 4 * (e & 1)
    V codes   [2 j][G / W][8 a][4 t][2 i][W groups] 16 bits: token 8j + 2t + i, values 4a .. 4a+3 of the
              group, value n in nibble n
    K scales  [16 tokens][G] fp16
    V scales  [4 t][G][2 j][2 i] fp16: token 8j + 2t + i
  value = scale * (code - 8): the Q4_0 block, its 32 values along head_dim.
"""
import math
import random

import torch

own = False

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # the logits of one decode step of a small batch over 256 experts in 8 groups, sigmoid scores with a
        # balancing bias (latency)
        dict(name="route_step", op="route", tokens=8, experts=256, k=8, scores="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, dtype="fp32", ragged=1),
        # the same layer's prompt tokens: memory bound
        dict(name="route_prompt", op="route", tokens=16384, experts=256, k=8, scores="sigmoid", bias=True, groups=8,
             top_groups=4, group_score="top2", renorm=True, scale=2.5, dtype="fp32", ragged=2),
        # softmax scores limited to the groups with the best expert, gates as they are, 16-bit logits (equal ones
        # among them), odd sizes
        dict(name="route_soft", op="route", tokens=4095, experts=160, k=6, scores="softmax", bias=False, groups=8,
             top_groups=3, group_score="max", renorm=False, scale=16.0, dtype="bf16", ragged=3),
        # the rows of one decode step of 64 requests far into their contexts (Llama-3-8B heads)
        dict(name="rope_step", op="rope", tokens=64, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             base=500000.0, far=131072, run=1, dtype="bf16", page=16, skip=0, ragged=4),
        # a long prompt's rows, one token short of a round number: memory bound
        dict(name="rope_prompt", op="rope", tokens=8191, heads=32, kv_heads=8, dim=128, rot=128, interleaved=False,
             base=500000.0, far=16384, run=8191, dtype="bf16", page=64, skip=0, ragged=5),
        # fp32 rows as the quantized GEMV writes them, odd head counts, half of each head rotated in neighbouring
        # pairs, chunks of several requests, some tokens without a place in the cache
        dict(name="rope_odd", op="rope", tokens=1023, heads=15, kv_heads=5, dim=64, rot=32, interleaved=True,
             base=10000.0, far=1000000, run=100, dtype="fp32", page=32, skip=5, ragged=6),
        # one request's decode step over a short context with a distance bias: the smallest call (latency)
        dict(name="bias_step_1", op="attn", batch=1, mode="step", max_q=1, max_ctx=977, heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=16, window=0, cap=0.0, bias=True, mask="", ragged=7),
        # a serving batch's decode step with capped scores, ragged contexts (Llama-3-8B heads): memory bound
        dict(name="cap_step_64", op="attn", batch=64, mode="step", max_q=1, max_ctx=16384, heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=16, window=0, cap=50.0, bias=False, mask="", ragged=8),
        # decode with capped scores, a sliding window and wide heads
        dict(name="cap_window", op="attn", batch=16, mode="step", max_q=1, max_ctx=8192, heads=8, kv_heads=4,
             dim=256, dtype="fp16", page=128, window=1024, cap=50.0, bias=False, mask="", ragged=9),
        # verification of a few drafted tokens per request with a distance bias, seven query heads to a KV head
        dict(name="bias_verify", op="attn", batch=20, mode="few", max_q=6, max_ctx=6000, heads=28, kv_heads=4,
             dim=128, dtype="fp16", page=32, window=0, cap=0.0, bias=True, mask="", ragged=10),
        # a chunk of a long prompt over what the cache holds, capped scores: compute bound, the largest call
        dict(name="cap_chunk", op="attn", batch=2, mode="chunk", max_q=2048, max_ctx=16384, heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=64, window=0, cap=30.0, bias=False, mask="", ragged=11),
        # fresh prompts of several documents each, whose first part is read both ways; one query head per KV
        # head, one request without new tokens
        dict(name="docs_prompts", op="attn", batch=7, mode="prompt", max_q=3001, max_ctx=0, heads=12, kv_heads=12,
             dim=64, dtype="fp16", page=16, window=0, cap=0.0, bias=False, mask="both", ragged=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "rope", "attn", "attn", "attn"])
    ragged = rng.randrange(1 << 20)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.randint(max(2, 16 // groups), 256 // groups)
        top = rng.randint(max(1, groups // 4), groups)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=rng.randint(1, min(8, top * experts // groups)),
                    scores=rng.choice(["sigmoid", "softmax"]), bias=rng.choice([True, False]), groups=groups,
                    top_groups=top, group_score=rng.choice(["top2", "max"]), renorm=rng.choice([True, True, False]),
                    scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    ragged=ragged)
    page = rng.choice([16, 32, 64, 128])
    kv_heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "rope":
        dim, tokens = rng.choice([64, 128, 128, 256]), _log(rng, 1, 8191)
        while tokens * kv_heads * (group + 2) * dim > 8191 * 48 * 128:
            tokens = tokens // 2
        return dict(op=op, tokens=tokens, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2, 32]), interleaved=rng.choice([True, False]),
                    base=rng.choice([10000.0, 500000.0]), far=_log(rng, 100, 1000000),
                    run=rng.choice([1, _log(rng, 1, 8191)]), dtype=rng.choice(["bf16", "fp16", "fp32"]), page=page,
                    skip=rng.choice([0, 0, 5]), ragged=ragged)
    dim, dtype = rng.choice([64, 128, 128, 256]), rng.choice(["fp16", "bf16"])
    mode = rng.choice(["step", "step", "few", "chunk", "prompt"])
    c = dict(op=op, batch=0, mode=mode, max_q=1, max_ctx=0, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
             dtype=dtype, page=page, window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]),
             cap=rng.choice([0.0, 30.0, 50.0]), bias=rng.choice([True, False]), mask="", ragged=ragged)
    if mode in ("step", "few"):
        c["max_q"] = 1 if mode == "step" else rng.randint(2, 8)
        c["max_ctx"] = _log(rng, 1, 131072)
        most = 2 * 131072 * 8 * 128 // (c["max_ctx"] * kv_heads * dim)
        c["batch"] = _log(rng, 1, max(1, min(128, most)))
    else:
        c["max_q"] = _log(rng, 16, 3001)
        c["max_ctx"] = 0 if mode == "prompt" else _log(rng, 16, 16384)
        rows = c["max_q"] * (c["max_q"] + c["max_ctx"]) * kv_heads * group * dim
        most = 2 * 2048 * (2048 + 16384) * 32 * 128 // rows
        c["batch"] = _log(rng, 1, max(1, min(16, most)))
        c["mask"] = rng.choice(["", "docs", "prefix", "both"])
    if not (c["cap"] or c["bias"] or c["mask"]):
        c["cap"] = 50.0
    return c


# ------------------------------------------------------------------------------------------------
# lengths: fixed by the case, so that the work of a pass is known
# ------------------------------------------------------------------------------------------------
def _lengths(case):
    """(tokens in the cache before, new tokens) of each request."""
    r = random.Random(case["ragged"])
    ctx, new = [], []
    for i in range(case["batch"]):
        c = r.randint(1, max(1, case["max_ctx"]))
        if case["mode"] == "step":                    # the first request: the length itself; else from short to full
            n = 1
            c = case["max_ctx"] if case["batch"] == 1 or i == 0 else c
        elif case["mode"] == "few":
            n = r.randint(1, case["max_q"])
        elif case["mode"] == "chunk":
            c, n = case["max_ctx"], case["max_q"]
        else:                                         # whole prompts, one request without new tokens
            c, n = 0, case["max_q"] if i == 0 else 0 if i == 1 else r.randint(1, case["max_q"])
        ctx.append(c)
        new.append(n)
    return ctx, new


def _spans(case):
    """(new tokens, cache lengths, every row's first position or None, every request's prefix or None)."""
    ctx, new = _lengths(case)
    r = random.Random(case["ragged"] + 1)
    first = prefix = None
    if case["mask"] in ("docs", "both"):
        first = []
        for c, n in zip(ctx, new):
            at, left = 0, 0                           # what the cache holds belongs to the first document
            for i in range(n):
                if left == 0:
                    at, left = (c + i if i else 0), r.randint(1, max(1, min(n, 1200)))
                first.append(at)
                left -= 1
    if case["mask"] in ("prefix", "both"):
        prefix = [r.choice([0, r.randint(0, (c + n) // 2)]) if i else (c + n) // 3
                  for i, (c, n) in enumerate(zip(ctx, new))]
    return new, [c + n for c, n in zip(ctx, new)], first, prefix


def _slopes(heads):
    return [2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]


# ------------------------------------------------------------------------------------------------
# packed blocks in elementary operations
# ------------------------------------------------------------------------------------------------
def _nibble_of(device):
    return torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=device)      # value e of a K word -> its nibble


def _quantise(x):
    """x [..., D] -> codes [..., D] (0..15) and fp16 scales [..., D / 32], in x's own bits."""
    x = x.clamp(-65504.0, 65504.0)
    g = x.reshape(*x.shape[:-1], -1, 32)
    a = g.abs()
    at = torch.arange(32, device=x.device)
    first = torch.where(a == a.amax(-1, keepdim=True), at, torch.full_like(at, 32)).amin(-1, keepdim=True)
    d = (g.gather(-1, first) * -0.125).to(torch.float16)
    df = d.to(x.dtype)
    c = torch.floor(g / torch.where(df == 0, torch.ones_like(df), df) + 8.5).clamp(0, 15)
    c = torch.where(df == 0, torch.full_like(c, 8.0), c)
    return c.to(torch.uint8).reshape(x.shape), d.squeeze(-1)


def _values(codes, d):
    g = codes.reshape(*codes.shape[:-1], -1, 32).float() - 8.0
    return (d.float().unsqueeze(-1) * g).reshape(codes.shape)


def _bytes_of(nib):
    """nibbles [..., 2n] -> bytes [..., n], the even one low."""
    n = nib.reshape(*nib.shape[:-1], -1, 2)
    return n[..., 0] | (n[..., 1] << 4)


def _pack(kc, kd, vc, vd):
    """codes [N, 16, D] and scales [N, 16, G] of K and V -> blocks [N, 18 D] (bytes)."""
    n, _, dim = kc.shape
    g = dim // 32
    w = min(g, 4)
    inv = torch.argsort(_nibble_of(kc.device))
    k = kc.reshape(n, 16, g // w, w, 4, 8)[..., inv].permute(0, 2, 1, 4, 3, 5)
    v = vc.reshape(n, 2, 4, 2, g // w, w, 8, 4).permute(0, 1, 4, 6, 2, 3, 5, 7)
    vs = vd.reshape(n, 2, 4, 2, g).permute(0, 2, 4, 1, 3).contiguous()
    return torch.cat([_bytes_of(k).reshape(n, 8 * dim), _bytes_of(v).reshape(n, 8 * dim),
                      kd.contiguous().view(torch.uint8).reshape(n, dim), vs.view(torch.uint8).reshape(n, dim)], 1)


def _nibbles(b):
    return torch.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)


def _unpack(blocks, dim):
    """blocks [..., 18 D] -> K and V values [..., 16, D] in 32 bits."""
    lead = blocks.shape[:-1]
    b = blocks.reshape(-1, 18 * dim)
    n, g = b.shape[0], dim // 32
    w = min(g, 4)
    kn = _nibbles(b[:, :8 * dim].reshape(n, g // w, 16, 4, w, 4))[..., _nibble_of(b.device)]
    kn = kn.permute(0, 2, 1, 4, 3, 5).reshape(n, 16, g, 32)
    vn = _nibbles(b[:, 8 * dim:16 * dim].reshape(n, 2, g // w, 8, 4, 2, w, 2))
    vn = vn.permute(0, 1, 4, 5, 2, 6, 3, 7).reshape(n, 16, g, 32)
    kd = b[:, 16 * dim:17 * dim].contiguous().view(torch.float16).reshape(n, 16, g, 1)
    vd = b[:, 17 * dim:].contiguous().view(torch.float16).reshape(n, 4, g, 2, 2).permute(0, 3, 1, 4, 2)
    k = kd.float() * (kn.float() - 8.0)
    v = vd.reshape(n, 16, g, 1).float() * (vn.float() - 8.0)
    return k.reshape(*lead, 16, dim), v.reshape(*lead, 16, dim)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _rows(g, shape, spread=None):
    x = torch.randn(shape, generator=g, device="cuda")
    return x if spread is None else x * spread


def _fill(cache, g, rows, dim):
    """Writes random K/V into every block of cache [pages, heads, nb, 18 D]; tokens past a page's first
    `rows[page]` keep scales that are NaN, as memory that nobody wrote may hold."""
    pages, heads, nb, _ = cache.shape
    spread = 1.0 + 3.0 * (torch.rand(heads, 1, 1, dim, generator=g, device="cuda") > 0.95)
    size = torch.tensor([0.5], device="cuda")
    at = torch.arange(nb * 16, device="cuda").reshape(1, 1, nb, 16, 1)
    step = max(1, (1 << 26) // (heads * nb * 16 * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        live = at < rows[p:p + n].reshape(n, 1, 1, 1, 1)
        parts = []
        for f in (spread.reshape(1, heads, 1, 1, dim), size):
            c, d = _quantise(_rows(g, (n, heads, nb, 16, dim)) * f)
            d = torch.where(live, d, torch.full_like(d, float("nan")))
            parts += [c.reshape(-1, 16, dim), d.reshape(-1, 16, dim // 32)]
        cache[p:p + n] = _pack(*parts).reshape(n, heads, nb, 18 * dim)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _positions(case):
    """Tokens of several requests, `run` consecutive positions each, from anywhere up to `far`."""
    r = random.Random(case["ragged"])
    t, pos = case["tokens"], []
    while len(pos) < t:
        n = min(t - len(pos), case["run"])
        at = 0 if case["run"] >= t else r.randint(0, case["far"])
        pos += range(at, at + n)
    return pos


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + case["ragged"])
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        # experts differ in how often they are wanted, which the bias evens out
        want = _rows(g, (e,), 0.5)
        logits = (_rows(g, (t, e), 1.2) + want).to(DT[case["dtype"]])
        return dict(case=case, logits=logits, bias=(want * -0.1).contiguous() if case["bias"] else None,
                    out=(torch.empty((t, case["k"]), dtype=torch.int32, device="cuda"),
                         torch.empty((t, case["k"]), dtype=torch.float32, device="cuda")))
    dim, hk, h, ps = case["dim"], case["kv_heads"], case["heads"], case["page"]
    if case["op"] == "rope":
        t = case["tokens"]
        n_pages = -(-t // ps) + 5
        cache = torch.full((n_pages, hk, ps // 16, 18 * dim), 255, dtype=torch.uint8, device="cuda")
        order = torch.randperm(n_pages, generator=g, device="cuda")
        at = torch.arange(3, t + 3, device="cuda")
        slots = order[at // ps] * ps + at % ps
        if case["skip"]:
            r = random.Random(case["ragged"] + 1)
            out = [i for i in range(t) if r.randrange(100) < case["skip"]]
            slots[torch.tensor(out, dtype=torch.int64, device="cuda")] = -1
        spread = 1.0 + 3.0 * (torch.rand(1, 1, dim, generator=g, device="cuda") > 0.95)
        # q, k and v are slices of one projection's rows
        qkv = torch.cat([_rows(g, (t, h, dim), 1.5), _rows(g, (t, hk, dim)) * spread, _rows(g, (t, hk, dim), 0.5)], 1)
        qkv = qkv.to(DT[case["dtype"]])
        q, k, v = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        freq = (case["base"] ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])).float().cuda()
        return dict(case=case, cache=cache, q=q, k=k, v=v, slots=slots, pos=_i32(_positions(case)), freq=freq, page=ps,
                    out=torch.empty((t, h, dim), dtype=q.dtype, device="cuda"),
                    kv=tuple(torch.empty((t, hk, dim), dtype=q.dtype, device="cuda") for _ in range(2)))
    new, kv, first, prefix = _spans(case)
    have = [-(-n // ps) for n in kv]
    n_pages = sum(have) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], max(have) + 1), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(have)), torch.tensor(have)).cuda()
    col = torch.cat([torch.arange(n) for n in have]).cuda()
    used = order[:sum(have)]
    table[row, col] = used
    rows = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    rows[used.long()] = (torch.tensor(kv).cuda()[row] - col * ps).clamp(max=ps)
    cache = torch.empty((n_pages, hk, ps // 16, 18 * dim), dtype=torch.uint8, device="cuda")
    _fill(cache, g, rows, dim)
    t = sum(new)
    # (capped scores reach up to where the cap bends them)
    q = _rows(g, (t, h, dim), 6.0 if case["cap"] else 1.5).to(DT[case["dtype"]])
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return dict(case=case, cache=cache, q=q, start=_i32(start), kv=_i32(kv), table=table, page=ps, max_q=max(new),
                max_kv=max(kv), slopes=torch.tensor(_slopes(h), device="cuda") if case["bias"] else None,
                first=None if first is None else _i32(first), prefix=None if prefix is None else _i32(prefix),
                out=torch.empty_like(q), lse=torch.empty((t, h), dtype=torch.float32, device="cuda"))


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _route_plain(s):
    case = s["case"]
    x = s["logits"].double()                          # 64 bits: experts next to the border of the selection
    t, e = x.shape
    if case["scores"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        w = torch.exp(x - x.amax(-1, keepdim=True))
        p = w / w.sum(-1, keepdim=True)
    sel = p if s["bias"] is None else p + s["bias"].double()
    n = case["groups"]
    if case["top_groups"] < n:
        g = sel.reshape(t, n, e // n)
        best = torch.sort(g, dim=-1, descending=True)[0]
        score = best[..., 0] if case["group_score"] == "max" else best[..., :2].sum(-1)
        keep = torch.sort(score, dim=-1, descending=True, stable=True)[1][:, :case["top_groups"]]
        live = (keep[:, :, None] == torch.arange(n, device=x.device)).any(1)
        sel = torch.where(live[..., None], g, torch.full_like(g, float("-inf"))).reshape(t, e)
    idx = torch.sort(sel, dim=-1, descending=True, stable=True)[1][:, :case["k"]]
    gate = p.gather(1, idx)
    if case["renorm"]:
        gate = gate / (gate.sum(-1, keepdim=True) + 1e-20)
    return dict(idx=idx.int(), gate=(gate * case["scale"]).float())


def _rotate(x, cos, sin, rot, interleaved):
    """x [T, H, D] in 64 bits, cos and sin [T, rot / 2]."""
    c, z = cos[:, None], sin[:, None]
    r = x[..., :rot]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * z, b * c + a * z], -1).reshape(r.shape)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * c - b * z, b * c + a * z], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _rope_plain(s):
    case = s["case"]
    # 64 bits: the angles of far positions, and values next to the border between two codes
    angle = s["pos"].double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _rotate(s["q"].double(), cos, sin, case["rot"], case["interleaved"])
    k = _values(*_quantise(_rotate(s["k"].double(), cos, sin, case["rot"], case["interleaved"])))
    v = _values(*_quantise(s["v"].float()))
    live = (s["slots"] >= 0)[:, None, None]
    zero = torch.zeros((), device=k.device)
    to = s["q"].dtype
    return dict(q=q.to(to), k=torch.where(live, k, zero).to(to), v=torch.where(live, v, zero).to(to))


def _attn_plain(s):
    case = s["case"]
    dim, ps, hk = case["dim"], s["page"], case["kv_heads"]
    rep = case["heads"] // hk
    b, mq = s["kv"].shape[0], s["max_q"]
    dev = s["q"].device
    cols = max(1, -(-s["max_kv"] // ps))
    kv, start = s["kv"].long(), s["start"].long()
    blocks = s["cache"][s["table"][:, :cols].clamp(min=0).long()]             # [B, P, H, nb, 18 D]
    k, v = _unpack(blocks, dim)
    length = cols * ps
    k = k.transpose(1, 2).reshape(b, hk, length, dim)
    v = v.transpose(1, 2).reshape(b, hk, length, dim)
    j = torch.arange(length, device=dev)
    live = (j[None] < kv[:, None])[:, None, :, None]
    zero = torch.zeros((), device=dev)
    k, v = torch.where(live, k, zero), torch.where(live, v, zero)
    i = torch.arange(mq, device=dev)
    at = (start[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][at].float().reshape(b, mq, hk, rep, dim).permute(0, 2, 1, 3, 4).reshape(b, hk, mq * rep, dim)
    n = start[1:] - start[:-1]
    pos = kv[:, None] - n[:, None] + i[None]                                  # [B, mq]
    end = pos + 1
    if s["prefix"] is not None:
        end = torch.maximum(end, s["prefix"].long()[:, None])
    see = (j[None, None] < kv[:, None, None]) & (j[None, None] < end[..., None])
    if case["window"]:
        see &= j[None, None] > pos[..., None] - case["window"]
    if s["first"] is not None:
        see &= j[None, None] >= s["first"].long()[at][..., None]
    see = see[:, None, :, None].expand(b, 1, mq, rep, length).reshape(b, 1, mq * rep, length)
    sc = torch.matmul(q, k.transpose(2, 3))
    sc.mul_(dim ** -0.5)
    if case["cap"]:
        sc.div_(case["cap"]).tanh_().mul_(case["cap"])
    if s["slopes"] is not None:
        far = (pos[..., None] - j).abs().float()                              # [B, mq, L]
        sc = sc.reshape(b, hk, mq, rep, length)
        for u in range(rep):
            sc[:, :, :, u] -= s["slopes"].reshape(1, hk, rep, 1, 1)[:, :, u] * far[:, None]
        sc = sc.reshape(b, hk, mq * rep, length)
    sc.masked_fill_(~see, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    sc.sub_(m).exp_()
    l = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc, v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + torch.log(l)).reshape(b, hk, mq, rep)
    t = torch.arange(s["q"].shape[0], device=dev)
    r = torch.searchsorted(start, t, right=True) - 1
    o = o.reshape(b, hk, mq, rep, dim)[r, :, t - start[r]]
    return dict(out=o.reshape(-1, case["heads"], dim).to(s["q"].dtype),
                lse=lse[r, :, t - start[r]].reshape(-1, case["heads"]))


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def _keep(dq, s):
    """What a program keeps: the routing, the cache handle and, for attention, the workspace."""
    c = s["case"]
    if "handle" not in s:
        if c["op"] == "route":
            s["handle"] = dq.MoeRouting(scores=c["scores"], bias=s["bias"], n_groups=c["groups"],
                                        top_groups=c["top_groups"], group_score=c["group_score"],
                                        renormalize=c["renorm"], scale=c["scale"])
            return s["handle"]
        s["handle"] = dq.KvCache(s["cache"], page_size=s["page"], n_kv_heads=c["kv_heads"], head_dim=c["dim"])
        if c["op"] == "attn":
            s["ws"] = torch.empty(dq.kv_attention_workspace_size(s["handle"], c["heads"], c["batch"], s["q"].shape[0],
                                                                 s["max_q"]), dtype=torch.uint8, device="cuda")
    return s["handle"]


def run(s):
    c = s["case"]
    if not own:
        return {"route": _route_plain, "rope": _rope_plain, "attn": _attn_plain}[c["op"]](s)
    import dequant_gemv_moe_gb300 as dq
    h = _keep(dq, s)
    if c["op"] == "route":
        idx, gate = dq.moe_route(s["logits"], c["k"], h, out=s["out"])
        return dict(idx=idx, gate=gate)
    if c["op"] == "rope":
        q = dq.kv_append_rope(h, s["q"], s["k"], s["v"], s["slots"], s["pos"], s["freq"],
                              interleaved=c["interleaved"], out=s["out"])
        k, v = dq.kv_read(h, s["slots"], out=s["kv"])
        return dict(q=q, k=k, v=v)
    out, lse = dq.kv_attention(h, s["q"], s["start"], s["kv"], s["table"], window=c["window"], max_q_len=s["max_q"],
                               softcap=c["cap"], slopes=s["slopes"], prefix_len=s["prefix"], first_pos=s["first"],
                               out=s["out"], lse=s["lse"], ws=s["ws"])
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        el = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": t * (e * el + 8 * case["k"]) + (4 * e if case["bias"] else 0), "flops": 4 * t * e}
    hk, h, dim = case["kv_heads"], case["heads"], case["dim"]
    if case["op"] == "rope":
        el = 4 if case["dtype"] == "fp32" else 2
        # rows in, q and blocks out; blocks in, values out
        per = 2 * h * dim * el + 2 * hk * dim * (2 * el + 2 * 0.5625) + 20
        return {"bytes": case["tokens"] * per + 2 * case["rot"], "flops": 3 * case["tokens"] * (h + hk) * case["rot"]}
    new, kv, first, prefix = _spans(case)
    pairs = seen = at = 0
    for r, (n, c) in enumerate(zip(new, kv)):
        w = case["window"] or c + 1
        low, top = c, 0
        for i in range(n):
            p = c - n + i
            lo, hi = max(0, p + 1 - w), min(c, max(p + 1, prefix[r] if prefix else 0))
            if first:
                lo = max(lo, first[at + i])
            pairs += max(0, hi - lo)
            low, top = min(low, lo), max(top, hi)
        at += n
        seen += max(0, top - low)
    rows = sum(new) * h
    return {"bytes": seen * hk * dim * 1.125 + rows * (dim * 4 + 4), "flops": 4 * pairs * h * dim}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _route64(case, s):
    l = s["logits"].double()
    p = torch.sigmoid(l) if case["scores"] == "sigmoid" else torch.softmax(l, -1)
    v = p + (0 if s["bias"] is None else s["bias"].double())
    t, e = v.shape
    per = e // case["groups"]
    at = torch.arange(t, device=v.device)
    if case["top_groups"] < case["groups"]:
        two = min(per, 2 if case["group_score"] == "top2" else 1)
        rank = torch.stack([v[:, i * per:(i + 1) * per].topk(two, -1)[0].sum(-1) for i in range(case["groups"])], 1)
        out = torch.ones_like(v, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            m = rank.amax(1, keepdim=True)
            b = (rank == m).double().cumsum(1).eq(0).sum(1)                  # the first of the largest
            out[at[:, None], b[:, None] * per + torch.arange(per, device=v.device)] = False
            rank[at, b] = -math.inf
        v = v.masked_fill(out, -math.inf)
    chosen = []
    for _ in range(case["k"]):
        b = (v == v.amax(1, keepdim=True)).double().cumsum(1).eq(0).sum(1)
        chosen.append(b)
        v[at, b] = -math.inf
    idx = torch.stack(chosen, 1)
    w = torch.gather(p, 1, idx)
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return {"idx": idx.int(), "gate": w * case["scale"]}


def _round_trip64(x):
    """Q4_0 of each 32 values: the value of the largest magnitude becomes code 0 (or the scale's own rounding of it)."""
    g = x.double().clamp(-65504, 65504).unflatten(-1, (-1, 32))
    top = torch.gather(g, -1, torch.sort(g.abs(), dim=-1, descending=True, stable=True).indices[..., :1])
    d = (top / -8).to(torch.float16).double()
    q = torch.where(d == 0, torch.zeros_like(g), torch.floor(g / torch.where(d == 0, 1.0, d) + 0.5).clamp(-8, 7))
    return (q * d).flatten(-2)


def _turned64(x, s, case):
    """Pairs as complex numbers, multiplied by e^(i angle)."""
    r = case["rot"]
    y = x.double().clone()
    z = torch.polar(torch.ones_like(s["freq"], dtype=torch.float64).expand(len(x), -1),
                    s["pos"].double()[:, None] * s["freq"].double())[:, None]
    one, two = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    w = torch.complex(y[..., one].contiguous(), y[..., two].contiguous()) * z
    y[..., one], y[..., two] = w.real, w.imag
    return y


def _where(dim, dev):
    """For each (token, value) of a block: byte of its K code, of its V code, and which half of the byte."""
    i = torch.arange(16, device=dev)[:, None]
    x = torch.arange(dim, device=dev)[None]
    grp, e = x // 32, x % 32
    w = min(dim // 32, 4)
    word = ((grp // w * 16 + i) * 4 + e // 8) * w + grp % w
    nib = (e % 8) // 2 + 4 * (e % 2)
    unit = ((((i // 8 * (dim // 32 // w) + grp // w) * 8 + e // 4) * 4 + i % 8 // 2) * 2 + i % 2) * w + grp % w
    kd = 16 * dim + 2 * (i * (dim // 32) + grp)
    vd = 17 * dim + 2 * (((i % 8 // 2) * (dim // 32) + grp) * 4 + i // 8 * 2 + i % 2)
    return (word * 4 + nib // 2, nib % 2 * 4, kd), (8 * dim + unit * 2 + e % 4 // 2, (e % 4 % 2 * 4).expand(16, dim), vd)


def _values64(blocks, dim, where):
    at, shift, scale = where
    code = (blocks[..., at] >> shift.to(torch.uint8)) & 15
    d = blocks[..., torch.stack([scale, scale + 1], -1)].contiguous().view(torch.float16)[..., 0]
    return d.double() * (code.double() - 8)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route64(case, s)
    if case["op"] == "rope":
        gone = (s["slots"] < 0)[:, None, None]
        return {"q": _turned64(s["q"], s, case), "k": _round_trip64(_turned64(s["k"], s, case)).masked_fill(gone, 0.0),
                "v": _round_trip64(s["v"]).masked_fill(gone, 0.0)}
    dim, ps, hk = case["dim"], case["page"], case["kv_heads"]
    rep = case["heads"] // hk
    new, kv, first, prefix = _spans(case)
    wk, wv = _where(dim, s["q"].device)
    slopes = [2.0 ** (-8.0 * (u + 1) / case["heads"]) for u in range(case["heads"])]
    outs, lses, at = [], [], 0
    for r, (n, c) in enumerate(zip(new, kv)):
        q = s["q"][at:at + n].double()
        low = first[at:at + n] if first else None
        at += n
        if n == 0:
            continue
        pages = s["table"][r, :-(-c // ps)].long()
        j = torch.arange(c, device=q.device)
        p = torch.arange(c - n, c, device=q.device)[:, None]
        hide = j[None] > p
        if prefix:
            hide = hide & (j[None] >= prefix[r])
        if case["window"]:
            hide = hide | (j[None] <= p - case["window"])
        if low:
            hide = hide | (j[None] < torch.tensor(low, device=q.device)[:, None])
        o = torch.zeros(n, case["heads"], dim, dtype=torch.float64, device=q.device)
        lse = torch.full((n, case["heads"]), -math.inf, dtype=torch.float64, device=q.device)
        for h in range(hk):
            blocks = s["cache"][pages, h].reshape(-1, 18 * dim)
            k = _values64(blocks, dim, wk).reshape(-1, dim)[:c]
            v = _values64(blocks, dim, wv).reshape(-1, dim)[:c]
            for u in range(h * rep, (h + 1) * rep):
                z = q[:, u] @ k.T / math.sqrt(dim)
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if case["bias"]:
                    z = z - float(torch.tensor(slopes[u]).float()) * (p - j[None]).abs().double()
                z = z.masked_fill(hide, -math.inf)
                lse[:, u] = torch.logsumexp(z, -1)
                o[:, u] = torch.nan_to_num(torch.softmax(z, -1), nan=0.0) @ v
        outs.append(o)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
