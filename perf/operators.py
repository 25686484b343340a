"""The 4-bit K/V cache operators as measured calls: plan, append + read back, attention.

`run` computes them in elementary torch operations in 32 bits where `own` is false, and through
dequant_gemv_moe_gb300 where it is true.  Both work on the same packed cache, whose layout is:

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
        # one decode step of a small serving batch: lengths in, tables and slots out (latency)
        dict(name="plan_step", op="plan", batch=48, mode="step", max_ctx=4096, chunk=1, page=16, ragged=1),
        # a large batch in which some requests finish, some are being prefilled and most decode
        dict(name="plan_mixed", op="plan", batch=1000, mode="mixed", max_ctx=30000, chunk=2000, page=32, ragged=2),
        # the K/V rows of one decode step of 64 requests (8 KV heads of 128, as Llama-3-8B has)
        dict(name="append_step", op="append", tokens=64, kv_heads=8, dim=128, dtype="bf16", page=16, skip=0, ragged=3),
        # the K/V rows of a long prompt, one token short of a round number
        dict(name="append_prompt", op="append", tokens=8191, kv_heads=8, dim=128, dtype="bf16", page=64, skip=0, ragged=4),
        # fp32 rows as the quantized GEMV writes them, odd head count, some tokens left out of the cache
        dict(name="append_odd", op="append", tokens=1023, kv_heads=5, dim=64, dtype="fp32", page=32, skip=5, ragged=5),
        # one request's decode step over a short context: the smallest call (latency)
        dict(name="attn_step_1", op="attn", batch=1, mode="step", max_q=1, max_ctx=977, heads=32, kv_heads=8, dim=128,
             dtype="bf16", page=16, window=0, ragged=6),
        # a serving batch's decode step, ragged contexts (Llama-3-8B heads): memory bound
        dict(name="attn_step_64", op="attn", batch=64, mode="step", max_q=1, max_ctx=16384, heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=16, window=0, ragged=7),
        # few requests with very long contexts (70B heads, eight query heads to a KV head)
        dict(name="attn_step_long", op="attn", batch=3, mode="step", max_q=1, max_ctx=131072, heads=64, kv_heads=8,
             dim=128, dtype="bf16", page=64, window=0, ragged=8),
        # verification of a few drafted tokens per request, seven query heads to a KV head
        dict(name="attn_verify", op="attn", batch=20, mode="few", max_q=6, max_ctx=6000, heads=28, kv_heads=4,
             dim=128, dtype="fp16", page=32, window=0, ragged=9),
        # decode with a sliding window and wide heads
        dict(name="attn_window", op="attn", batch=16, mode="step", max_q=1, max_ctx=8192, heads=8, kv_heads=4,
             dim=256, dtype="fp16", page=128, window=1024, ragged=10),
        # a chunk of a long prompt over what the cache already holds: compute bound, the largest call
        dict(name="attn_chunk", op="attn", batch=2, mode="chunk", max_q=2048, max_ctx=16384, heads=32, kv_heads=8,
             dim=128, dtype="bf16", page=64, window=0, ragged=11),
        # fresh prompts of all lengths, one query head per KV head, one request without new tokens and one
        # whose first rows see nothing
        dict(name="attn_prompts", op="attn", batch=7, mode="prompt", max_q=3001, max_ctx=0, heads=12, kv_heads=12,
             dim=64, dtype="fp16", page=16, window=0, ragged=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    ragged = rng.randrange(1 << 20)
    if op == "plan":
        mode = rng.choice(["step", "mixed"])
        return dict(op=op, batch=_log(rng, 1, 2048), mode=mode, max_ctx=_log(rng, 100, 30000),
                    chunk=1 if mode == "step" else _log(rng, 2, 2000), page=page, ragged=ragged)
    dim, dtype = rng.choice([64, 128, 128, 256]), rng.choice(["fp16", "bf16"])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8191), kv_heads=rng.randint(1, 8), dim=rng.choice([64, 128]),
                    dtype=rng.choice(["fp16", "bf16", "fp32"]), page=page, skip=rng.choice([0, 0, 5]), ragged=ragged)
    mode = rng.choice(["step", "step", "few", "chunk", "prompt"])
    kv_heads, group = rng.randint(1, 8), rng.choice([1, 2, 3, 4, 5, 7, 8])
    window = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
    c = dict(op=op, batch=0, mode=mode, max_q=1, max_ctx=0, heads=kv_heads * group, kv_heads=kv_heads, dim=dim,
             dtype=dtype, page=page, window=window, ragged=ragged)
    if mode in ("step", "few"):
        c["max_q"] = 1 if mode == "step" else rng.randint(2, 8)
        c["max_ctx"] = _log(rng, 1, 131072)
        most = 3 * 131072 * 8 * 128 // (c["max_ctx"] * kv_heads * dim)
        c["batch"] = _log(rng, 1, max(1, min(128, most)))
    else:
        c["max_q"] = _log(rng, 16, 3001)
        c["max_ctx"] = 0 if mode == "prompt" else _log(rng, 16, 16384)
        rows = c["max_q"] * (c["max_q"] + c["max_ctx"]) * kv_heads * group * dim
        most = 2 * 2048 * (2048 + 16384) * 32 * 128 // rows
        c["batch"] = _log(rng, 1, max(1, min(16, most)))
    return c


# ------------------------------------------------------------------------------------------------
# lengths: fixed by the case, so that the work of a pass is known
# ------------------------------------------------------------------------------------------------
def _lengths(case):
    """(tokens in the cache before, new tokens) of each request; -1 new tokens: the request has finished."""
    r = random.Random(case["ragged"])
    ctx, new = [], []
    for i in range(case["batch"]):
        c = r.randint(1, max(1, case["max_ctx"]))
        if case["mode"] == "step":                    # one request: the length itself; else from short to full
            n = 1
            c = case["max_ctx"] if case["batch"] == 1 or i == 0 else c
            if case["op"] == "attn" and case["batch"] <= 4:
                c = r.randint(max(1, case["max_ctx"] * 3 // 4), case["max_ctx"]) if i else case["max_ctx"]
        elif case["mode"] == "few":
            n = r.randint(1, case["max_q"])
        elif case["mode"] == "mixed":
            u = r.random()
            n = -1 if u < 0.1 else r.randint(1, case["chunk"]) if u < 0.15 else 1
        elif case["mode"] == "chunk":
            c, n = case["max_ctx"], case["max_q"]
        else:                                         # whole prompts
            c, n = 0, case["max_q"] if i == 0 else 0 if i == 1 else r.randint(1, case["max_q"])
        ctx.append(c)
        new.append(n)
    return ctx, new


def _attn_lengths(case):
    ctx, new = _lengths(case)
    kv = [c + n for c, n in zip(ctx, new)]
    if case["mode"] == "prompt" and len(kv) > 2:      # a request whose cache starts after its first rows
        kv[2] = (new[2] + 1) // 2
    return new, kv


# ------------------------------------------------------------------------------------------------
# packed blocks in elementary operations
# ------------------------------------------------------------------------------------------------
def _nibble_of(device):
    return torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device=device)      # value e of a K word -> its nibble


def _quantise(x):
    """x [..., D] -> codes [..., D] (0..15) and fp16 scales [..., D / 32], in 32 bits."""
    x = x.float().clamp(-65504.0, 65504.0)
    g = x.reshape(*x.shape[:-1], -1, 32)
    a = g.abs()
    first = (a == a.amax(-1, keepdim=True)).to(torch.int8).argmax(-1, keepdim=True)
    d = (g.gather(-1, first) * -0.125).half()
    df = d.float()
    c = torch.floor(g / torch.where(df == 0, torch.ones_like(df), df) + 8.5).clamp(0, 15)
    c = torch.where(df == 0, torch.full_like(c, 8.0), c)
    return c.to(torch.uint8).reshape(x.shape), d.squeeze(-1)


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


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + case["ragged"])
    ps = case["page"]
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        have = [-(-c // ps) for c in ctx]
        width = -(-(case["max_ctx"] + case["chunk"]) // ps)
        total = sum(-(-(c + max(n, 0)) // ps) for c, n in zip(ctx, new)) + 16
        pages = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
        held = sum(have)
        row = torch.repeat_interleave(torch.arange(len(have)), torch.tensor(have)).cuda()
        col = torch.cat([torch.arange(h) for h in have]).cuda()
        table[row, col] = pages[:held]
        stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        stack[:total - held] = pages[held:]
        t = sum(max(n, 0) for n in new)
        return dict(case=case, ctx=_i32(ctx), new=_i32(new), table=table, stack=stack, count=_i32([total - held]),
                    tokens=t, page=ps)
    dim, heads = case["dim"], case["kv_heads"]
    if case["op"] == "append":
        t = case["tokens"]
        n_pages = -(-t // ps) + 5
        cache = torch.full((n_pages, heads, ps // 16, 18 * dim), 255, dtype=torch.uint8, device="cuda")
        order = torch.randperm(n_pages, generator=g, device="cuda")
        at = torch.arange(3, t + 3, device="cuda")                # the request already holds three tokens
        slots = order[at // ps] * ps + at % ps
        if case["skip"]:
            r = random.Random(case["ragged"])
            out = [i for i in range(t) if r.randrange(100) < case["skip"]]
            slots[torch.tensor(out, dtype=torch.int64, device="cuda")] = -1
        spread = 1.0 + 3.0 * (torch.rand(1, 1, dim, generator=g, device="cuda") > 0.95)
        kv = torch.cat([_rows(g, (t, heads, dim)) * spread, _rows(g, (t, heads, dim)) * 0.5], 1).to(DT[case["dtype"]])
        # K and V are the halves of one projection's rows
        k, v = kv[:, :heads], kv[:, heads:]
        return dict(case=case, cache=cache, k=k, v=v, slots=slots, page=ps,
                    out=(torch.empty_like(k, memory_format=torch.contiguous_format),
                         torch.empty_like(v, memory_format=torch.contiguous_format)))
    new, kv = _attn_lengths(case)
    have = [-(-n // ps) for n in kv]
    n_pages = sum(have) + 3
    width = max(have) + 1
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    row = torch.repeat_interleave(torch.arange(len(have)), torch.tensor(have)).cuda()
    col = torch.cat([torch.arange(h) for h in have]).cuda()
    used = order[:sum(have)]
    table[row, col] = used
    rows = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    rows[used.long()] = (torch.tensor(kv).cuda()[row] - col * ps).clamp(max=ps)
    cache = torch.empty((n_pages, heads, ps // 16, 18 * dim), dtype=torch.uint8, device="cuda")
    _fill(cache, g, rows, dim)
    t = sum(new)
    q = _rows(g, (t, case["heads"], dim), 1.5).to(DT[case["dtype"]])
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    return dict(case=case, cache=cache, q=q, start=_i32(start), kv=_i32(kv), table=table, page=ps, max_q=max(new),
                max_kv=max(kv), out=torch.empty_like(q),
                lse=torch.empty((t, case["heads"]), dtype=torch.float32, device="cuda"))


# ------------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------------
def _plan_plain(s):
    ps, t, dev = s["page"], s["tokens"], s["ctx"].device
    ctx, new = s["ctx"].long(), s["new"].long()
    table, stack = s["table"].clone(), s["stack"].clone()
    count = s["count"].long()
    b, width = table.shape
    done, n = new < 0, new.clamp(min=0)
    have, want = (ctx + ps - 1) // ps, (ctx + n + ps - 1) // ps
    col = torch.arange(width, device=dev)
    # finished requests push their pages, in request and page order
    back = done[:, None] & (col[None] < have[:, None])
    at = (count + back.reshape(-1).cumsum(0) - 1).reshape(b, width)
    spare = torch.cat([stack, stack.new_zeros(1)])                # the last entry takes what is not pushed
    spare[torch.where(back, at, torch.full_like(at, stack.numel()))] = table
    stack = spare[:-1]
    top = count + back.sum()
    # pages are popped in request and page order
    fits = ~done & (want <= width)
    need = torch.where(fits, want - have, torch.zeros_like(have))
    incl = need.cumsum(0)
    ok = fits & ((need == 0) | (incl <= top))
    take = ok[:, None] & (col[None] >= have[:, None]) & (col[None] < want[:, None])
    place = top - 1 - (incl - need)[:, None] - (col[None] - have[:, None])
    table = torch.where(take, stack[place.clamp(0, stack.numel() - 1)], table)
    kv = torch.where(done, torch.zeros_like(ctx), torch.where(ok, ctx + n, ctx))
    start = torch.cat([n.new_zeros(1), n.cumsum(0)])
    i = torch.arange(t, device=dev)
    r = torch.searchsorted(start, i, right=True) - 1
    p = ctx[r] + i - start[r]
    page = table[r, (p // ps).clamp(max=width - 1)].long()
    slots = torch.where(ok[r], page * ps + p % ps, torch.full_like(p, -1))
    left = top - torch.where(ok, incl, torch.zeros_like(incl)).amax()
    return dict(table=table, stack=stack, kv_len=kv.int(), q_start=start.int(), slots=slots, positions=p.int(),
                free_count=left.int(), unserved=(~done & ~ok).sum().int().reshape(1))


def _append_plain(s):
    dim, ps = s["case"]["dim"], s["page"]
    kc, kd = _quantise(s["k"])
    vc, vd = _quantise(s["v"])
    g = dim // 32
    up = lambda c, d: d.float().unsqueeze(-1) * (c.float().reshape(*c.shape[:-1], g, 32) - 8.0)  # noqa: E731
    live = (s["slots"] >= 0)[:, None, None]
    k, v = up(kc, kd).reshape(kc.shape), up(vc, vd).reshape(vc.shape)
    zero = torch.zeros((), device=k.device)
    to = s["k"].dtype
    return dict(k=torch.where(live, k, zero).to(to), v=torch.where(live, v, zero).to(to))


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
    see = (j[None, None] < kv[:, None, None]) & (j[None, None] <= pos[..., None])
    if case["window"]:
        see &= j[None, None] > pos[..., None] - case["window"]
    see = see[:, None, :, None].expand(b, 1, mq, rep, length).reshape(b, 1, mq * rep, length)
    sc = torch.matmul(q, k.transpose(2, 3)) * (dim ** -0.5)
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
def _handle(dq, s):
    """The cache handle and, for attention, the workspace: a program keeps both."""
    if "handle" not in s:
        c = s["case"]
        s["handle"] = dq.KvCache(s["cache"], page_size=s["page"], n_kv_heads=c["kv_heads"], head_dim=c["dim"])
        if c["op"] == "attn":
            s["ws"] = torch.empty(dq.kv_attention_workspace_size(s["handle"], c["heads"], c["batch"], s["q"].shape[0]),
                                  dtype=torch.uint8, device="cuda")
    return s["handle"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plan_plain, "append": _append_plain, "attn": _attn_plain}[op](s)
    import dequant_gemv_moe_gb300 as dq
    if op == "plan":
        # a decode loop keeps the step's buffers
        p = s["plan"] = dq.kv_plan(s["ctx"], s["new"], s["table"], s["stack"], s["count"], page_size=s["page"],
                                   n_tokens=s["tokens"], out=s.get("plan"))
        return dict(table=s["table"], stack=s["stack"], kv_len=p.kv_len, q_start=p.q_start, slots=p.slots,
                    positions=p.positions, free_count=p.free_count, unserved=p.unserved)
    h = _handle(dq, s)
    if op == "append":
        dq.kv_append(h, s["k"], s["v"], s["slots"])
        k, v = dq.kv_read(h, s["slots"], out=s["out"])
        return dict(k=k, v=v)
    out, lse = dq.kv_attention(h, s["q"], s["start"], s["kv"], s["table"], window=s["case"]["window"],
                               max_q_len=s["max_q"], out=s["out"], lse=s["lse"], ws=s["ws"])
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    ps = case["page"]
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        t = sum(max(n, 0) for n in new)
        taken = sum(-(-(c + max(n, 0)) // ps) - -(-c // ps) for c, n in zip(ctx, new))
        given = sum(-(-c // ps) for c, n in zip(ctx, new) if n < 0)
        last = sum(1 for c, n in zip(ctx, new) if n > 0 and c % ps)   # pages that were there and take new tokens
        return {"bytes": 16 * len(ctx) + 12 * t + 8 * (taken + given) + 4 * last, "flops": 0}
    heads, dim = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        el = 4 if case["dtype"] == "fp32" else 2
        row = 2 * heads * dim
        # rows in, blocks out; blocks in, values out
        return {"bytes": case["tokens"] * (row * (2 * el + 2 * 0.5625) + 16), "flops": 0}
    new, kv = _attn_lengths(case)
    pairs = seen = 0
    for n, c in zip(new, kv):
        w = case["window"] or c + 1
        low = c
        for i in range(n):
            p = c - n + i
            pairs += max(0, min(p + 1, w))
        if n:
            low = max(0, c - n + 1 - w)
            seen += c - low
    rows = sum(new) * case["heads"]
    return {"bytes": seen * heads * dim * 1.125 + rows * (dim * 4 + 4), "flops": 4 * pairs * case["heads"] * dim}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _round_trip64(x):
    """Q4_0 of each 32 values: the value of the largest magnitude becomes code 0 (or the scale's own rounding of it)."""
    g = x.double().clamp(-65504, 65504).unflatten(-1, (-1, 32))
    top = torch.gather(g, -1, torch.sort(g.abs(), dim=-1, descending=True, stable=True).indices[..., :1])
    d = (top / -8).to(torch.float16).double()
    q = torch.where(d == 0, torch.zeros_like(g), torch.floor(g / torch.where(d == 0, 1.0, d) + 0.5).clamp(-8, 7))
    return (q * d).flatten(-2)


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
    if case["op"] == "plan":
        return None                                   # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "append":
        gone = (s["slots"] < 0)[:, None, None]
        return {n: _round_trip64(s[n]).masked_fill(gone, 0.0) for n in ("k", "v")}
    dim, ps, hk = case["dim"], case["page"], case["kv_heads"]
    rep = case["heads"] // hk
    new, kv = _attn_lengths(case)
    wk, wv = _where(dim, s["q"].device)
    outs, lses, at = [], [], 0
    for r, (n, c) in enumerate(zip(new, kv)):
        q = s["q"][at:at + n].double()
        at += n
        if n == 0:
            continue
        pages = s["table"][r, :-(-c // ps)].long()
        first = 0
        if case["window"]:
            first = max(0, c - n + 1 - case["window"]) // ps
        j = torch.arange(first * ps, c, device=q.device)
        p = torch.arange(c - n, c, device=q.device)
        hide = j[None] > p[:, None]
        if case["window"]:
            hide = hide | (j[None] <= p[:, None] - case["window"])
        o = torch.zeros(n, case["heads"], dim, dtype=torch.float64, device=q.device)
        lse = torch.full((n, case["heads"]), -math.inf, dtype=torch.float64, device=q.device)
        for h in range(hk):
            blocks = s["cache"][pages[first:], h].reshape(-1, 18 * dim)
            k = _values64(blocks, dim, wk).reshape(-1, dim)[:j.numel()]
            v = _values64(blocks, dim, wv).reshape(-1, dim)[:j.numel()]
            for u in range(rep):
                z = (q[:, h * rep + u] @ k.T / math.sqrt(dim)).masked_fill(hide, -math.inf)
                lse[:, h * rep + u] = torch.logsumexp(z, -1)
                o[:, h * rep + u] = torch.nan_to_num(torch.softmax(z, -1), nan=0.0) @ v
        outs.append(o)
        lses.append(lse)
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
