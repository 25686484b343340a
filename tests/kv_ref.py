"""The 4-bit K/V cache's operators from their definitions (include/dqmoe.h), in
plain numpy and 64 bits: the block layout byte by byte, the Q4_0 rounding, a
step's plan one request at a time, and attention row by row."""
import numpy as np


def k_code(D, i, x):
    """(byte, shift) of token i's K code of value x inside a block."""
    G = D // 32
    W = min(G, 4)
    g, e = divmod(x, 32)
    t, n = divmod(e, 8)
    nib = (n >> 1) + 4 * (n & 1)
    word = (((g // W) * 16 + i) * 4 + t) * W + g % W
    return 4 * word + nib // 2, 4 * (nib % 2)


def v_code(D, i, x):
    G = D // 32
    W = min(G, 4)
    g, e = divmod(x, 32)
    a, n = divmod(e, 4)
    j, rest = divmod(i, 8)
    t, ii = divmod(rest, 2)
    unit = ((((j * (G // W) + g // W) * 8 + a) * 4 + t) * 2 + ii) * W + g % W
    return 8 * D + 2 * unit + n // 2, 4 * (n % 2)


def k_scale(D, i, g):
    return 16 * D + 2 * (i * (D // 32) + g)


def v_scale(D, i, g):
    j, rest = divmod(i, 8)
    t, ii = divmod(rest, 2)
    return 17 * D + 2 * ((t * (D // 32) + g) * 4 + j * 2 + ii)


_TABLES = {}


def tables(D):
    """Index arrays [16][D] of the four fields: code bytes, shifts, scale bytes, for K and V."""
    if D not in _TABLES:
        out = []
        for code, scale in ((k_code, k_scale), (v_code, v_scale)):
            b = np.array([[code(D, i, x)[0] for x in range(D)] for i in range(16)])
            s = np.array([[code(D, i, x)[1] for x in range(D)] for i in range(16)], dtype=np.uint8)
            d = np.array([[scale(D, i, x // 32) for x in range(D)] for i in range(16)])
            out.append((b, s, d))
        _TABLES[D] = out
    return _TABLES[D]


def quantise(x):
    """x [..., D] float -> (codes, scales as float64 [..., D / 32]): every group of 32 in exact arithmetic
    but for the scale's own rounding to fp16."""
    x = np.clip(np.asarray(x, dtype=np.float64), -65504.0, 65504.0)
    g = x.reshape(*x.shape[:-1], -1, 32)
    first = np.argmax(np.abs(g), axis=-1)            # the first of equal ones
    m = np.take_along_axis(g, first[..., None], -1)[..., 0]
    d = (m / -8.0).astype(np.float16).astype(np.float64)
    safe = np.where(d == 0, 1.0, d)[..., None]
    c = np.clip(np.floor(g / safe + 8.5), 0, 15)
    c = np.where(d[..., None] == 0, 8, c)
    return c.reshape(x.shape).astype(np.int64), d


def write(cache, page_size, D, h, slot, kx, vx):
    """Puts one token's K and V rows of head h into cache (uint8 [pages][heads][blocks][18 D])."""
    page, off = divmod(int(slot), page_size)
    blk = cache[page, h, off // 16]
    i = off % 16
    for x, (b, s, d) in zip((kx, vx), tables(D)):
        c, sc = quantise(x)
        for v in range(D):
            at, sh = b[i, v], s[i, v]
            blk[at] = (int(blk[at]) & ~(15 << int(sh)) & 255) | (int(c[v]) << int(sh))
        for g in range(D // 32):
            blk[d[i, 32 * g]:d[i, 32 * g] + 2] = np.array([sc[g]], dtype=np.float16).view(np.uint8)


def read(cache, page_size, D, h, slots):
    """K and V values [n][D] of head h at `slots`."""
    slots = np.asarray(slots, dtype=np.int64)
    blk = cache[slots // page_size, h, slots % page_size // 16]          # [n][18 D]
    i = slots % 16
    out = []
    for b, s, d in tables(D):
        code = (np.take_along_axis(blk, b[i], 1) >> s[i]) & 15
        sc = np.stack([np.take_along_axis(blk, d[i], 1), np.take_along_axis(blk, d[i] + 1, 1)], -1)
        sc = np.ascontiguousarray(sc).view(np.float16)[..., 0].astype(np.float64)
        out.append(sc * (code.astype(np.float64) - 8))
    return out


def plan(ctx, new, table, free, count, page_size, T):
    """One step, request by request.  free: the stack (list of page ids, bottom first; `count` of them live)."""
    table, stack = table.copy(), list(free[:count])
    B, width = table.shape
    stack_out = np.array(free).copy()
    for r in range(B):
        if new[r] < 0:
            for i in range(min(-(-int(ctx[r]) // page_size), width)):
                stack_out[len(stack)] = table[r, i]
                stack.append(int(table[r, i]))
    top, asked, popped = len(stack), 0, 0
    kv, start, served = [], [0], []
    slots, pos = [], []
    for r in range(B):
        c, n = int(ctx[r]), max(int(new[r]), 0)
        have, want = -(-c // page_size), -(-(c + n) // page_size)
        ok = new[r] >= 0 and want <= width
        if ok and want > have:
            asked += want - have
            ok = asked <= top
            if ok:
                for i in range(have, want):
                    table[r, i] = stack.pop()
                    popped += 1
        served.append(bool(ok))
        kv.append(0 if new[r] < 0 else c + n if ok else c)
        start.append(start[-1] + n)
        for i in range(n):
            p = c + i
            pos.append(p)
            slots.append(int(table[r, p // page_size]) * page_size + p % page_size if ok else -1)
    slots, pos = (slots + [-1] * T)[:T], (pos + [-1] * T)[:T]
    missed = sum(1 for r in range(B) if new[r] >= 0 and not served[r])
    return dict(table=table, stack=stack_out, kv_len=kv, q_start=start, slots=slots, positions=pos,
                free_count=top - popped, unserved=missed)


def attention(cache, page_size, D, q, start, kv_len, table, scale, causal, window, n_kv):
    """(out, lse, a, e): a = sum_j p_j |v_j| per output, e = the largest scale * sum |q| |k| a row meets: what the
    rounding of operands is multiplied with."""
    T, H, _ = q.shape
    rep = H // n_kv
    q = np.asarray(q, dtype=np.float64)
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, big = np.full((T, H), -np.inf), np.zeros((T, H))
    for r in range(len(kv_len)):
        n, L = int(start[r + 1] - start[r]), int(kv_len[r])
        if n == 0 or L == 0:
            continue
        j = np.arange(L)
        slots = table[r, j // page_size].astype(np.int64) * page_size + j % page_size
        p = L - n + np.arange(n)
        see = np.ones((n, L), dtype=bool)
        if causal:
            see &= j[None] <= p[:, None]
        if window:
            see &= j[None] > p[:, None] - window
        some = see.any(1)
        for h in range(n_kv):
            k, v = read(cache, page_size, D, h, slots)
            for u in range(h * rep, (h + 1) * rep):
                x = q[start[r]:start[r] + n, u]
                s = np.where(see, scale * (x @ k.T), -np.inf)
                m = np.where(some, s.max(1), 0.0)[:, None]
                w = np.exp(s - m)
                l = np.where(some, w.sum(1), 1.0)[:, None]
                rows = slice(start[r], start[r] + n)
                out[rows, u] = (w / l) @ v
                mag[rows, u] = (w / l) @ np.abs(v)
                lse[rows, u] = np.where(some, (m + np.log(l))[:, 0], -np.inf)
                big[rows, u] = np.where(see, scale * (np.abs(x) @ np.abs(k).T), 0.0).max(1)
    return out, lse, mag, big
