"""Attention with capped and biased scores, prefixes and first positions from its definition (include/dqmoe.h,
dq_kv_scores), row by row in numpy and 64 bits."""
import numpy as np

import kv_ref


def rows_see(n, L, causal=True, window=0, prefix=0, first=None):
    """[n][L]: what the n rows of a request of L tokens see."""
    j, p = np.arange(L)[None], (L - n + np.arange(n))[:, None]
    see = np.ones((n, L), dtype=bool)
    if causal:
        see &= (j <= p) | (j < prefix)
    if window:
        see &= j > p - window
    if first is not None:
        see &= j >= np.asarray(first)[:, None]
    return see


def attention(cache, page_size, D, q, start, kv_len, table, scale, n_kv, causal=True, window=0, softcap=0.0, slopes=None,
              prefix_len=None, first_pos=None):
    """(out, lse, mag, big, eff): mag = sum_j p_j |v_j|, big = the largest scale * sum |q| |k| a row meets, eff = the
    largest |score| and |bias| that a row's sum is formed of."""
    T, H, _ = q.shape
    rep = H // n_kv
    q = np.asarray(q, dtype=np.float64)
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, big, eff = np.full((T, H), -np.inf), np.zeros((T, H)), np.zeros((T, H))
    for r in range(len(kv_len)):
        n, L = int(start[r + 1] - start[r]), int(kv_len[r])
        if n == 0 or L == 0:
            continue
        rows = slice(int(start[r]), int(start[r]) + n)
        j = np.arange(L)
        slots = table[r, j // page_size].astype(np.int64) * page_size + j % page_size
        see = rows_see(n, L, causal, window, 0 if prefix_len is None else int(prefix_len[r]),
                       None if first_pos is None else first_pos[rows])
        some = see.any(1)
        dist = np.abs((L - n + np.arange(n))[:, None] - j[None]).astype(np.float64)
        for h in range(n_kv):
            k, v = kv_ref.read(cache, page_size, D, h, slots)
            for u in range(h * rep, (h + 1) * rep):
                x = q[rows, u]
                s = scale * (x @ np.where(see.any(0)[:, None], k, 0.0).T)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                b = np.zeros_like(s) if slopes is None else float(np.float32(slopes[u])) * dist
                s = np.where(see, s - b, -np.inf)
                m = np.where(some, s.max(1), 0.0)[:, None]
                w = np.exp(s - m)
                l = np.where(some, w.sum(1), 1.0)[:, None]
                vv = np.where(see.any(0)[:, None], v, 0.0)
                out[rows, u] = (w / l) @ vv
                mag[rows, u] = (w / l) @ np.abs(vv)
                lse[rows, u] = np.where(some, (m + np.log(l))[:, 0], -np.inf)
                kk = np.where(see.any(0)[:, None], np.abs(k), 0.0)
                big[rows, u] = np.where(see, scale * (np.abs(x) @ kk.T), 0.0).max(1)
                # a bias is rounded where it counts: in scores within 30 of the largest
                eff[rows, u] = np.where(see & (s >= m - 30), np.abs(s) + 2 * b, 0.0).max(1)
    return out, lse, mag, big, eff
