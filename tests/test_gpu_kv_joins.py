"""dq_kv_attention's shares and joins with bars that a lost, doubled or misplaced tile
of tokens cannot meet (-m gpu).

1. lse.  Kernels that take K exactly (few rows; items that see at most 1024 tokens) sum in fp32:
   2^-18 (1 + |lse|).  Else K is rounded to fp16, each value by 2^-12 of itself at most, about
   evenly: scores are off by s_j = 2^-12 scale sqrt(sum_d q_d^2 k_jd^2) / sqrt(3) (rms) and the lse by
   sqrt(sum_j p_j^2 s_j^2), taken eight times.  A tile of 32 tokens left out of 40000 moves it by
   8e-4, eighteen times the bar.
2. Flat rows.  q = 0 makes every weight the same power of two, and V scales of 6 bits make every
   product exact: out is V's mean with fp32's own rounding, within 2^-16 of the mean magnitude
   (sums of up to 2^16 terms of rounding 2^-24, in blocks).  V grows along the request and differs from value to value,
   so that a tile missing, doubled or taken from elsewhere shows in every output."""
import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Case, dq  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

CALLS = [
    # new, kv, H, n_kv, D, ps, window
    ([1], [40000], 4, 1, 128, 64, 0),              # one item over every CTA of the streaming kernel
    ([2, 1], [30011, 9000], 3, 1, 64, 64, 0),
    ([1], [20000], 8, 1, 256, 64, 0),
    ([1] * 3, [4000, 700, 16000], 8, 8, 128, 16, 0),         # whole, in clusters, in shares
    ([1], [4000], 8, 8, 64, 32, 0),
    ([1], [1900], 16, 8, 256, 32, 0),
    ([3, 1, 6, 2, 8], [3, 2000, 600, 129, 4000], 28, 4, 128, 32, 0),
    ([1] * 16, [300 + 97 * i for i in range(16)], 8, 4, 256, 128, 500),
    ([1] * 700, [(37 * i) % 300 for i in range(700)], 2, 1, 64, 16, 0),
    ([70], [30000], 1, 1, 128, 64, 0),             # the many-row kernel
    ([300, 20], [6000, 9000], 1, 1, 64, 64, 0),
    ([66], [9000], 2, 2, 256, 64, 0),
    ([900, 1500, 300, 2200, 64, 1100], [900, 1500, 300, 2200, 64, 1100], 3, 3, 64, 16, 0),   # CTAs go from exact scores
    ([900, 1500, 300, 2200, 64, 1100], [900, 1500, 300, 2200, 64, 1100], 2, 2, 128, 16, 0),  # to rounded ones and back:
    ([700, 1300, 90, 1100], [700, 1300, 90, 1100], 2, 2, 256, 16, 0),                        # buffers by twos and by ones
    ([513, 1, 1025, 40], [2000, 900, 1025, 1600], 8, 2, 128, 16, 0),
    ([400, 700, 129], [3000, 700, 2000], 4, 4, 128, 32, 1500),
    ([400, 700, 129], [3000, 700, 2000], 4, 4, 64, 32, 600),
]


def exact_rows(c, window):
    """Which rows of c the kernels score exactly: of few rows per K/V head, or in items that end by 1024 tokens (an
    item's rows span 256 tokens at most) or whose window is no wider."""
    few = max(c.new) * c.H // c.n_kv <= 64
    out = []
    for n, kv in zip(c.new, c.kv):
        one = few or n * c.H // c.n_kv <= 32 or 0 < window <= 1024
        out += [one or kv - n + i + 1 <= 1024 - 256 for i in range(n)]
    return np.array(out)


def rounding_of_lse(c, window):
    """The rms error of each lse from K's rounding (2^-12 of each value, evenly)."""
    out = np.zeros((len(c.q64), c.H))
    scale, rep = c.D ** -0.5, c.H // c.n_kv
    for r, (n, kv) in enumerate(zip(c.new, c.kv)):
        if n == 0 or kv == 0:
            continue
        j = np.arange(kv)
        slots = c.table[r, j // c.ps].astype(np.int64) * c.ps + j % c.ps
        p = kv - n + np.arange(n)
        see = j[None] <= p[:, None]
        if window:
            see &= j[None] > p[:, None] - window
        for h in range(c.n_kv):
            k, _ = kv_ref.read(c.host, c.ps, c.D, h, slots)
            for u in range(h * rep, (h + 1) * rep):
                x = c.q64[c.start[r]:c.start[r] + n, u]
                s = np.where(see, scale * (x @ k.T), -np.inf)
                w = np.exp(s - np.max(s, 1, keepdims=True, initial=-1e300))
                w /= np.maximum(w.sum(1, keepdims=True), 1e-300)
                off = (x * x) @ (k * k).T * (scale * 2.0 ** -12) ** 2 / 3
                out[c.start[r]:c.start[r] + n, u] = np.sqrt((w * w * np.where(see, off, 0)).sum(1))
    return out


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_lse_counts_every_token_once(dq, i):  # noqa: F811
    new, kv, H, n_kv, D, ps, window = CALLS[i]
    c = Case(dq, 50 + i, new, kv, H, n_kv, D, ps, "fp16")
    out, lse = c.run(max_q_len=max(new), window=window)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    ref = kv_ref.attention(c.host, ps, D, c.q64, c.start, kv, c.table, D ** -0.5, True, window, n_kv)[1]
    none = np.isneginf(ref)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), none)
    ref, got = np.where(none, 0, ref), np.where(none, 0, got)
    bar = 2.0 ** -18 * (1 + np.abs(ref))
    exact = exact_rows(c, window)
    if not exact.all():
        bar = bar + np.where(exact[:, None], 0, 8 * rounding_of_lse(c, window))
    off = np.abs(got - ref)
    assert (off <= bar).all(), (off / bar).max()


@pytest.mark.parametrize("i", range(len(CALLS)))
def test_flat_rows_are_the_mean_of_every_token(dq, i):  # noqa: F811
    new, kv, H, n_kv, D, ps, window = CALLS[i]
    c = Case(dq, 80 + i, new, kv, H, n_kv, D, ps, "fp16")
    c.q.zero_()
    c.q64 = np.zeros_like(c.q64)
    vs = c.host[..., 17 * D:].view(np.float16)
    bits = vs.view(np.uint16)
    bits &= np.uint16(0xFFE0)                      # 6 significant bits (NaN keeps its own)
    for r, n in enumerate(kv):
        for p in range(-(-n // ps)):
            vs[c.table[r, p]] *= np.float16(2.0 ** (8 * p * ps // n - 4))     # 2^-4 .. 2^3 along the request
    c.cache.pages.copy_(torch.from_numpy(c.host))
    out, lse = c.run(max_q_len=max(new), window=window, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    ref, rl, mag, _ = kv_ref.attention(c.host, ps, D, c.q64, c.start, kv, c.table, D ** -0.5, True, window, n_kv)
    off = np.abs(out.double().cpu().numpy() - ref)
    assert (off <= 2.0 ** -16 * mag).all(), (off / np.maximum(mag, 1e-300)).max()
    none = np.isneginf(rl)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), none)
    rl = np.where(none, 0, rl)
    assert 32 / max(kv) > 10 * 2.0 ** -18 * (1 + np.log(max(kv)))           # what a lost tile would do to it
    assert (np.abs(np.where(none, 0, got) - rl) <= 2.0 ** -18 * (1 + np.abs(rl))).all()
