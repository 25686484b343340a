"""dq_kv_attention_ex: capped and biased scores, prefixes and first positions against their definition in 64 bits
(tests/scores_ref.py).

Bars: test_gpu_kv's, with the score's own roundings added to E.  A cap moves a score by less than what it is given
moves, and is itself held to 2.5e-7 of it (4e-7 of the cap for many rows: its own bar below); a bias is a product
and a sum of fp32: 2^-22 of the largest of both.  A row's largest weight is 2^4 or more where scores are capped or
biased, so what fp16 rounds off below its normal range is 2^-25 / 2^4 of it for each token.  No K is rounded
whatever the number of rows: the lse is held to fp32's sums and these alone."""
import numpy as np
import pytest
import torch

import kv_ref
import scores_ref
from test_gpu_kv import U, Case, _i32, dq  # noqa: F401  (dq is the fixture)

pytestmark = pytest.mark.gpu


class Scored(Case):
    def call(self, exact=False, scale=None, causal=True, window=0, softcap=0.0, slopes=None, prefix_len=None,
             first_pos=None, **kw):
        out, lse = self.run(max_q_len=max(self.new), scale=scale, causal=causal, window=window, softcap=softcap,
                            slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32).cuda(),
                            prefix_len=None if prefix_len is None else _i32(prefix_len),
                            first_pos=None if first_pos is None else _i32(first_pos), **kw)
        torch.cuda.synchronize()
        assert self.dq.device_status() == 0
        ref, rl, mag, big, eff = scores_ref.attention(
            self.host, self.ps, self.D, self.q64, self.start, self.kv, self.table, self.D ** -0.5 if scale is None else scale,
            self.n_kv, causal, window, softcap, slopes, prefix_len, first_pos)
        own = 2.0 ** -21 * eff + (4e-7 * min(softcap, 100.0) + (2.5e-7 * softcap if softcap > 100 else 0.0))
        e = 2.0 ** -11 * big + own
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        vs = np.abs(self.host[..., 17 * self.D:].view(np.float16).astype(np.float64))
        w = 2.0 ** -25 if out.dtype == torch.float16 else 0.0
        bar = (U[out.dtype] * np.abs(ref) + w + (4 * 2.0 ** -11 + 2 * e[..., None]) * mag +
               max(self.kv) * 2.0 ** -29 * 8 * np.nanmax(vs))
        assert np.isfinite(o).all()
        off = np.abs(o - ref)
        worst = np.max(np.where(off == 0, 0.0, off / np.where(bar == 0, 1e-300, bar)))
        assert worst <= 1, worst
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l), none) and (o[none] == 0).all()
        off = np.abs(np.where(none, 0, l) - np.where(none, 0, rl))
        assert (off <= (own if exact else e) + 2.0 ** -18 * (1 + np.abs(np.where(none, 0, rl)))).all(), off.max()
        return out, lse


def steep(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def documents(new, kv, rng, longest=90):
    """Ascending first positions: what the cache holds belongs to the first document."""
    first = []
    for n, c in zip(new, kv):
        at, left = 0, 0
        for i in range(n):
            if left == 0:
                at, left = (c - n + i if i else 0), int(rng.integers(1, longest))
            first.append(max(at, 0))
            left -= 1
    return np.array(first, dtype=np.int32)


SHAPES = [
    # new, kv, H, n_kv, D, ps, dtype
    ([1], [1], 8, 8, 64, 16, "fp16"),
    ([1], [977], 32, 8, 128, 16, "bf16"),
    ([1] * 7, [1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, "bf16"),
    ([1] * 3, [700, 0, 33], 8, 1, 256, 32, "bf16"),
    ([1, 0, 1], [300, 300, 257], 3, 1, 128, 256, "fp16"),
    ([3, 1, 6, 2], [3, 1, 600, 129], 28, 4, 128, 32, "fp16"),
    ([4, 7], [2, 3], 8, 2, 128, 16, "fp16"),                 # rows before the cache's first token
    ([5, 8], [40, 1000], 5, 5, 64, 16, "bf16"),
    ([1], [20000], 8, 1, 128, 64, "bf16"),                   # over many shares, joined
    ([130], [130], 4, 1, 128, 16, "bf16"),                   # prompts
    ([300, 1, 77], [300, 150, 77], 4, 4, 64, 64, "fp16"),
    ([257, 100], [700, 356], 8, 2, 128, 32, "fp16"),
    ([129, 64], [500, 64], 6, 2, 256, 16, "bf16"),
    ([200, 333], [90, 1000], 7, 1, 128, 128, "bf16"),
    ([31, 65, 1, 0, 500], [31, 800, 640, 20, 500], 8, 2, 128, 16, "bf16"),
    ([700], [2600], 2, 2, 128, 16, "fp16"),                  # rows that see more than 1024 tokens
]
MODS = [
    dict(softcap=50.0), dict(softcap=2.0), dict(slopes=True), dict(softcap=0.5, slopes=True), dict(prefix=True),
    dict(docs=True), dict(docs=True, prefix=True), dict(docs=True, softcap=3.0, slopes=True, prefix=True),
    dict(window=40, prefix=True), dict(window=70, softcap=1.0, docs=True), dict(causal=False, slopes=True),
    dict(causal=False, docs=True, softcap=5.0), dict(slopes=True, prefix=True, window=200),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
@pytest.mark.parametrize("m", range(len(MODS)))
def test_scores(dq, i, m):  # noqa: F811
    new, kv, H, n_kv, D, ps, dtype = SHAPES[i]
    rng = np.random.default_rng(1000 * i + m)
    c = Scored(dq, 300 + i, new, kv, H, n_kv, D, ps, dtype)
    kw = dict(MODS[m])
    if kw.pop("slopes", False):
        kw["slopes"] = steep(H)
    if kw.pop("prefix", False):
        kw["prefix_len"] = np.array([int(rng.integers(-3, k + 20)) for k in kv], dtype=np.int32)
    if kw.pop("docs", False):
        kw["first_pos"] = documents(new, kv, rng)
    out, lse = c.call(exact=True, **kw)
    again, lse2 = c.call(exact=True, **kw)                       # the same bits every time
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,kv,H,n_kv,D", [([1] * 4, [5, 100, 3000, 0], 8, 2, 128), ([3, 7], [900, 33], 8, 8, 64),
                                             ([400, 90], [400, 900], 4, 2, 64), ([600], [1500], 2, 1, 128),
                                             ([300, 200], [2500, 200], 3, 3, 256)])
def test_counts_of_what_rows_see(dq, new, kv, H, n_kv, D):  # noqa: F811
    # rows of zeros weigh all that they see alike: lse is the count's logarithm, and a tile that is lost, doubled or
    # misplaced shows; with slopes and no scores it is the bias' own sum
    rng = np.random.default_rng(sum(new))
    c = Scored(dq, 77, new, kv, H, n_kv, D, 16, "fp16")
    c.q.zero_()
    c.q64 = c.q64 * 0
    for kw in (dict(prefix_len=[k // 2 for k in kv]), dict(first_pos=documents(new, kv, rng, 300)),
               dict(first_pos=documents(new, kv, rng, 5), prefix_len=[k // 3 for k in kv]),
               dict(prefix_len=[k // 2 for k in kv], window=37), dict(softcap=30.0), dict(slopes=[0.0] * H),
               dict(slopes=steep(H)), dict(slopes=[-1e-3] * H), dict(slopes=steep(H), prefix_len=[k // 2 for k in kv])):
        _, lse = c.call(exact=True, **kw)
        if "slopes" not in kw:
            got = lse.double().cpu().numpy()
            at = 0
            for r, (n, L) in enumerate(zip(new, kv)):
                if L:
                    f = kw.get("first_pos")
                    see = scores_ref.rows_see(n, L, True, kw.get("window", 0), int(kw.get("prefix_len", [0] * 9)[r]),
                                              None if f is None else f[at:at + n]).sum(1)
                    assert np.array_equal(np.rint(np.exp(got[at:at + n])), np.repeat(see[:, None], H, 1))
                at += n


@pytest.mark.parametrize("new,kv,D", [([1] * 3, [300, 77, 500], 128), ([150, 40], [300, 40], 64), ([6], [2000], 256)])
@pytest.mark.parametrize("skew", [0.05, 1.0, 30.0])
def test_caps_from_flat_to_saturated(dq, new, kv, D, skew):  # noqa: F811
    c = Scored(dq, 9, new, kv, 8, 2, D, 16, "bf16")
    c.q.mul_(skew)
    c.q64 = c.q.double().cpu().numpy()
    for cap in (0.01, 1.0, 5.0, 50.0, 1e6):
        c.call(exact=True, softcap=cap)


def test_first_positions_that_leave_rows_empty(dq):  # noqa: F811
    for new, kv, H, n_kv, D in (([1, 3], [50, 40], 4, 2, 128), ([200], [260], 2, 2, 64)):
        c = Scored(dq, 10, new, kv, H, n_kv, D, 16, "fp16")
        T = sum(new)
        first = np.concatenate([np.sort(np.random.default_rng(1).integers(0, L + 9, n)) for n, L in zip(new, kv)])
        c.call(exact=True, first_pos=first)
        c.call(exact=True, first_pos=np.full(T, 2 ** 31 - 1))
        out, lse = c.call(exact=True, first_pos=np.full(T, -2 ** 31), prefix_len=[2 ** 31 - 1] * len(new))
        plain, l2 = c.run(max_q_len=max(new), causal=False)
        assert torch.allclose(out.float(), plain.float(), atol=2e-2) and torch.allclose(lse, l2, atol=1e-4)


def test_nothing_given_is_the_plain_call(dq):  # noqa: F811
    import ctypes
    c = Scored(dq, 11, [40, 1], [90, 300], 4, 2, 128, 16, "fp16")
    a, b = c.run(max_q_len=40), c.run(max_q_len=40, softcap=0.0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # a descriptor of zeros is no descriptor
    from dequant_gemv_moe_gb300 import _lib, kv as kvm
    seen = []
    f, kvm._attention = kvm._attention, lambda *p: seen.append(p) or f(p[0], p[1], ctypes.byref(_lib.KvScores()), *p[3:])
    try:
        d = c.run(max_q_len=40)
    finally:
        kvm._attention = f
    assert seen and seen[0][2] is None and all(torch.equal(x, y) for x, y in zip(a, d))


def test_rows_outside_are_not_written(dq):  # noqa: F811
    new, kv = [3, 70], [30, 200]
    c = Scored(dq, 12, new, kv, 4, 2, 64, 16, "fp16")
    T = sum(new)
    q = torch.cat([c.q, c.q[:5]])
    out, lse = torch.full_like(q, 7.0), torch.full((T + 5, 4), 7.0, device="cuda")
    first = _i32(np.concatenate([np.zeros(T), np.full(5, 9)]))
    dq.kv_attention(c.cache, q, _i32(c.start), _i32(kv), _i32(c.table), max_q_len=70, softcap=20.0, first_pos=first, out=out,
                    lse=lse)
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (lse[T:] == 7).all() and not (out[:T] == 7).any()


def test_python_refusals(dq):  # noqa: F811
    c = Scored(dq, 13, [2, 1], [9, 4], 4, 2, 64, 16, "fp16")
    f32 = lambda n: torch.zeros(n, device="cuda")  # noqa: E731
    for kw in (dict(slopes=f32(3)), dict(slopes=f32(4).double()), dict(slopes=f32(4).cpu()), dict(prefix_len=f32(2)),
               dict(prefix_len=_i32([1])), dict(first_pos=_i32([0, 0])), dict(first_pos=_i32([0, 0, 0]).long()),
               dict(first_pos=_i32([0, 0, 0]).cpu())):
        with pytest.raises(ValueError):
            c.run(**kw)
    for cap in (-1.0, 1e-3, 1e7, float("nan"), float("inf")):
        with pytest.raises(dq.DqError):
            c.run(softcap=cap)


def test_one_graph_serves_other_masks(dq):  # noqa: F811
    c = Scored(dq, 14, [1] * 5, [300, 40, 900, 1, 77], 8, 2, 128, 16, "bf16")
    prefix, first = _i32([0] * 5), _i32([0] * 5)
    slopes = torch.tensor(steep(8)).cuda()
    dev = [_i32(x) for x in (c.start, c.kv, c.table)]
    ws = torch.empty(dq.kv_attention_workspace_size(c.cache, 8, 5, 5, 1), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(5, 8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    kw = dict(max_q_len=1, softcap=30.0, slopes=slopes, prefix_len=prefix, first_pos=first, out=out, lse=lse, ws=ws)
    with torch.cuda.stream(s):
        dq.kv_attention(c.cache, c.q, *dev, **kw)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            dq.kv_attention(c.cache, c.q, *dev, **kw)
    for a in ([5, 39, 899, 0, 70], [0, 3, 100, 0, 77]):
        first.copy_(_i32(a))
        g.replay()
        torch.cuda.synchronize()
        want, wl = c.call(softcap=30.0, slopes=steep(8), first_pos=a)
        assert torch.equal(out, want) and torch.equal(lse, wl)


GAPS = [([4, 9, 1], [50, 40, 7], 8, 2, 128), ([6], [700], 3, 3, 64), ([5, 8], [30, 600], 8, 1, 256),
        ([200, 90], [260, 400], 4, 2, 64), ([300], [1900], 2, 2, 128), ([150, 40], [900, 40], 4, 1, 256)]


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(softcap=300.0), dict(slopes=True),
                                dict(softcap=20.0, slopes=True), dict(prefix=True), dict(window=25)])
@pytest.mark.parametrize("new,kv,H,n_kv,D", GAPS)
def test_what_no_row_sees_may_hold_anything(dq, new, kv, H, n_kv, D, kw):  # noqa: F811
    # documents with rows between and behind them that see nothing, as padding does: their tokens hold NaN scales
    c = Scored(dq, 15, new, kv, H, n_kv, D, 16, "bf16")
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = steep(H)
    prefix = [k // 4 for k in kv] if kw.pop("prefix", False) else None
    first = []
    for n, L in zip(new, kv):
        at, far = max(L - n - 5, 0), 2 ** 31 - 1
        for i in range(n):
            third = i * 3 // n
            # the first third sees its document, the second one nothing up to the next one, the last rows nothing at all
            first.append(at if third == 0 else max(at, L - n + n * 2 // 3) if i < n - n // 5 else far)
    first = np.array(first)
    nan = np.frombuffer(np.float16(np.nan).tobytes(), dtype=np.uint8)
    lost = 0
    for r, (n, L) in enumerate(zip(new, kv)):
        f = first[int(c.start[r]):int(c.start[r + 1])]
        see = scores_ref.rows_see(n, L, True, kw.get("window", 0), 0 if prefix is None else prefix[r], f).any(0)
        for j in np.nonzero(~see)[0]:
            page, off = c.table[r, j // 16], j % 16
            for at in [kv_ref.k_scale(D, off, g) for g in range(D // 32)] + [kv_ref.v_scale(D, off, g) for g in range(D // 32)]:
                c.host[page, :, 0, at:at + 2] = nan
            lost += j >= L - n
    assert lost > 0
    c.cache.pages.copy_(torch.from_numpy(c.host).cuda().reshape(c.cache.pages.shape))
    if prefix is not None:
        kw["prefix_len"] = prefix
    c.call(exact=True, first_pos=first, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(softcap=300.0), dict(slopes=True), dict(softcap=2.0, slopes=True)])
@pytest.mark.parametrize("new,kv,H,n_kv,D", [([8], [500], 8, 2, 128), ([64, 70], [300, 900], 2, 2, 64), ([250], [1500], 4, 2, 128)])
def test_first_positions_that_descend_show_no_row_more(dq, new, kv, H, n_kv, D, kw):  # noqa: F811
    # out of contract, but a row still sees no position below its own: all V there is 100 times as large
    c = Scored(dq, 16, new, kv, H, n_kv, D, 16, "fp16")
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = [0.0] * H
    c.q.zero_()
    T, rng = sum(new), np.random.default_rng(3)
    for low in (200, 420):
        first = np.full(T, low)
        first[rng.permutation(T)[:T // 2]] = 5              # rows that may see what others may not
        first[int(c.start[-1]) - 1] = 5                     # (the last row among them)
        host = c.host.copy()
        for r, L in enumerate(kv):
            for j in range(L):
                for g in range(D // 32):
                    at = kv_ref.v_scale(D, j % 16, g)
                    host[c.table[r, j // 16], :, 0, at:at + 2] = np.frombuffer(
                        np.float16(64.0 if j < low else 2.0 ** -6).tobytes(), dtype=np.uint8)
        c.cache.pages.copy_(torch.from_numpy(host).cuda().reshape(c.cache.pages.shape))
        out, _ = c.run(max_q_len=max(new), first_pos=_i32(first), softcap=kw.get("softcap", 0.0),
                       slopes=None if "slopes" not in kw else torch.zeros(H, device="cuda"))
        torch.cuda.synchronize()
        assert dq.device_status() == 0
        assert out.float().abs().amax((1, 2)).cpu().numpy()[first == low].max() <= 8 * 2.0 ** -6
