"""The 4-bit K/V cache's kernels (dq_kv_plan, dq_kv_append, dq_kv_read,
dq_kv_attention) against their definitions in 64 bits (-m gpu).

Bars.  Plan: whole numbers, equal.  Append: the cache's bytes, equal for 16-bit
rows (their codes and scales have one right value); for fp32 rows a quotient
within 2^-20 of half-way may round to the neighbouring code, one step away.
Read: the fp32 values, equal.  Attention, per output element, with u the
rounding of the output type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32):
  |out - ref| <= u |ref| + w + (4 * 2^-11 + 2 E) sum_j p_j |v_j| + n 2^-33 max |v|,
  |lse - ref| <= E + 2^-18 (1 + |ref|),  E = 2^-11 max_j scale sum_d |q_d k_jd|:
E is what one fp16 rounding of an operand moves a score by (a weight p moves by
the factor e^E in the numerator and in the denominator, hence twice); a weight,
a V scale and their product are rounded to fp16 at most four times; below the
normal range these roundings are absolute: w = 2^-25 for an fp16 output, and
2^-25 for each of the n weights, held with the row's largest at 2^8 or more."""
import numpy as np
import pytest
import torch

import kv_ref

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import dequant_gemv_moe_gb300 as dq
    return dq


def bar_of(dtype, ref, mag, big, n, vmax):
    e = 2.0 ** -11 * big[..., None]
    w = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return U[dtype] * np.abs(ref) + w + (4 * 2.0 ** -11 + 2 * e) * mag + n * 2.0 ** -33 * vmax


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan
def _plan_case(rng, B, ps, width, kinds, spare, ctx_max=None):
    cap = min(width * ps, ctx_max or width * ps)
    ctx = rng.integers(0, cap + 1, B)
    new = np.array([{"one": 1, "none": 0, "gone": -1, "many": int(rng.integers(1, 3 * ps))}[kinds[rng.integers(len(kinds))]]
                    for _ in range(B)])
    have = -(-ctx // ps)
    total = int(have.sum()) + spare
    ids = rng.permutation(total)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for r in range(B):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    stack = np.full(total, -1, dtype=np.int32)
    stack[:spare] = ids[at:]
    return ctx.astype(np.int32), new.astype(np.int32), table, stack, spare


@pytest.mark.parametrize("seed,B,ps,width,kinds,spare,extra", [
    (1, 1, 16, 4, ["one"], 3, 0),
    (2, 1, 16, 1, ["many"], 8, 5),             # a row that cannot list what it needs
    (3, 48, 16, 9, ["one"], 64, 0),
    (4, 48, 32, 9, ["one", "none", "gone", "many"], 500, 7),
    (5, 48, 64, 9, ["one", "many", "gone"], 0, 0),     # every page that is popped was pushed by this call
    (6, 48, 16, 30, ["one", "many"], 11, 3),           # the stack runs out on the way
    (7, 1000, 128, 5, ["one", "none", "gone", "many"], 700, 0),
    (8, 1025, 16, 6, ["many"], 4000, 0),               # more than one round of the block's threads
    (9, 8192, 256, 3, ["one", "gone"], 1000, 100),
    (10, 5, 16, 300, ["gone"], 2, 4),                  # nothing but returns
])
def test_plan(dq, seed, B, ps, width, kinds, spare, extra):
    rng = np.random.default_rng(seed)
    ctx, new, table, stack, count = _plan_case(rng, B, ps, width, kinds, spare)
    T = int(np.maximum(new, 0).sum()) + extra
    ref = kv_ref.plan(ctx, new, table, stack.tolist(), count, ps, T)
    dt, ds = _i32(table), _i32(stack)
    args = (_i32(ctx), _i32(new), dt, ds, _i32([count]))
    out = dq.kv_plan(*args, page_size=ps, n_tokens=T)
    for again in range(2):                     # a repeated call repeats its results
        assert np.array_equal(dt.cpu().numpy(), ref["table"])
        assert np.array_equal(ds.cpu().numpy(), ref["stack"])
        assert out.kv_len.cpu().tolist() == ref["kv_len"]
        assert out.q_start.cpu().tolist() == ref["q_start"]
        assert out.slots.cpu().tolist() == ref["slots"]
        assert out.positions.cpu().tolist() == ref["positions"]
        assert out.free_count.item() == ref["free_count"]
        assert out.unserved.item() == ref["unserved"]
        out = dq.kv_plan(*args, page_size=ps, n_tokens=T, out=out)


def test_plan_with_fewer_rows_than_tokens(dq):
    rng = np.random.default_rng(5)
    ctx, new, table, stack, count = _plan_case(rng, 20, 16, 8, ["many", "one"], 300, ctx_max=60)
    T = int(new.sum()) - 9
    ref = kv_ref.plan(ctx, new, table, stack.tolist(), count, 16, T)
    out = dq.kv_plan(_i32(ctx), _i32(new), _i32(table), _i32(stack), _i32([count]), page_size=16, n_tokens=T)
    assert out.slots.cpu().tolist() == ref["slots"] and out.q_start.cpu().tolist() == ref["q_start"]


# ---------------------------------------------------------- append, read
def _rows(rng, T, H, D, dtype, wide):
    x = rng.standard_normal((T, H, D)) * np.exp(rng.uniform(-3, 3, (T, H, 1)))
    t = torch.tensor(x, dtype=torch.float32).to(DT[dtype])
    if wide:                                   # a slice of a fused projection's rows
        buf = torch.zeros(T, H + 3, D, dtype=DT[dtype])
        buf[:, 1:H + 1] = t
        return buf.cuda()[:, 1:H + 1], t.double().numpy()
    return t.cuda(), t.double().numpy()


@pytest.mark.parametrize("T,H,D,dtype,ps,wide", [
    (1, 1, 64, "fp16", 16, False), (1, 8, 128, "bf16", 16, False), (37, 5, 64, "fp32", 32, True),
    (130, 3, 128, "fp16", 64, True), (61, 2, 256, "bf16", 128, False), (33, 2, 256, "fp32", 256, True),
    (65, 1, 128, "fp32", 16, False),
])
def test_append_and_read(dq, T, H, D, dtype, ps, wide):
    rng = np.random.default_rng(T * 1000 + H)
    n_pages = -(-T // ps) + 4
    k, kr = _rows(rng, T, H, D, dtype, wide)
    v, vr = _rows(rng, T, H, D, dtype, wide)
    slots = rng.permutation(n_pages * ps)[:T].astype(np.int64)
    skip = rng.random(T) < 0.1
    slots[skip] = rng.choice([-1, n_pages * ps, 1 << 40], skip.sum())
    start = rng.integers(0, 256, (n_pages, H, ps // 16, 18 * D), dtype=np.uint8)
    buf = torch.from_numpy(start.copy()).cuda()
    cache = dq.KvCache(buf, ps, H, D)
    dq.kv_append(cache, k, v, torch.from_numpy(slots).cuda())
    got = buf.cpu().numpy()
    ref = start.copy()
    for t in range(T):
        if not skip[t]:
            for h in range(H):
                kv_ref.write(ref, ps, D, h, slots[t], kr[t, h], vr[t, h])
    if dtype != "fp32":
        assert np.array_equal(got, ref)
    else:
        # scales are equal; codes may differ by one where the quotient is that near to half-way
        assert np.array_equal(got[..., 16 * D:], ref[..., 16 * D:])
        a, b = got[..., :16 * D], ref[..., :16 * D]
        lo, hi = np.abs((a & 15).astype(int) - (b & 15)), np.abs((a >> 4).astype(int) - (b >> 4))
        assert max(lo.max(), hi.max()) <= 1 and (lo + hi).sum() <= 1 + 2 * T * H * D * 2.0 ** -16
    for to in ("fp32", "fp16", "bf16"):
        ko, vo = dq.kv_read(cache, torch.from_numpy(slots).cuda(), dtype=DT[to])
        for h in range(H):
            live = np.where(skip, 0, slots)
            want = [np.where(skip[:, None], 0.0, x) for x in kv_ref.read(got, ps, D, h, live)]
            for x, w in zip((ko, vo), want):
                w = torch.from_numpy(w).float()          # a value has at most 15 significant bits
                assert torch.equal(x[:, h].cpu(), w.to(DT[to]))


def test_append_extremes(dq):
    # zeros, subnormal and saturating magnitudes, ties of both signs, one value that is not zero
    D, ps = 64, 16
    x = np.zeros((8, 1, D))
    x[1] = 1e-7
    x[2, 0, 5], x[2, 0, 6] = 3.0, -3.0
    x[3, 0, 5], x[3, 0, 6] = -3.0, 3.0
    x[4] = 3.0e38
    x[5, 0, 40] = -65504.0
    x[6] = np.float64(np.float32(6e-8)) * np.arange(D)
    x[7] = (np.arange(D) - 31.5) / 4
    t = torch.tensor(x, dtype=torch.float32).cuda()
    buf = torch.zeros(1, 1, 1, 18 * D, dtype=torch.uint8, device="cuda")
    cache = dq.KvCache(buf, ps, 1, D)
    dq.kv_append(cache, t, t, torch.arange(8, device="cuda"))
    ref = np.zeros((1, 1, 1, 18 * D), dtype=np.uint8)
    for i in range(8):
        kv_ref.write(ref, ps, D, 0, i, t[i, 0].double().cpu().numpy(), t[i, 0].double().cpu().numpy())
    assert np.array_equal(buf.cpu().numpy()[0, 0, 0], ref[0, 0, 0])
    k, _ = dq.kv_read(cache, torch.arange(8, device="cuda"))
    assert torch.isfinite(k).all()


# ------------------------------------------------------------- attention
class Case:
    """A cache of random blocks whose unwritten places hold NaN scales, and a step's rows over it."""

    def __init__(self, dq, seed, new, kv, H, n_kv, D, ps, dtype, wide=False, skew=1.0, pages_before=0):
        rng = np.random.default_rng(seed)
        B = len(new)
        have = [-(-n // ps) for n in kv]
        used = sum(have) + 2
        width = max(max(have), 1) + 1
        ids = rng.permutation(used)
        self.table = np.full((B, width), -1, dtype=np.int32)
        cache = rng.integers(0, 256, (used, n_kv, ps // 16, 18 * D), dtype=np.uint8)
        # a scale that an append can write is at most 65504 / 8
        d = np.clip(rng.standard_normal((used, n_kv, ps // 16, D)) * 0.15 * skew, -8188, 8188).astype(np.float16)
        live = np.zeros((used, ps), dtype=bool)
        at = 0
        for r in range(B):
            for i in range(have[r]):
                self.table[r, i] = ids[at]
                live[ids[at], :min(ps, kv[r] - i * ps)] = True
                at += 1
        i16, g = np.arange(16), D // 32
        ks = np.array([[kv_ref.k_scale(D, i, x) for x in range(g)] for i in i16]) - 16 * D
        vs = np.array([[kv_ref.v_scale(D, i, x) for x in range(g)] for i in i16]) - 17 * D
        dead = ~live.reshape(used, 1, ps // 16, 16).repeat(n_kv, 1)
        dk, dv = d[..., :D // 2].copy(), d[..., D // 2:].copy()
        for s, x in ((ks, dk), (vs, dv)):
            for i in i16:
                x[..., s[i] // 2] = np.where(dead[..., i, None], np.float16(np.nan), x[..., s[i] // 2])
        cache[..., 16 * D:17 * D] = np.ascontiguousarray(dk).view(np.uint8)
        cache[..., 17 * D:] = np.ascontiguousarray(dv).view(np.uint8)
        self.host, self.ps, self.D, self.n_kv, self.H = cache, ps, D, n_kv, H
        self.new, self.kv = new, kv
        self.start = np.concatenate([[0], np.cumsum(new)])
        T = int(self.start[-1])
        q = torch.tensor(rng.standard_normal((T, H, D)) / max(skew, 1e-3), dtype=torch.float32).to(DT[dtype])
        self.q64 = q.double().numpy()
        if wide:
            buf = torch.zeros(T, H + 2 * n_kv, D, dtype=DT[dtype])
            buf[:, :H] = q
            self.q = buf.cuda()[:, :H]
        else:
            self.q = q.cuda()
        dev = torch.from_numpy(cache).cuda()
        self.cache = dq.KvCache(dev, ps, n_kv, D)
        self.dq, self.dtype = dq, DT[dtype]

    def run(self, **kw):
        return self.dq.kv_attention(self.cache, self.q, _i32(self.start), _i32(self.kv), _i32(self.table), **kw)

    def check(self, out, lse, scale=None, causal=True, window=0):
        scale = self.D ** -0.5 if scale is None else scale
        ref, rl, mag, big = kv_ref.attention(self.host, self.ps, self.D, self.q64, self.start, self.kv, self.table,
                                             scale, causal, window, self.n_kv)
        e = 2.0 ** -11 * big
        o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
        vs = np.abs(self.host[..., 17 * self.D:].view(np.float16).astype(np.float64))
        bar = bar_of(out.dtype, ref, mag, big, max(self.kv), 8 * np.nanmax(vs))
        assert np.isfinite(o).all()
        off = np.abs(o - ref)
        worst = np.max(np.where(off == 0, 0.0, off / np.where(bar == 0, 1e-300, bar)))
        assert worst <= 1, worst
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(l), none)
        assert (o[none] == 0).all()
        off = np.abs(np.where(none, 0, l) - np.where(none, 0, rl))
        assert (off <= e + 2.0 ** -18 * (1 + np.abs(np.where(none, 0, rl)))).all()


ATTN = [
    # new, kv, H, n_kv, D, ps, dtype, kwargs
    ([1], [1], 8, 8, 64, 16, "fp16", {}),
    ([1], [977], 32, 8, 128, 16, "bf16", {}),
    ([1] * 7, [1, 15, 16, 17, 63, 64, 65], 8, 2, 128, 16, "bf16", {}),
    ([1] * 5, [127, 128, 129, 255, 2000], 7, 1, 128, 64, "fp16", {}),
    ([1] * 3, [700, 0, 33], 8, 1, 256, 32, "bf16", {}),                  # a request with nothing cached
    ([1] * 4, [900, 31, 500, 64], 16, 1, 64, 128, "fp16", {}),           # 16 heads to a K/V head
    ([1, 0, 1], [300, 300, 257], 3, 1, 128, 256, "fp16", {}),            # a request without rows
    ([3, 1, 6, 2], [3, 1, 600, 129], 28, 4, 128, 32, "fp16", {}),
    ([5, 8], [40, 1000], 5, 5, 64, 16, "bf16", {}),
    ([4, 7], [2, 3], 8, 2, 128, 16, "fp16", {}),                         # rows before the cache's first token
    ([2] * 3, [400, 17, 1000], 8, 4, 256, 128, "fp16", dict(window=100)),
    ([1] * 3, [400, 17, 1000], 8, 8, 128, 16, "bf16", dict(window=1)),
    ([1] * 2, [1000, 640], 8, 1, 64, 16, "fp16", dict(window=64)),
    ([9, 3], [500, 3], 4, 2, 128, 16, "bf16", dict(causal=False)),
    ([1, 1], [77, 400], 4, 4, 128, 16, "fp16", dict(causal=False, window=50, scale=0.3)),
    ([130], [130], 4, 1, 128, 16, "bf16", {}),                           # prompts
    ([300, 1, 77], [300, 150, 77], 4, 4, 64, 64, "fp16", {}),
    ([257, 100], [700, 356], 8, 2, 128, 32, "fp16", {}),
    ([129, 64], [500, 64], 6, 2, 256, 16, "bf16", {}),
    ([200, 333], [90, 1000], 7, 1, 128, 128, "bf16", {}),                # rows that see nothing in a prompt
    ([260], [900], 8, 2, 128, 16, "fp16", dict(window=130)),
    ([150, 140], [400, 140], 4, 2, 64, 16, "bf16", dict(causal=False)),
    ([128, 256], [128, 512], 8, 8, 128, 128, "fp16", {}),
    ([31, 65, 1, 0, 500], [31, 800, 640, 20, 500], 8, 2, 128, 16, "bf16", {}),   # all kinds in one step
]


@pytest.mark.parametrize("i", range(len(ATTN)))
def test_attention(dq, i):
    new, kv, H, n_kv, D, ps, dtype, kw = ATTN[i]
    c = Case(dq, 100 + i, new, kv, H, n_kv, D, ps, dtype)
    out, lse = c.run(max_q_len=max(new), **kw)
    c.check(out, lse, **kw)
    assert dq.device_status() == 0
    again, lse2 = c.run(max_q_len=max(new), **kw)              # the same bits every time
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,kv", [([1] * 3, [300, 77, 500]), ([150, 40], [300, 40])])
@pytest.mark.parametrize("to", ["fp16", "bf16", "fp32"])
def test_attention_output_types_and_strides(dq, new, kv, to):
    c = Case(dq, 7, new, kv, 8, 2, 128, 16, "bf16", wide=True)
    T = sum(new)
    buf = torch.full((T, 11, 128), 7.0, dtype=DT[to], device="cuda")
    out, lse = c.run(out=buf[:, 2:10])
    c.check(out, lse)
    assert (buf[:, :2] == 7).all() and (buf[:, 10:] == 7).all()


@pytest.mark.parametrize("new,kv", [([1] * 3, [300, 77, 500]), ([150, 40], [300, 40])])
@pytest.mark.parametrize("skew", [2.0 ** -14, 2.0 ** -9, 64.0, 30000.0])
def test_attention_scale_regimes(dq, new, kv, skew):
    # K and V from far below 1 to the largest that the cache holds: no overflow, no lost weights
    c = Case(dq, 8, new, kv, 8, 2, 128, 16, "bf16", skew=skew)
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("new,kv", [([1] * 2, [900, 300]), ([140], [900])])
def test_attention_peaked_and_flat(dq, new, kv):
    for scale in (1e-6, 4.0):
        c = Case(dq, 9, new, kv, 8, 2, 128, 32, "fp16")
        out, lse = c.run(scale=scale)
        c.check(out, lse, scale=scale)


@pytest.mark.parametrize("new,kv", [([1] * 4, [900, 300, 5, 64]), ([140, 1], [400, 300])])
def test_attention_v_scales_that_grow_along_the_row(dq, new, kv):
    # V 2^14 times larger in the last tokens than in the first: sums held in any fixed 16-bit unit would lose them
    c = Case(dq, 10, new, kv, 8, 2, 128, 16, "fp16")
    vs = c.host[..., 17 * 128:].view(np.float16)
    for r, n in enumerate(kv):
        for i in range(-(-n // 16)):
            vs[c.table[r, i]] = (vs[c.table[r, i]].astype(np.float32) * 2.0 ** (14 * i / (n / 16) - 7)).astype(np.float16)
    c.cache.pages.copy_(torch.from_numpy(c.host))
    out, lse = c.run()
    c.check(out, lse)


@pytest.mark.parametrize("new,kv,H,n_kv,D", [
    ([1], [40000], 4, 1, 128),                     # one item over every CTA of the streaming kernel
    ([2, 1], [30011, 9000], 3, 1, 64),
    ([1], [20000], 8, 1, 256),
    ([70], [30000], 1, 1, 128),                    # and of the tensor-core kernel
    ([300, 20], [6000, 9000], 1, 1, 64),
    ([66], [9000], 2, 2, 256),
])
def test_attention_one_item_over_many_shares(dq, new, kv, H, n_kv, D):
    c = Case(dq, 20, new, kv, H, n_kv, D, 64, "fp16")
    out, lse = c.run(max_q_len=max(new))
    c.check(out, lse)


@pytest.mark.parametrize("longest", [20, 200, 900, 1500, 2500, 4500])
@pytest.mark.parametrize("B,H,n_kv,D,rows,window", [
    (1, 8, 2, 64, 1, 0), (3, 8, 8, 64, 1, 0), (1, 8, 2, 128, 1, 0), (5, 16, 4, 128, 2, 0), (7, 8, 8, 128, 1, 700),
    (2, 9, 3, 256, 3, 0), (6, 4, 4, 256, 1, 300),
])
def test_attention_few_row_tiles(dq, B, H, n_kv, D, rows, window, longest):
    # fewer row tiles than SMs: as the table's width and the window have it, each has a CTA, a cluster or shares;
    # requests shorter than the table, of no tokens and of no rows among them
    rng = np.random.default_rng(B * 1000 + longest)
    new = [int(n) for n in rng.integers(0, rows + 1, B)]
    kv = [int(n) for n in np.exp(rng.uniform(0, np.log(longest), B))]
    new[0], kv[0] = rows, longest
    if B > 2:
        kv[1], new[1] = 0, 1
        kv[2] = new[2] = rows
    c = Case(dq, 23, new, kv, H, n_kv, D, 32, "fp16")
    out, lse = c.run(max_q_len=rows, window=window)
    c.check(out, lse, window=window)
    again, _ = c.run(max_q_len=rows, window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("B,rows,most", [(1000, 1, 40), (600, 2, 300), (3000, 1, 20), (8192, 1, 3), (700, 70, 75)])
def test_attention_many_requests(dq, B, rows, most):
    # many short requests, more of them than a CTA has threads: shares hold many items, warps none or several
    rng = np.random.default_rng(B)
    new = [int(n) for n in rng.integers(0, rows + 1, B)]
    new[B // 2] = rows
    kv = [int(n) for n in rng.integers(0, most + 1, B)]
    c = Case(dq, 21, new, kv, 2, 1, 64, 16, "bf16")
    out, lse = c.run(max_q_len=rows)
    c.check(out, lse)
    again, _ = c.run(max_q_len=rows)
    assert torch.equal(out, again)


def test_attention_rows_above_max_q_len_are_not_written(dq):
    for most, new in ((2, [3, 2]), (70, [90, 65])):
        c = Case(dq, 22, new, [200, 300], 2, 2, 64, 16, "fp16")
        out = torch.full_like(c.q, 7.0)
        lse = torch.full((sum(new), 2), 7.0, device="cuda")
        c.run(max_q_len=most, out=out, lse=lse)
        torch.cuda.synchronize()
        rest = torch.arange(sum(new), device="cuda")
        keep = (rest < new[0]) & (rest >= most)
        assert (out[keep] == 7).all() and (lse[keep] == 7).all()
        assert not (out[~keep] == 7).all(-1).any()
        # request 1 has no row too many: its rows are right
        full, fl = c.run(max_q_len=max(new))
        assert torch.allclose(out[new[0]:].float(), full[new[0]:].float(), atol=2e-2)
        assert torch.allclose(lse[new[0]:], fl[new[0]:], atol=1e-3)


def test_attention_lse_of_few_tokens(dq):
    # where rows see few tokens their lse carries no rounding of K: within 2^-18 (1 + |lse|), as fp32 sums give it
    for new, kv, window in (([17] * 9, [17] * 9, 0), ([300], [300], 0), ([200], [4000], 100)):
        c = Case(dq, 23, new, kv, 10, 2, 128, 16, "bf16")
        out, lse = c.run(max_q_len=max(new), window=window)
        _, rl, _, _ = kv_ref.attention(c.host, 16, 128, c.q64, c.start, kv, c.table, 128 ** -0.5, True, window, 2)
        off = np.abs(lse.double().cpu().numpy() - rl)
        assert (off <= 2.0 ** -18 * (1 + np.abs(rl))).all(), off.max()


@pytest.mark.parametrize("new,kv", [([1] * 3, [900, 300, 5]), ([140, 1], [400, 300])])
def test_attention_scores_that_vanish(dq, new, kv):
    # a tiny scale on tiny rows: every visible token weighs the same, a masked one nothing
    c = Case(dq, 24, new, kv, 4, 2, 128, 16, "bf16")
    c.q = c.q * 2.0 ** -100
    c.q64 = c.q64 * 2.0 ** -100
    out, lse = c.run(max_q_len=max(new), scale=1e-25)
    c.check(out, lse, scale=1e-25)


def test_attention_rows_outside_are_not_written(dq):
    c = Case(dq, 11, [2, 3], [50, 70], 8, 2, 128, 16, "fp16")
    q = torch.cat([c.q, torch.full((4, 8, 128), float("nan"), dtype=c.q.dtype, device="cuda")])
    out = torch.full((9, 8, 128), 7.0, dtype=c.q.dtype, device="cuda")
    lse = torch.full((9, 8), 7.0, device="cuda")
    dq.kv_attention(c.cache, q, _i32(c.start), _i32(c.kv), _i32(c.table), out=out, lse=lse, max_q_len=3)
    c.check(out[:5], lse[:5])
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()


@pytest.mark.parametrize("new,kv", [([1, 2], [300, 1000]), ([150], [500])])
def test_attention_past_32_bit_offsets(dq, new, kv):
    # the pages in use lie more than 4 GiB into the cache
    c = Case(dq, 12, new, kv, 8, 2, 128, 64, "bf16")
    page = c.host[0].nbytes
    before = (5 << 30) // page
    buf = torch.empty((before + len(c.host)) * page, dtype=torch.uint8, device="cuda")
    buf[before * page:] = torch.from_numpy(c.host).reshape(-1).cuda()
    c.cache = dq.KvCache(buf, 64, 2, 128)
    table, c.table = c.table, np.where(c.table >= 0, c.table + before, -1)
    out, lse = c.run()
    c.table = table
    c.check(out, lse)
    # and the append and the read there
    k = torch.randn(3, 2, 128, device="cuda").half()
    slots = torch.tensor([(before + 1) * 64 + 5, (before + 2) * 64 - 1, (before + len(c.host)) * 64 - 1], device="cuda")
    dq.kv_append(c.cache, k, k, slots)
    got, _ = dq.kv_read(c.cache, slots)
    code, d = kv_ref.quantise(k.double().cpu().numpy())
    want = (code.reshape(3, 2, 4, 32) - 8) * d[..., None]
    assert np.array_equal(got.double().cpu().numpy().reshape(want.shape), want)


def test_one_graph_serves_every_length(dq):
    # plan, append and attention of a decode step captured once; lengths, rows and slots change between replays
    B, H, n_kv, D, ps, width = 6, 8, 2, 128, 16, 12
    rng = np.random.default_rng(3)
    ctx0 = np.array([0, 15, 16, 40, 100, 3])
    have = -(-ctx0 // ps)
    n_pages = B * width
    ids = rng.permutation(n_pages)
    table = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for r in range(B):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    stack = np.concatenate([ids[at:], np.full(at, -1)]).astype(np.int32)
    cache = dq.KvCache.empty(n_pages, ps, n_kv, D)
    cache.pages.fill_(255)
    dtab, dst = _i32(table), _i32(stack)
    lens = [_i32(ctx0), torch.empty(B, dtype=torch.int32, device="cuda")]
    cnt = [_i32([n_pages - at]), torch.empty(1, dtype=torch.int32, device="cuda")]
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    k = torch.zeros(B, n_kv, D, dtype=torch.bfloat16, device="cuda")
    v, q = torch.zeros_like(k), torch.zeros(B, H, D, dtype=torch.bfloat16, device="cuda")
    # what is cached already
    hist = {r: (rng.standard_normal((ctx0[r], n_kv, D)), rng.standard_normal((ctx0[r], n_kv, D))) for r in range(B)}
    for r in range(B):
        if ctx0[r]:
            j = np.arange(ctx0[r])
            s = torch.from_numpy(table[r, j // ps].astype(np.int64) * ps + j % ps).cuda()
            a, b = (torch.tensor(x, dtype=torch.bfloat16).cuda() for x in hist[r])
            dq.kv_append(cache, a, b, s)
    plan = dq.kv_plan(lens[0], one, dtab.clone(), dst.clone(), cnt[0], page_size=ps, n_tokens=B)
    ws = torch.empty(dq.kv_attention_workspace_size(cache, H, B, B, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    lse = torch.empty(B, H, device="cuda")

    def step():
        dq.kv_plan(lens[0], one, dtab, dst, cnt[0], page_size=ps, n_tokens=B, out=plan)
        dq.kv_append(cache, k, v, plan.slots)
        dq.kv_attention(cache, q, plan.q_start, plan.kv_len, dtab, max_q_len=1, out=out, lse=lse, ws=ws)
        lens[0].copy_(plan.kv_len)
        cnt[0].copy_(plan.free_count)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for it in range(40):
        for t in (k, v, q):
            t.copy_(torch.tensor(rng.standard_normal(t.shape), dtype=torch.float32))
        g.replay()
        torch.cuda.synchronize()
        kv = (ctx0 + it + 1).tolist()
        assert lens[0].cpu().tolist() == kv and plan.unserved.item() == 0
        host = cache.pages.cpu().numpy().reshape(n_pages, n_kv, ps // 16, 18 * D)
        tab = dtab.cpu().numpy()
        ref, rl, mag, big = kv_ref.attention(host, ps, D, q.double().cpu().numpy(), np.arange(B + 1), kv, tab, D ** -0.5,
                                             True, 0, n_kv)
        bar = bar_of(out.dtype, ref, mag, big, max(kv), 8.0)
        assert (np.abs(out.double().cpu().numpy() - ref) <= bar).all()
    live = np.concatenate([tab[r, :-(-kv[r] // ps)] for r in range(B)])
    assert len(set(live.tolist())) == len(live)                # no page has two owners
    assert dq.device_status() == 0


def test_on_another_stream(dq):
    c = Case(dq, 13, [1, 1], [500, 70], 8, 2, 128, 16, "fp16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse = c.run()
    s.synchronize()
    c.check(out, lse)


def test_python_refusals(dq):
    c = Case(dq, 14, [1], [20], 4, 2, 64, 16, "fp16")
    with pytest.raises(ValueError):
        dq.KvCache(torch.empty(1000, dtype=torch.uint8, device="cuda"), 16, 2, 64)
    with pytest.raises(ValueError):
        dq.kv_append(c.cache, c.q, c.q, torch.zeros(1, dtype=torch.int64, device="cuda"))     # four heads, not two
    with pytest.raises(ValueError):
        dq.kv_attention(c.cache, c.q, _i32(c.start).long(), _i32(c.kv), _i32(c.table))
    with pytest.raises(dq.DqError):
        dq.kv_attention(c.cache, c.q.float(), _i32(c.start), _i32(c.kv), _i32(c.table))
    with pytest.raises(dq.DqError):
        c.run(ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
