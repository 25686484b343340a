"""dq_kv_append_rope against the rotation and the Q4_0 rounding in 64 bits: what the cache holds equal, q's rows within
the rounding of fp32 and of their type."""
import numpy as np
import pytest
import torch

import kv_ref
import rope_ref

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
# half a step, relative; fp16's subnormals absolute
HALF = {"fp32": (2.0 ** -24, 0.0), "fp16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 0.0)}
# of |a| + |b|: cos and sin (2.3e-7 together with the factor's product), a product and a sum of 2^-24 each
ROT = 4e-7
ROT_FAR = 2e-6            # positions from 2^24 on: turns of 2^-53 of up to 3.4e8, and the 64-bit angle's own rounding


@pytest.fixture(scope="module")
def dq():
    import dequant_gemv_moe_gb300 as m
    return m


def data(T, heads, kv_heads, D, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, heads + 2 * kv_heads, D, generator=g) * spread
    x[:, :, ::17] *= 4.0
    x = x.to(DT[dtype]).cuda()
    return x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]


def quantise32(x):
    """v's blocks by dq_kv_append's formula, whose quotient and sum are fp32."""
    g = np.clip(x.astype(np.float32), -65504, 65504).reshape(*x.shape[:-1], -1, 32)
    m = np.take_along_axis(g, np.argmax(np.abs(g), -1)[..., None], -1)
    d = (m / np.float32(-8)).astype(np.float16).astype(np.float32)
    q = np.floor(g / np.where(d == 0, np.float32(1), d) + np.float32(8.5))
    c = np.where(d == 0, 8, np.clip(q, 0, 15)).astype(np.int64)
    return c.reshape(x.shape), d[..., 0].astype(np.float64)


def run(dq, q, k, v, pos, freq, page=16, interleaved=False, factor=1.0, slots=None, out_dtype=None, out=None):
    T, hk, D = k.shape
    n_pages = -(-T // page) + 2
    cache = dq.KvCache(torch.full((dq.KvCache.size(n_pages, page, hk, D),), 0x5A, dtype=torch.uint8, device="cuda"),
                       page, hk, D)
    before = cache.pages.clone()
    if slots is None:
        perm = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(T))[:T]
        slots = perm.cuda()
    p = torch.as_tensor(np.asarray(pos, dtype=np.int32)).cuda()
    f = torch.as_tensor(freq).cuda()
    got = dq.kv_append_rope(cache, q, k, v, slots, p, f, interleaved=interleaved, factor=factor, out=out,
                            out_dtype=out_dtype)
    torch.cuda.synchronize()
    sl, pn = slots.cpu().numpy(), np.asarray(pos)
    live = (pn >= 0) & (sl >= 0) & (sl < n_pages * page)
    kf, vf = k.float().cpu().numpy(), v.float().cpu().numpy()
    kr, _ = rope_ref.rotate(kf, np.maximum(pn, 0), freq, interleaved, factor)
    pages = cache.pages.cpu().numpy().reshape(n_pages, hk, page // 16, 18 * D)
    want_cache = before.cpu().numpy().reshape(pages.shape)
    kc, kd = rope_ref.quantise(kr)
    vc, vd = quantise32(vf)
    wk = (kd[..., None] * (kc.reshape(T, hk, -1, 32) - 8)).reshape(T, hk, D)
    wv = (vd[..., None] * (vc.reshape(T, hk, -1, 32) - 8)).reshape(T, hk, D)
    for h in range(hk):
        gk, gv = kv_ref.read(pages, page, D, h, sl[live])
        np.testing.assert_array_equal(gk, wk[live, h])
        np.testing.assert_array_equal(gv, wv[live, h])
    # what no token was given stays as it was
    idle = np.setdiff1d(np.arange(n_pages * page), sl[live])
    for h in range(hk):
        for a, b in zip(kv_ref.read(pages, page, D, h, idle), kv_ref.read(want_cache, page, D, h, idle)):
            np.testing.assert_array_equal(a, b)
    if q is not None:
        return got, pn
    assert got is None


def check_q(got, q, pn, freq, interleaved=False, factor=1.0, name=None):
    qf = q.float().cpu().numpy()
    want, size = rope_ref.rotate(qf, np.maximum(pn, 0), freq, interleaved, factor)
    rel, ab = HALF[name]
    rot = np.where(pn >= 1 << 24, ROT_FAR, ROT)[:, None, None]
    diff = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    ok = diff <= rot * size * (1 + rel) + rel * np.abs(want) + ab
    live = pn >= 0
    assert ok[live].all(), diff[live].max()


CASES = [(1, 1, 1, 64, 64, False), (1, 32, 8, 128, 128, False), (3, 5, 5, 64, 32, True), (5, 4, 1, 256, 256, False),
         (37, 6, 2, 128, 64, False), (37, 6, 3, 128, 96, True), (64, 8, 8, 256, 64, True), (200, 7, 1, 128, 16, False),
         (33, 16, 2, 64, 48, False), (601, 3, 1, 256, 64, False), (1203, 2, 3, 64, 48, True), (2402, 1, 1, 128, 128, False),
         (1025, 3, 1, 128, 128, False), (1026, 2, 2, 64, 64, True), (1030, 4, 2, 256, 112, False)]


@pytest.mark.parametrize("T,H,HK,D,R,inter", CASES)
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
def test_rows(dq, T, H, HK, D, R, inter, dtype):
    freq = rope_ref.frequencies(R, 500000.0 if D == 128 else 10000.0)
    r = np.random.default_rng(T + D)
    pos = r.integers(0, 131072, T)
    pos[: min(T, 3)] = [0, 1, 1000000][: min(T, 3)]
    q, k, v = data(T, H, HK, D, dtype, T + R)
    got, pn = run(dq, q, k, v, pos, freq, page=[16, 32, 64, 128, 256][T % 5], interleaved=inter)
    assert got.dtype == DT[dtype]
    check_q(got, q, pn, freq, inter, name=dtype)


@pytest.mark.parametrize("inter", [False, True])
def test_many_rows_hold_the_codes_of_64_bits(dq, inter):
    # 2 million K values: some hundred lie closer to a border than fp32 can tell
    T, D = 2000, 128
    freq = rope_ref.frequencies(D)
    for dtype, seed in (("bf16", 1), ("fp32", 2), ("fp16", 3)):
        q, k, v = data(T, 1, 8, D, dtype, seed)
        run(dq, None, k, v, np.arange(T) * 37 % 20011, freq, page=64, interleaved=inter)


def test_borders(dq):
    # rows of few different magnitudes: equal ones of both signs, quotients on borders, scales between two fp16
    T, D = 300, 64
    r = np.random.default_rng(5)
    k = torch.tensor(r.integers(-4, 5, (T, 4, D)).astype(np.float32) * 0.25)
    k[10:20] = 0.0
    k[20:30] = 1.0
    k[30:40, :, ::2] = -1.0
    k[40:50] *= 1e-7
    k[50:60] *= 2.0 ** 16
    v = k.flip(0).contiguous()
    freq = rope_ref.frequencies(D)
    for R in (64, 32):
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            kk, vv = k.to(dtype).clamp(-60000, 60000).cuda(), v.to(dtype).clamp(-60000, 60000).cuda()
            for pos in (np.zeros(T, dtype=int), np.arange(T)):
                run(dq, None, kk, vv, pos, freq[: R // 2])
    # a quarter turn: the pair changes places, nearly, and zeros meet values
    quarter = np.full(32, np.pi / 2, dtype=np.float32)
    run(dq, None, k.cuda(), v.cuda(), np.arange(T) % 9, quarter / 2)
    # values beyond fp16
    big = (k * 3e5).cuda()
    run(dq, None, big, big, np.arange(T), freq)


def test_positions_far_and_left_out(dq):
    T, D, R = 24, 128, 128
    freq = rope_ref.frequencies(R)
    pos = np.array([-1, 0, 5, (1 << 24) - 1, 1 << 24, (1 << 31) - 1, 999999937, -5] * 3)
    q, k, v = data(T, 4, 2, D, "fp32", 9)
    slots = torch.arange(T).cuda()
    slots[3] = -1
    slots[10] = 1 << 40
    out = torch.full((T, 4, D), -3.0, device="cuda")
    got, pn = run(dq, q, k, v, pos, freq, slots=slots, out=out)
    check_q(got, q, pn, freq, name="fp32")
    assert (got[torch.tensor(pos < 0).cuda()] == -3.0).all()


def test_factor_types_strides_and_in_place(dq):
    T, D = 19, 128
    freq = rope_ref.frequencies(D)
    pos = np.arange(T) * 1000
    for dtype, to in (("fp32", "bf16"), ("fp32", "fp16"), ("bf16", "fp32"), ("fp16", "bf16")):
        q, k, v = data(T, 6, 2, D, dtype, 4)
        got, pn = run(dq, q, k, v, pos, freq, factor=1.25, out_dtype=DT[to])
        check_q(got, q, pn, freq, factor=1.25, name=to)
    q, k, v = data(T, 6, 2, D, "bf16", 4)
    wide = torch.full((T, 10, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, pn = run(dq, q, k, v, pos, freq, out=wide[:, 2:8])
    check_q(got, q, pn, freq, name="bf16")
    assert (wide[:, :2] == 7).all() and (wide[:, 8:] == 7).all()
    mine = q.clone()
    want = got.clone()
    run(dq, mine, k, v, pos, freq, out=mine)
    assert torch.equal(mine, want)
    # q as a slice of the projection, in place
    x = torch.cat([q, k, v], 1).contiguous()
    run(dq, x[:, :6], x[:, 6:8], x[:, 8:], pos, freq, out=x[:, :6])
    assert torch.equal(x[:, :6], want) and torch.equal(x[:, 6:8], k) and torch.equal(x[:, 8:], v)


def test_python_refusals(dq):
    T, D = 4, 64
    q, k, v = data(T, 2, 1, D, "bf16", 1)
    cache = dq.KvCache.empty(4, 16, 1, D)
    slots, pos = torch.arange(T).cuda(), torch.arange(T, dtype=torch.int32).cuda()
    f = torch.ones(32, device="cuda")
    bad = [dict(q=q.float()), dict(q=q[:2]), dict(k=k.float()), dict(v=v[:2]), dict(pos=pos.long()), dict(pos=pos[:2]),
           dict(slots=slots.int()), dict(f=f.double()), dict(f=f.cpu()), dict(out=q[:, :1].contiguous()),
           dict(q=q.transpose(1, 2)), dict(q=None, out=q.contiguous()), dict(q=q.cpu())]
    for kw in bad:
        a = {**dict(q=q, k=k, v=v, slots=slots, pos=pos, f=f, out=None), **kw}
        with pytest.raises(ValueError):
            dq.kv_append_rope(cache, a["q"], a["k"], a["v"], a["slots"], a["pos"], a["f"], out=a["out"])
    for n in (33, 4, 0):
        with pytest.raises(dq.DqError):
            dq.kv_append_rope(cache, q, k, v, slots, pos, torch.ones(n, device="cuda"))
    assert dq.kv_append_rope(cache, q[:0], k[:0], v[:0], slots[:0], pos[:0], f).shape == (0, 2, D)


def test_captured(dq):
    T, D = 8, 128
    freq = rope_ref.frequencies(D)
    q, k, v = (t.contiguous() for t in data(T, 4, 2, D, "bf16", 6))
    cache = dq.KvCache.empty(2, 16, 2, D)
    slots, pos = torch.arange(T).cuda(), torch.zeros(T, dtype=torch.int32).cuda()
    f = torch.tensor(freq).cuda()
    out = torch.empty_like(q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dq.kv_append_rope(cache, q, k, v, slots, pos, f, out=out)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            dq.kv_append_rope(cache, q, k, v, slots, pos, f, out=out)
    for at in (3, 70000):
        pos.fill_(at)
        g.replay()
        torch.cuda.synchronize()
        check_q(out, q, np.full(T, at), freq, name="bf16")
        kr, _ = rope_ref.rotate(k.float().cpu().numpy(), np.full(T, at), freq)
        c, d = rope_ref.quantise(kr)
        want = (d[..., None] * (c.reshape(T, 2, -1, 32) - 8)).reshape(T, 2, D)
        np.testing.assert_array_equal(dq.kv_read(cache, slots)[0].cpu().numpy(), want)
