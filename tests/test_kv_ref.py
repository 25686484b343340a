"""The plain 4-bit K/V cache definitions the GPU tests compare with, held to
independent facts; and the entry points' refusals, which launch nothing (CPU)."""
import ctypes
import os

import numpy as np
import pytest

import kv_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_layout_covers_every_bit_once(D):
    # 16 tokens x D codes of K and V in 16 D bytes, then 2 D bytes of scales: no overlap, no gap
    seen = np.zeros(18 * D * 2, dtype=int)                   # half-bytes
    for code in (kv_ref.k_code, kv_ref.v_code):
        for i in range(16):
            for x in range(D):
                b, s = code(D, i, x)
                seen[2 * b + s // 4] += 1
    for scale in (kv_ref.k_scale, kv_ref.v_scale):
        for i in range(16):
            for g in range(D // 32):
                b = scale(D, i, g)
                assert b % 2 == 0
                seen[2 * b:2 * b + 4] += 1
    assert (seen == 1).all()


def test_quantise_is_q4_0():
    # hand-made groups: the largest magnitude becomes code 0, halves round up, ties take the first value
    x = np.zeros(32)
    x[3], x[9] = -8.0, 8.0                                   # tie: the first, -8, sets d = 1
    x[10], x[11], x[12] = 0.5, -0.5, 7.4
    c, d = kv_ref.quantise(x)
    assert d[0] == 1.0
    assert (c[3], c[9], c[10], c[11], c[12], c[0]) == (0, 15, 9, 8, 15, 8)
    x[3] = 8.0                                               # the first is +8 now: d = -1, the signs turn
    c, d = kv_ref.quantise(x)
    assert d[0] == -1.0 and (c[3], c[9], c[12]) == (0, 0, 1)
    c, d = kv_ref.quantise(np.zeros(32))
    assert d[0] == 0 and (c == 8).all()
    c, d = kv_ref.quantise(np.full(32, 1e6))                 # saturates
    assert d[0] == -8188.0 and (c == 0).all()


def test_quantise_error_bound():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((200, 128))
    c, d = kv_ref.quantise(x)
    y = (c.reshape(200, 4, 32) - 8) * d[..., None]
    err = np.abs(y - x.reshape(200, 4, 32))
    # half a step, a whole one at the end the codes do not reach (+8 d), and the scale's rounding (8 d 2^-11)
    assert (err <= np.abs(d)[..., None] * (1.0 + 2.0 ** -8)).all()
    assert np.sqrt((err ** 2).mean()) < 0.1


@pytest.mark.parametrize("D", [64, 256])
def test_write_then_read(D):
    rng = np.random.default_rng(D)
    cache = rng.integers(0, 256, (2, 3, 2, 18 * D), dtype=np.uint8)
    k, v = rng.standard_normal(D), rng.standard_normal(D)
    before = cache.copy()
    kv_ref.write(cache, 32, D, 1, 32 + 21, k, v)
    got = kv_ref.read(cache, 32, D, 1, [32 + 21])
    for x, y in zip((k, v), got):
        c, d = kv_ref.quantise(x)
        assert np.array_equal(y[0], ((c.reshape(-1, 32) - 8) * d[:, None]).reshape(-1))
    changed = np.argwhere(before != cache)
    assert (changed[:, 0] == 1).all() and (changed[:, 1] == 1).all() and (changed[:, 2] == 1).all()


def test_plan_by_hand():
    table = np.array([[5, 7, -1, -1], [2, -1, -1, -1], [9, 8, -1, -1]])
    got = kv_ref.plan([17, 16, 20], [15, 1, -1], table, [1, 3, -1, -1], 2, 16, 20)
    # request 2 returns 9, 8 on top of 1, 3; request 0 fills its second page; request 1 takes 8
    assert got["table"].tolist() == [[5, 7, -1, -1], [2, 8, -1, -1], [9, 8, -1, -1]]
    assert got["stack"].tolist() == [1, 3, 9, 8] and got["free_count"] == 3
    assert got["kv_len"] == [32, 17, 0] and got["q_start"] == [0, 15, 16, 16]
    assert got["slots"][:2] == [7 * 16 + 1, 7 * 16 + 2] and got["slots"][15] == 8 * 16
    assert got["slots"][16:] == [-1] * 4 and got["positions"][15] == 16


def test_attention_by_hand():
    # two tokens, one head: out = the softmax-weighted mean of the two V rows
    D = 64
    cache = np.zeros((1, 1, 1, 18 * D), dtype=np.uint8)
    k = np.zeros((2, D))
    k[0, 0], k[1, 0] = -8.0, -4.0
    v = np.stack([np.full(D, -8.0), np.full(D, -16.0)])
    for t in range(2):
        kv_ref.write(cache, 16, D, 0, t, k[t], v[t])
    q = np.zeros((1, 1, D))
    q[0, 0, 0] = 0.25
    out, lse, _, _ = kv_ref.attention(cache, 16, D, q, [0, 1], [2], np.array([[0]]), 1.0, True, 0, 1)
    w = np.exp([-2.0, -1.0])
    assert np.allclose(out[0, 0], (w[0] * -8 + w[1] * -16) / w.sum())
    assert np.isclose(lse[0, 0], np.log(w.sum()))
    out, lse, _, _ = kv_ref.attention(cache, 16, D, q, [0, 1], [0], np.array([[0]]), 1.0, True, 0, 1)
    assert (out == 0).all() and lse[0, 0] == -np.inf


# ------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def so():
    import importlib.util
    path = os.path.join(ROOT, "dequant_gemv_moe_gb300", "build.py")
    spec = importlib.util.spec_from_file_location("_dqmoe_build", path)
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    b.build()
    import dequant_gemv_moe_gb300 as dq
    return dq._lib


ARG, ALIGN, UNSUP, WS = -1, -2, -3, -4
A = 4096                      # fake, aligned; never dereferenced on the error paths


def _desc(so, **kw):
    d = dict(fmt=4, n_kv_heads=8, head_dim=128, page_size=16, n_pages=10, pages=A)
    d.update(kw)
    return so.KvCacheDesc(**d)


def test_cache_size_and_refusals(so):
    n = ctypes.c_size_t()
    f = so.lib.dq_kv_cache_size
    assert f(ctypes.byref(_desc(so)), ctypes.byref(n)) == 0 and n.value == 10 * 8 * 18 * 128
    assert f(ctypes.byref(_desc(so, page_size=64, head_dim=64)), ctypes.byref(n)) == 0
    assert n.value == 10 * 8 * 4 * 18 * 64
    # 9,000,000 pages: the size passes 32 bits
    assert f(ctypes.byref(_desc(so, n_pages=9000000)), ctypes.byref(n)) == 0
    assert n.value == 9000000 * 8 * 18 * 128
    for kw, rc in [(dict(fmt=0), ARG), (dict(fmt=9), ARG), (dict(fmt=6), UNSUP), (dict(head_dim=96), UNSUP),
                   (dict(head_dim=0), ARG), (dict(page_size=24), ARG), (dict(page_size=8), ARG),
                   (dict(page_size=512), ARG), (dict(n_pages=0), ARG), (dict(n_kv_heads=0), ARG),
                   (dict(n_kv_heads=1025), UNSUP)]:
        assert f(ctypes.byref(_desc(so, **kw)), ctypes.byref(n)) == rc, kw
    assert f(None, ctypes.byref(n)) == ARG
    assert f(ctypes.byref(_desc(so)), None) == ARG


PLAN = dict(ctx=A, new=A, B=4, ps=16, table=A, width=8, stack=A, n_pages=64, count=A, T=4, kv=2 * A, start=A, slots=A,
            pos=A, left=2 * A, missed=A)


@pytest.mark.parametrize("change,rc", [
    (dict(ctx=None), ARG), (dict(new=None), ARG), (dict(table=None), ARG), (dict(stack=None), ARG),
    (dict(count=None), ARG), (dict(kv=None), ARG), (dict(start=None), ARG), (dict(slots=None), ARG),
    (dict(pos=None), ARG), (dict(left=None), ARG), (dict(missed=None), ARG), (dict(B=0), ARG), (dict(T=-1), ARG),
    (dict(ps=17), ARG), (dict(width=0), ARG), (dict(n_pages=0), ARG), (dict(width=1 << 27), ARG), (dict(kv=A), ARG),
    (dict(left=A), ARG), (dict(B=8193), UNSUP), (dict(slots=A + 4), ALIGN), (dict(ctx=A + 2), ALIGN),
    (dict(missed=A + 1), ALIGN),
])
def test_plan_refusals(so, change, rc):
    a = dict(PLAN)
    a.update(change)
    assert so.lib.dq_kv_plan(*a.values(), None) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(T=0), ARG), (dict(dt=3), ARG),
    (dict(ks=1023), ARG), (dict(vs=0), ARG), (dict(k=A + 8), ALIGN), (dict(ks=1028), ALIGN), (dict(vs=1026), ALIGN),
    (dict(slots=A + 4), ALIGN), (dict(desc=dict(pages=None)), ARG), (dict(desc=dict(pages=A + 64)), ALIGN),
    (dict(desc=dict(fmt=1)), UNSUP),
])
def test_append_refusals(so, change, rc):
    a = dict(desc={}, k=A, ks=1024, v=A, vs=1024, dt=1, slots=A, T=3)
    a.update(change)
    a["desc"] = ctypes.byref(_desc(so, **a["desc"]))
    assert so.lib.dq_kv_append(*a.values(), None) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(k=None), ARG), (dict(v=None), ARG), (dict(slots=None), ARG), (dict(T=0), ARG), (dict(dt=-1), ARG),
    (dict(v=A + 4), ALIGN), (dict(slots=A + 2), ALIGN), (dict(desc=dict(pages=None)), ARG),
])
def test_read_refusals(so, change, rc):
    a = dict(desc={}, slots=A, T=3, k=A, v=A, dt=0)
    a.update(change)
    a["desc"] = ctypes.byref(_desc(so, **a["desc"]))
    assert so.lib.dq_kv_read(*a.values(), None) == rc


@pytest.mark.parametrize("change,rc", [
    (dict(q=None), ARG), (dict(q_start=None), ARG), (dict(kv_len=None), ARG), (dict(block_table=None), ARG),
    (dict(out=None), ARG), (dict(T=0), ARG), (dict(B=0), ARG), (dict(n_q_heads=0), ARG), (dict(n_q_heads=12), ARG),
    (dict(max_q_len=0), ARG), (dict(max_q_len=6), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(causal=2), ARG), (dict(window=-1), ARG),
    (dict(q_dtype=3), ARG), (dict(out_dtype=-1), ARG), (dict(max_pages=0), ARG), (dict(q_stride=4088), ARG),
    (dict(out_stride=1), ARG), (dict(q_dtype=0), UNSUP), (dict(n_q_heads=4104, q_stride=1 << 20, out_stride=1 << 20), UNSUP),
    (dict(B=8193), UNSUP), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN), (dict(q_stride=4100), ALIGN),
    (dict(lse=A + 2), ALIGN), (dict(kv_len=A + 1), ALIGN),
])
def test_attention_refusals(so, change, rc):
    a = dict(q=A, q_stride=4096, q_dtype=1, n_q_heads=32, T=5, B=3, q_start=A, kv_len=A, block_table=A, max_pages=9,
             max_q_len=3, scale=0.1, causal=1, window=0, out=A, out_stride=4096, out_dtype=1, lse=A)
    a.update(change)
    f = so.lib.dq_kv_attention
    assert f(ctypes.byref(_desc(so)), ctypes.byref(so.KvAttn(**a)), A, 1 << 40, None) == rc


def test_attention_workspace_refusals(so):
    a = so.KvAttn(q=A, q_stride=4096, q_dtype=1, n_q_heads=32, T=5, B=3, q_start=A, kv_len=A, block_table=A,
                  max_pages=9, max_q_len=3, scale=0.1, causal=1, window=0, out=A, out_stride=4096, out_dtype=1, lse=A)
    d = ctypes.byref(_desc(so))
    f = so.lib.dq_kv_attention
    assert f(d, ctypes.byref(a), None, 1 << 40, None) == WS
    assert f(d, ctypes.byref(a), A, 0, None) == WS
    assert f(d, ctypes.byref(a), A + 128, 1 << 40, None) == ALIGN
    assert f(d, None, A, 1 << 40, None) == ARG
    n = ctypes.c_size_t()
    g = so.lib.dq_kv_attention_workspace_size
    assert g(d, 32, 5, 3, 3, ctypes.byref(n)) == 0 and n.value > 0
    assert g(d, 32, 5, 3, 3, None) == ARG
    assert g(d, 31, 5, 3, 3, ctypes.byref(n)) == ARG
    assert g(d, 32, 5, 3, 6, ctypes.byref(n)) == ARG
