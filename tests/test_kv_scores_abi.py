"""dq_kv_attention_ex's argument checks (before any launch), the 64-bit reference of its scores and masks by hand, and
the polynomial of its cap against tanh."""
import ctypes
import os
import re

import numpy as np
import pytest

import scores_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Cache(ctypes.Structure):
    _fields_ = [("fmt", I32), ("n_kv_heads", I32), ("head_dim", I32), ("page_size", I32), ("n_pages", I32), ("pages", P)]


class Attn(ctypes.Structure):
    _fields_ = [("q", P), ("q_stride", I64), ("q_dtype", I32), ("n_q_heads", I32), ("T", I32), ("B", I32), ("q_start", P),
                ("kv_len", P), ("block_table", P), ("max_pages", I32), ("max_q_len", I32), ("scale", ctypes.c_float),
                ("causal", I32), ("window", I32), ("out", P), ("out_stride", I64), ("out_dtype", I32), ("lse", P)]


class Scores(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("slopes", P), ("prefix_len", P), ("first_pos", P)]


@pytest.fixture(scope="module")
def so():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_dqmoe_build", os.path.join(ROOT, "dequant_gemv_moe_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return ctypes.CDLL(b.build())


A = 4096


def test_refusals(so):
    f = so.dq_kv_attention_ex
    f.argtypes = [P, P, P, P, ctypes.c_size_t, P]
    cache = Cache(4, 2, 128, 16, 10, A)
    a = Attn(A, 512, 1, 4, 3, 2, A, A, A, 5, 3, 0.1, 1, 0, A, 512, 1, A)

    def call(**kw):
        x = Scores(**{**dict(softcap=30.0, slopes=A, prefix_len=A, first_pos=A), **kw})
        return f(ctypes.byref(cache), ctypes.byref(a), ctypes.byref(x), A, 0, None)

    assert call() == -4                                     # all that is looked at before the workspace is right
    for cap in (-1.0, 0.009, 2e6, float("nan"), float("inf"), -float("inf")):
        assert call(softcap=cap) == -1, cap
    for bad in (dict(slopes=A + 2), dict(prefix_len=A + 1), dict(first_pos=A + 2)):
        assert call(**bad) == -2, bad
    assert f(ctypes.byref(cache), ctypes.byref(a), None, A, 0, None) == -4
    assert f(ctypes.byref(cache), None, ctypes.byref(Scores()), A, 0, None) == -1


def test_masks_by_hand():
    see = scores_ref.rows_see(3, 5, prefix=4)               # positions 2, 3, 4
    assert see.astype(int).tolist() == [[1, 1, 1, 1, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    see = scores_ref.rows_see(3, 5, first=[0, 3, 3])
    assert see.astype(int).tolist() == [[1, 1, 1, 0, 0], [0, 0, 0, 1, 0], [0, 0, 0, 1, 1]]
    see = scores_ref.rows_see(3, 5, window=2, prefix=5)
    assert see.astype(int).tolist() == [[0, 1, 1, 1, 1], [0, 0, 1, 1, 1], [0, 0, 0, 1, 1]]
    see = scores_ref.rows_see(2, 3, causal=False, first=[1, 9])
    assert see.astype(int).tolist() == [[0, 1, 1], [0, 0, 0]]


def test_reference_by_hand():
    # one token of K = 1, V = 3 in every value, head of 64; q = 1: the score is 64 / 8 = 8 before the cap
    import kv_ref
    cache = np.zeros((1, 1, 1, 18 * 64), dtype=np.uint8)
    for s in range(2):
        kv_ref.write(cache, 16, 64, 0, s, -np.ones(64), -3 * np.ones(64) * (s + 1))
    q = -np.ones((1, 1, 64))
    kw = dict(page_size=16, D=64, q=q, start=[0, 1], kv_len=[2], table=np.zeros((1, 1), dtype=int), scale=1 / 8, n_kv=1)
    for cap, slope in ((0, None), (5.0, None), (0, [0.5]), (5.0, [0.5])):
        out, lse, *_ = scores_ref.attention(cache, softcap=cap, slopes=slope, **kw)
        s = 5 * np.tanh(8 / 5) if cap else 8.0
        w = np.array([s - (0.5 if slope else 0.0), s])
        assert np.allclose(lse, np.log(np.exp(w).sum())) and np.allclose(out, (np.exp(w) * [-3, -6]).sum() / np.exp(w).sum())


def test_polynomial_of_the_cap():
    src = open(os.path.join(ROOT, "dequant_gemv_moe_gb300", "csrc", "kv_attn.cu")).read()
    c = [float(x) for x in re.search(r"kTanh\[7\] = \{([^}]*)\}", src).group(1).split(",")]
    for cap in (0.01, 1.0, 30.0, 1e6):
        top = np.float32(cap * 1.4426950408889634)
        k = (np.array(c) * np.float64(top)).astype(np.float32)
        u = np.linspace(0, 1, 100001).astype(np.float32)
        y = u * u
        r = np.full_like(u, k[6])
        for x in k[5::-1]:
            r = (r.astype(np.float64) * y + x).astype(np.float32)          # one rounding, as an FMA
        got = (r * u).astype(np.float64)
        want = np.tanh(u.astype(np.float64)) * top
        # the interpolation itself is off by 5.2e-8; its coefficients' rounding, the last step's and the product's:
        # 2^-24 each, 1.79e-7 (the steps before enter times y c[k] / c[0], a third of that at most, here unlike signs)
        assert np.abs(got[1:] / want[1:] - 1).max() < 5.2e-8 + 3 * 2.0 ** -24
