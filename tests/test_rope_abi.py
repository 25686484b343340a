"""dq_kv_append_rope's argument checks (before any launch), and the rotation that the GPU tests compare with."""
import ctypes
import os

import numpy as np
import pytest

import rope_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


class Cache(ctypes.Structure):
    _fields_ = [("fmt", I32), ("n_kv_heads", I32), ("head_dim", I32), ("page_size", I32), ("n_pages", I32), ("pages", P)]


class Rope(ctypes.Structure):
    _fields_ = [("q", P), ("q_stride", I64), ("k", P), ("k_stride", I64), ("v", P), ("v_stride", I64), ("dtype", I32),
                ("n_q_heads", I32), ("T", I32), ("slots", P), ("positions", P), ("inv_freq", P), ("rotary_dim", I32),
                ("interleaved", I32), ("factor", ctypes.c_float), ("q_out", P), ("out_stride", I64), ("out_dtype", I32)]


@pytest.fixture(scope="module")
def so():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_dqmoe_build", os.path.join(ROOT, "dequant_gemv_moe_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return ctypes.CDLL(b.build())


A = 4096                    # an aligned address that no refused call reads


def test_refusals(so):
    so.dq_kv_append_rope.argtypes = [P, P, P]
    cache = Cache(4, 2, 128, 16, 10, A)
    good = dict(q=A, q_stride=1024, k=A, k_stride=1024, v=A, v_stride=1024, dtype=2, n_q_heads=4, T=3, slots=A,
                positions=A, inv_freq=A, rotary_dim=128, interleaved=0, factor=1.0, q_out=2 * A, out_stride=512, out_dtype=2)

    def call(c=cache, **kw):
        a = Rope(**{**good, **kw})
        return so.dq_kv_append_rope(ctypes.byref(c) if c else None, ctypes.byref(a), None)

    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(positions=None), dict(inv_freq=None), dict(q_out=None),
                dict(T=0), dict(T=-1), dict(dtype=3), dict(dtype=-1), dict(out_dtype=3), dict(out_dtype=-1),
                dict(n_q_heads=0), dict(q_stride=511), dict(out_stride=504), dict(k_stride=255), dict(v_stride=248),
                dict(rotary_dim=0), dict(rotary_dim=144), dict(rotary_dim=-16), dict(interleaved=2), dict(factor=0.0),
                dict(factor=float("nan")), dict(factor=float("inf")), dict(factor=-1.0), dict(c=None),
                dict(q_out=A), dict(q_out=A, out_stride=1024, out_dtype=1), dict(k_stride=1 << 33)):
        assert call(**bad) == -1, bad
    for bad in (dict(rotary_dim=24), dict(rotary_dim=127), dict(n_q_heads=4097, q_stride=1 << 24, out_stride=1 << 24),
                dict(T=(1 << 24) + 1), dict(c=Cache(4, 2, 96, 16, 10, A)), dict(c=Cache(3, 2, 128, 16, 10, A))):
        assert call(**bad) == -3, bad
    for bad in (dict(q=A + 8), dict(k=A + 2), dict(v=A + 8), dict(q_out=2 * A + 8), dict(slots=A + 4), dict(positions=A + 2),
                dict(inv_freq=A + 1), dict(k_stride=1025), dict(v_stride=1028), dict(q_stride=1025), dict(out_stride=516),
                dict(c=Cache(4, 2, 128, 16, 10, A + 64))):
        assert call(**bad) == -2, bad


def test_rotation_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.array([np.pi / 2, 0.0], dtype=np.float32)
    y, size = rope_ref.rotate(x, [1], quarter)                       # pairs (1, 3) and (2, 4); the rest stays
    assert np.allclose(y, [[[-3, 2, 1, 4, 5, 6, 7, 8]]], atol=1e-6)
    assert size[0, 0].tolist() == [4, 6, 4, 6, 0, 0, 0, 0]
    y, _ = rope_ref.rotate(x, [1], quarter, interleaved=True, factor=2.0)     # pairs (1, 2) and (3, 4)
    assert np.allclose(y, [[[-4, 2, 6, 8, 5, 6, 7, 8]]], atol=1e-6)
    # a rotation leaves q . k to the distance
    r = np.random.default_rng(0)
    q, k = r.normal(size=(2, 1, 1, 64))
    f = rope_ref.frequencies(64)
    dots = [float((rope_ref.rotate(q, [p + 7], f)[0] * rope_ref.rotate(k, [p], f)[0]).sum()) for p in (0, 100, 100000)]
    assert np.allclose(dots, dots[0], atol=1e-6)
