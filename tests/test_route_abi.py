"""dq_moe_route's argument checks (before any launch), and the 64-bit routing that the GPU tests compare with
against its definition by hand."""
import ctypes
import os

import numpy as np
import pytest

import route_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P, I, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class Routing(ctypes.Structure):
    _fields_ = [("scores", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_score", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("bias", P)]


@pytest.fixture(scope="module")
def so():
    import importlib.util
    spec = importlib.util.spec_from_file_location("_dqmoe_build", os.path.join(ROOT, "dequant_gemv_moe_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    return ctypes.CDLL(b.build())


A = 4096                    # an aligned address that no refused call reads


def test_refusals(so):
    f = so.dq_moe_route
    f.argtypes = [P, I, L, I, I, I, P, P, P, P]

    def call(logits=A, dtype=0, stride=64, T=3, E=64, k=4, idx=A, gate=A, null=False, **kw):
        r = Routing(**{**dict(scores=1, n_groups=8, top_groups=4, group_score=1, renormalize=1, scale=1.0, bias=A), **kw})
        return f(logits, dtype, stride, T, E, k, None if null else ctypes.byref(r), idx, gate, None)

    for bad in (dict(logits=None), dict(idx=None), dict(gate=None), dict(null=True), dict(dtype=3), dict(dtype=-1),
                dict(T=0), dict(E=0), dict(k=0), dict(k=65, E=64), dict(stride=63), dict(scores=2), dict(scores=-1),
                dict(group_score=2), dict(renormalize=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(n_groups=0), dict(n_groups=7), dict(top_groups=0), dict(top_groups=9),
                dict(n_groups=32, top_groups=1)):
        assert call(**bad) == -1, bad
    for bad in (dict(E=320, stride=320), dict(k=9), dict(E=192, stride=192, n_groups=64),
                dict(E=60, stride=60, n_groups=3, top_groups=3)):
        assert call(**bad) == -3, bad
    for bad in (dict(logits=A + 2), dict(logits=A + 1, dtype=2), dict(idx=A + 2), dict(gate=A + 1), dict(bias=A + 2)):
        assert call(**bad) == -2, bad


def test_layer_refusals(so):
    class Desc(ctypes.Structure):
        _fields_ = [(n, ctypes.c_int32) for n in ("E", "top_k", "hidden", "ffn", "n_shared", "fmt")] + \
                   [(n, P) for n in ("router_W", "w_gate", "w_up", "w_down", "sh_gate", "sh_up", "sh_down")]
    d = Desc(16, 4, 512, 512, 0, 1, A, A, A, A, None, None, None)
    good = dict(scores=1, n_groups=4, top_groups=2, group_score=1, renormalize=1, scale=1.0, bias=None)
    so.dq_moe_forward_ex.argtypes = [P, P, P, I, I, P, P, ctypes.c_size_t, P, P, P, P]
    so.dq_moe_forward_noalloc_ex.argtypes = [P, P, P, I, I, P, P, P, P, P]
    so.dq_moe_router_ex.argtypes = [P, I, I, P, I, I, I, P, P, P, P, P]
    for kw, rc in ((dict(n_groups=5), -1), (dict(n_groups=16, top_groups=2), -1), (dict(scale=0.0), -1),
                   (dict(bias=A + 1), -2), (dict(scores=5), -1)):
        r = ctypes.byref(Routing(**{**good, **kw}))
        assert so.dq_moe_forward_ex(ctypes.byref(d), r, A, 1, 3, A, A, 1 << 30, None, None, None, None) == rc
        assert so.dq_moe_router_ex(A, 16, 512, A, 1, 3, 4, r, A, A, A, None) == rc
    so.dq_expert_cache_set_routing.argtypes = [P, P]
    assert so.dq_expert_cache_set_routing(None, None) == -1


def test_reference_by_hand():
    l = np.log(np.array([[1.0, 2.0, 3.0, 4.0, 5.0, 6.0]]))
    i, g = route_ref.route(l, 2)
    assert i.tolist() == [[5, 4]] and np.allclose(g, [[6 / 11, 5 / 11]])
    i, g = route_ref.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(g, [[12 / 21, 10 / 21]])
    i, g = route_ref.route(l, 2, scores="sigmoid", renormalize=False)
    assert np.allclose(g, [[6 / 7, 5 / 6]])
    # groups (1 2) (3 4) (5 6): a bias that lifts the first expert, gates without it
    i, g = route_ref.route(l, 2, scores="sigmoid", bias=[9, 0, 0, 0, 0, 0], n_groups=3, top_groups=1, renormalize=False)
    assert i.tolist() == [[0, 1]] and np.allclose(g, [[0.5, 2 / 3]])
    # the largest alone, and the two largest's sum
    x = np.array([[3.0, -9.0, 2.0, 2.0]])
    assert route_ref.route(x, 1, n_groups=2, top_groups=1)[0].tolist() == [[0]]
    assert route_ref.route(x, 1, scores="sigmoid", n_groups=2, top_groups=1, group_score="top2")[0].tolist() == [[2]]
    # ties: the lowest first; experts that are out come last, with gate 0
    assert route_ref.route(np.zeros((1, 5)), 3)[0].tolist() == [[0, 1, 2]]
    i, g = route_ref.route(np.array([[-np.inf, 1.0, np.nan, -np.inf]]), 3)
    assert i.tolist() == [[1, 0, 2]] and g.tolist() == [[1.0, 0.0, 0.0]]
