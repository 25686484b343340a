"""examples/paged_decode.py as a user runs it (-m gpu): plan, append, attention,
GEMVs and the MoE layer in one captured decode step, replayed; the last step's
attention against the definition over what the cache then holds."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import bar_of

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_paged_decode(example):
    steps = 20
    server, last, _ = example.run(requests=5, steps=steps)
    layer, cache, ps = server.layer, server.cache, server.page_size
    lengths = [p + steps + 1 for p in last["prompts"]]
    assert server.length.tolist() == lengths
    assert last["plan"].positions.tolist() == [n - 1 for n in lengths]
    # every request's pages are its own, and the rest is on the stack
    table = server.table.cpu().numpy()
    held = [table[r, :-(-n // ps)].tolist() for r, n in enumerate(lengths)]
    left = server.free[:server.count.item()].tolist()
    assert sorted(sum(held, left)) == list(range(cache.n_pages))
    host = cache.pages.cpu().numpy().reshape(cache.n_pages, layer.kv_heads, ps // 16, 18 * layer.head_dim)
    ref, lse, mag, big = kv_ref.attention(host, ps, layer.head_dim, last["q"].double().cpu().numpy(),
                                          np.arange(6), lengths, table, layer.head_dim ** -0.5, True, 0, layer.kv_heads)
    slots = np.concatenate([table[r, np.arange(n) // ps].astype(np.int64) * ps + np.arange(n) % ps
                            for r, n in enumerate(lengths)])
    vmax = max(np.abs(kv_ref.read(host, ps, layer.head_dim, h, slots)[1]).max() for h in range(layer.kv_heads))
    bar = bar_of(last["att"].dtype, ref, mag, big, max(lengths), vmax)
    assert (np.abs(last["att"].double().cpu().numpy() - ref) <= bar).all()
    assert np.abs(last["lse"].double().cpu().numpy() - lse).max() <= 2.0 ** -11 * big.max() + 2.0 ** -18 * (1 + np.abs(lse).max())
    assert torch.isfinite(last["y"]).all()
