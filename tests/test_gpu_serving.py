"""A run of rotated append, attention of capped or biased scores and grouped routing as a serving loop has them
(-m gpu): examples/paged_decode.py with each of its options.  The captured steps' last attention against the
definition over what the cache then holds; one more step, its calls recorded, against each operator's definition."""
import numpy as np
import pytest
import torch

import kv_ref
import rope_ref
import route_ref
import scores_ref
from test_gpu_kv import U
from test_gpu_kv_example import example  # noqa: F401  (a fixture)
from test_gpu_rope import check_q, quantise32
from test_gpu_route import GATE_TOL

pytestmark = pytest.mark.gpu


def attention_holds(server, q, att, lse, lengths):
    """The bar of test_gpu_kv_scores: fp16 weights over few rows, whose K is exact."""
    layer, cache, ps, B = server.layer, server.cache, server.page_size, len(lengths)
    D = layer.head_dim
    host = cache.pages.cpu().numpy().reshape(cache.n_pages, layer.kv_heads, ps // 16, 18 * D)
    slopes = None if layer.slopes is None else layer.slopes.cpu().numpy()
    ref, rl, mag, big, eff = scores_ref.attention(
        host, ps, D, q.double().cpu().numpy(), np.arange(B + 1), lengths, server.table.cpu().numpy(), D ** -0.5,
        layer.kv_heads, softcap=layer.softcap, slopes=slopes)
    own = 2.0 ** -21 * eff + 4e-7 * layer.softcap
    e = 2.0 ** -11 * big + own
    vs = np.abs(host[..., 17 * D:].view(np.float16).astype(np.float64))
    bar = U[att.dtype] * np.abs(ref) + (4 * 2.0 ** -11 + 2 * e[..., None]) * mag + max(lengths) * 2.0 ** -26 * np.nanmax(vs)
    assert (np.abs(att.double().cpu().numpy() - ref) <= bar).all()
    assert (np.abs(lse.double().cpu().numpy() - rl) <= own + 2.0 ** -18 * (1 + np.abs(rl))).all()


@pytest.mark.parametrize("rope,softcap,alibi,groups", [(True, 20.0, False, 4), (True, 0.0, False, 2),
                                                       (False, 0.0, True, 4), (True, 5.0, True, 1)])
def test_serving_loop(example, monkeypatch, rope, softcap, alibi, groups):  # noqa: F811
    dq, B, steps = example.dq, 3, 6
    layer = example.Layer(rope=rope, softcap=softcap, alibi=alibi, groups=groups)
    server, last, _ = example.run(requests=B, steps=steps, layer=layer)
    lengths = [p + steps + 1 for p in last["prompts"]]
    assert server.length.tolist() == lengths
    attention_holds(server, last["q"], last["att"], last["lse"], lengths)
    # one more step, with what its calls are given and return
    seen = {}
    append, forward = dq.kv_append_rope, dq.moe_forward

    def kv_append_rope(*a, **kw):
        seen["rope"] = (a, append(*a, **kw))
        return seen["rope"][1]

    def moe_forward(desc, x, **kw):
        y, *seen["route"] = forward(desc, x, want_routing=True, **kw)
        return y

    monkeypatch.setattr(dq, "kv_append_rope", kv_append_rope)
    monkeypatch.setattr(dq, "moe_forward", moe_forward)
    y, q, att, lse, plan = server.step(last["y"], torch.ones(B, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert dq.device_status() == 0 and torch.isfinite(y).all()
    attention_holds(server, q, att, lse, [n + 1 for n in lengths])
    idx, gate, logits = seen["route"]
    want_i, want_g = route_ref.route(logits.cpu().numpy(), 2, "sigmoid", layer.routing.bias.cpu().numpy(), groups,
                                     max(groups // 2, 1), "top2", True, 2.5)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    assert (np.abs(gate.cpu().numpy() - want_g) <= GATE_TOL["sigmoid"] * np.abs(want_g)).all()
    assert ("rope" in seen) == rope
    if rope:
        (cache, q_in, k, v, slots, positions, freq), got = seen["rope"]
        pos = positions.cpu().numpy()
        assert pos.tolist() == lengths
        # check_q's bars are of the output's type: bf16's half step here, of fp32 rows
        check_q(got, q_in, pos, freq.cpu().numpy(), name="bf16")
        kr, _ = rope_ref.rotate(k.cpu().numpy(), pos, freq.cpu().numpy())
        kc, kd = rope_ref.quantise(kr)
        vc, vd = quantise32(v.cpu().numpy())
        host = cache.pages.cpu().numpy().reshape(cache.n_pages, layer.kv_heads, server.page_size // 16, 18 * layer.head_dim)
        for h in range(layer.kv_heads):
            gk, gv = kv_ref.read(host, server.page_size, layer.head_dim, h, slots.cpu().numpy())
            np.testing.assert_array_equal(gk, (kd[..., None] * (kc.reshape(B, -1, layer.head_dim // 32, 32) - 8))
                                          .reshape(B, -1, layer.head_dim)[:, h])
            np.testing.assert_array_equal(gv, (vd[..., None] * (vc.reshape(B, -1, layer.head_dim // 32, 32) - 8))
                                          .reshape(B, -1, layer.head_dim)[:, h])
