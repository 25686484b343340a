"""dq_moe_route and the layer's routing against the definition in 64 bits (tests/route_ref.py): indices equal,
gates within the rounding of fp32."""
import numpy as np
import pytest
import torch

import route_ref
import synth

pytestmark = pytest.mark.gpu

# A gate is exp or a sigmoid (at most 3 units in the last place), a sum of 8 (3 additions deep), a division, the
# scale: 3 + 4 + 2 + 1 roundings of 2^-24 and, of a softmax, the common sum of 256 (13 additions deep, each
# term an ex2 whose argument is rounded: 2^-22 |l - max| e^(l - max), at most 0.37 * 2^-22 of the largest term) and
# the rounding of l - max, which is the exponential's relative error
GATE_TOL = {"sigmoid": 10 * 2.0 ** -24, "softmax": 28 * 2.0 ** -24}

NP = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def dq():
    import dequant_gemv_moe_gb300 as m
    return m


def check(dq, logits, top_k, small=1e-37, **kw):
    bias = kw.get("bias")
    r = dq.MoeRouting(**{**kw, "bias": None if bias is None else torch.tensor(bias, dtype=torch.float32).cuda()})
    idx, gate = dq.moe_route(logits, top_k, r)
    torch.cuda.synchronize()
    host = logits.float().cpu().numpy()
    if bias is not None:
        kw["bias"] = np.asarray(bias, dtype=np.float32)
    want_i, want_g = route_ref.route(host, top_k, **kw)
    np.testing.assert_array_equal(idx.cpu().numpy(), want_i)
    got = gate.cpu().numpy().astype(np.float64)
    tol = GATE_TOL[kw.get("scores", "softmax")]
    if kw.get("scores", "softmax") == "softmax":
        x = np.where(np.isfinite(host), host, 0.0).astype(np.float64)
        far = np.abs(np.take_along_axis(x, want_i, 1) - x.max(1, keepdims=True))
        tol = tol + np.minimum(far, 100.0).max(1, keepdims=True) * 2.0 ** -24
    assert (np.abs(got - want_g) <= tol * np.abs(want_g) + small).all(), np.abs(got / want_g - 1).max()
    return idx, gate


def normal(T, E, dtype="fp32", seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(NP[dtype]).cuda()


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (256, 1, 1, 8), (160, 8, 3, 6), (60, 4, 2, 4), (64, 32, 5, 7),
                                            (8, 1, 1, 2), (1, 1, 1, 1), (255, 1, 1, 8), (96, 16, 16, 8), (34, 2, 1, 8),
                                            (8, 8, 8, 8), (33, 1, 1, 8)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score,bias,renorm", [("top2", True, True), ("max", False, False), ("max", True, False),
                                                     ("top2", False, True)])
def test_route(dq, E, groups, top, k, scores, group_score, bias, renorm):
    for dtype, T in (("fp32", 67), ("bf16", 40), ("fp16", 1)):
        b = np.linspace(-0.2, 0.2, E)[np.random.default_rng(E).permutation(E)] if bias else None
        check(dq, normal(T, E, dtype, seed=E + T), k, scores=scores, bias=b, n_groups=groups, top_groups=top,
              group_score=group_score, renormalize=renorm, scale=2.5)


def test_values_that_fp32_cannot_tell_apart(dq):
    # saturated sigmoids, sums with the bias that meet within an ulp, and exact ties
    rng = np.random.default_rng(3)
    l = rng.normal(size=(64, 256)).astype(np.float32)
    l[:, ::3] = 17.0 + rng.normal(size=l[:, ::3].shape) * 0.5
    l[5] = 0.0
    l[6] = 20.0
    l[7, :128] = l[7, 128:]
    b = np.zeros(256)
    for kw in (dict(scores="sigmoid", bias=b), dict(scores="sigmoid", bias=b, n_groups=8, top_groups=3, group_score="top2"),
               dict(scores="softmax", bias=b + 1.0), dict(scores="sigmoid", n_groups=8, top_groups=2, group_score="top2"),
               dict(scores="softmax", n_groups=4, top_groups=2)):
        check(dq, torch.tensor(l).cuda(), 8, **kw)
    # neighbouring floats, whose keys differ in the bits that the place takes
    x = np.full((8, 256), 1.0, dtype=np.float32)
    x += (rng.permutation(8 * 256).reshape(8, 256) % 40).astype(np.float32) * 2.0 ** -23
    for s in ("softmax", "sigmoid"):
        check(dq, torch.tensor(x).cuda(), 8, scores=s)
        check(dq, torch.tensor(-x).cuda(), 8, scores=s)
    # a bias that cancels the score
    s = 1.0 / (1.0 + np.exp(-l[0].astype(np.float64)))
    check(dq, torch.tensor(l[:1]).cuda(), 8, scores="sigmoid", bias=-s)


@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("E,groups,top", [(256, 1, 1), (256, 8, 4), (60, 4, 2)])
def test_zeros_of_both_signs_are_equal(dq, dtype, E, groups, top):
    g = torch.Generator().manual_seed(E)
    l = torch.where(torch.rand(30, E, generator=g) < 0.5, -0.0, 0.0)
    l[10:] = torch.where(torch.rand(20, E, generator=g) < 0.9, l[10:], -1.0)
    l[20:, 3] = 1.0
    for scores in ("softmax", "sigmoid"):
        for group_score in ("max", "top2"):
            for bias in (None, np.zeros(E)):
                check(dq, l.to(NP[dtype]).cuda(), 6, scores=scores, n_groups=groups, top_groups=top, group_score=group_score,
                      bias=bias)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top,group_score", [(1, 1, "max"), (4, 2, "top2"), (4, 2, "max")])
@pytest.mark.parametrize("bias", [True, False])
def test_scores_that_fp32_has_not(dq, scores, groups, top, group_score, bias):
    # e^-60 to e^-800: beside a bias of 0 64 bits tell them apart (below e^-745, or 1 / e^710, they are 0 there too)
    E = 32
    g = torch.Generator().manual_seed(5)
    l = -60 - 740 * torch.rand(40, E, generator=g)
    l[:20, 8:16] = l[:20, :8].round()                       # some groups near one another
    l[:20, :8] = l[:20, :8].round() + torch.randint(-1, 2, (20, 8), generator=g) * 2.0 ** -14
    l[::3, 5] = 1.0
    b = np.zeros(E)
    b[::7] = 1e-40
    # an fp32 score below 2^-126 is off by 2^-149, and its gate, a share of a sum of 1e-20 and more, by 2^-149 / 1e-20
    check(dq, l.cuda(), 8, small=2.0 ** -149 * 1e20, scores=scores, bias=b if bias else None, n_groups=groups, top_groups=top,
          group_score=group_score)


def test_experts_that_are_out(dq):
    for E, groups, top in ((64, 8, 2), (60, 1, 1), (256, 4, 1)):
        l = normal(9, E, seed=2)
        l[1] = float("-inf")
        l[2, 3:] = float("-inf")
        l[3, ::2] = float("nan")
        l[4, : E // 2] = float("-inf")
        l[5] = float("nan")
        l[6, 5] = float("inf")
        l[7] = -200.0                            # sigmoids of 1e-87: their sum vanishes beside 1e-20
        l[8] = torch.linspace(-3e38, 3e38, E)
        for scores in ("softmax", "sigmoid"):
            for b in (None, np.linspace(1, 0, E)):
                for gs in ("max", "top2"):
                    idx, gate = check(dq, l, 4, scores=scores, bias=b, n_groups=groups, top_groups=top, group_score=gs)
                    assert (gate[1] == 0).all() and idx[1].tolist() == [0, 1, 2, 3]


def test_strided_rows_and_offsets(dq):
    wide = normal(33, 300, seed=9)
    for off in (0, 1, 3):
        check(dq, wide[:, off:off + 256], 8, scores="sigmoid", n_groups=8, top_groups=4, group_score="top2")
        check(dq, wide.bfloat16()[:, off:off + 160], 6, scores="softmax", n_groups=8, top_groups=3)


def test_many_tokens_and_guard_rows(dq):
    T, E, k = 40000, 128, 5
    l = normal(T, E, seed=11)
    b = torch.linspace(-0.1, 0.1, E).cuda()
    idx = torch.full((T + 2, k), -7, dtype=torch.int32, device="cuda")
    gate = torch.full((T + 2, k), -7.0, device="cuda")
    r = dq.MoeRouting("sigmoid", b, 4, 2, "top2")
    dq.moe_route(l, k, r, out=(idx[1:-1], gate[1:-1]))
    torch.cuda.synchronize()
    rows = [0, 1, 777, 20001, T - 1]
    wi, wg = route_ref.route(l[rows].cpu().numpy(), k, "sigmoid", b.cpu().numpy(), 4, 2, "top2")
    np.testing.assert_array_equal(idx[1:-1][rows].cpu().numpy(), wi)
    assert (idx[[0, -1]] == -7).all() and (gate[[0, -1]] == -7).all()


@pytest.mark.parametrize("E,groups,top,k", [(256, 8, 4, 8), (256, 1, 1, 8), (160, 8, 3, 6), (60, 1, 1, 4), (16, 4, 2, 7),
                                            (4, 1, 1, 4), (36, 1, 1, 8), (256, 8, 4, 1)])
@pytest.mark.parametrize("scores,group_score,bias,renorm", [("sigmoid", "top2", True, True), ("sigmoid", "max", True, False),
                                                            ("sigmoid", "top2", False, True), ("softmax", "max", False, False),
                                                            ("sigmoid", "max", False, True), ("softmax", "top2", True, True)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_prompts(dq, E, groups, top, k, scores, group_score, bias, renorm, dtype):
    T = 2051
    b = np.linspace(-0.2, 0.2, E)[np.random.default_rng(E).permutation(E)] if bias else None
    l = normal(T, E, dtype, seed=E + k)
    if dtype == "fp32":                          # rows that a warp takes by itself: beyond the fixed point, out, tied
        l[3] *= 20.0
        l[100, ::2] = float("-inf")
        l[101, 1] = float("nan")
        l[500] = 0.25
        l[777, : E // 2] = l[777, 0]
        l[2050] = float("-inf")
    check(dq, l, k, scores=scores, bias=b, n_groups=groups, top_groups=top, group_score=group_score, renormalize=renorm)


def test_prompts_biased_beyond_the_fixed_point(dq):
    l = normal(2048, 64, seed=1)
    for b in (np.linspace(-5, 5, 64), np.full(64, 1.99), np.linspace(100, 101, 64)):
        check(dq, l, 8, scores="sigmoid", bias=b, n_groups=4, top_groups=2, group_score="top2")
    # a row stride and a base that are no multiples of four logits
    wide = normal(2048, 70, seed=3)
    check(dq, wide[:, 1:65], 8, scores="sigmoid", bias=np.zeros(64))
    check(dq, wide[:, 2:66].bfloat16(), 8)


def test_capture_and_streams(dq):
    l = normal(50, 256, seed=4)
    r = dq.MoeRouting("sigmoid", torch.zeros(256, device="cuda"), 8, 4, "top2", scale=2.5)
    out = (torch.empty(50, 8, dtype=torch.int32, device="cuda"), torch.empty(50, 8, device="cuda"))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        dq.moe_route(l, 8, r, out=out)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            dq.moe_route(l, 8, r, out=out)
    for seed in (5, 6):
        l.copy_(normal(50, 256, seed=seed))
        g.replay()
        torch.cuda.synchronize()
        wi, _ = route_ref.route(l.cpu().numpy(), 8, "sigmoid", np.zeros(256), 8, 4, "top2", scale=2.5)
        np.testing.assert_array_equal(out[0].cpu().numpy(), wi)


# ---------------------------------------------------------------- the layer
def layer(dq, E, k, H, F, ns, seed):
    w = synth.moe_weights(synth.BASE_SEED + seed, E, H, F, ns, 1)
    dev = {n: (torch.from_numpy(v).cuda() if v is not None else None) for n, v in w.items()}
    desc = dq.ops.make_desc(E, k, H, F, ns, 1, dev["router_W"], dev["w_gate"], dev["w_up"], dev["w_down"],
                            dev["sh_gate"], dev["sh_up"], dev["sh_down"])
    return w, dev, desc


@pytest.mark.parametrize("T", [1, 2, 8, 33, 100])
@pytest.mark.parametrize("E,groups,top,k,ns", [(32, 8, 4, 8, 1), (8, 1, 1, 2, 0)])
def test_layer(dq, orc, T, E, groups, top, k, ns):
    H, F = 512, 512
    w, dev, desc = layer(dq, E, k, H, F, ns, 40 + E)
    x = synth.activations(synth.streams(synth.BASE_SEED + T, 1)[0], (T, H), 1)
    bias = torch.linspace(-0.3, 0.3, E).cuda()
    r = dq.MoeRouting("sigmoid", bias, groups, top, "top2", True, 2.5)
    xd = torch.from_numpy(x).cuda()
    y, idx, gate, logits = dq.moe_forward(desc, xd, want_routing=True, routing=r)
    torch.cuda.synchronize()
    # the layer's selection is the operator's on the layer's logits
    i2, g2 = dq.moe_route(logits, k, r)
    assert torch.equal(idx, i2) and torch.equal(gate, g2)
    lg, i3, g3 = dq.moe_router(dev["router_W"], E, H, xd, k, routing=r)
    i4, g4 = dq.moe_route(lg, k, r)
    assert torch.equal(i3, i4) and torch.equal(g3, g4)
    # the gates' sum of the oracle's experts
    gu, dn = F * H // 256 * 144, H * F // 256 * 144

    def ffn(pre, e, t):
        m = [w[pre + n] for n in ("gate", "up", "down")]
        return orc.expert_ffn(1, m[0][e * gu:(e + 1) * gu], m[1][e * gu:(e + 1) * gu], m[2][e * dn:(e + 1) * dn], H, F,
                              orc.act_to_f64(1, x[t:t + 1]).reshape(H))

    want = np.zeros((T, H))
    for t in range(T):
        for i in range(k):
            want[t] += float(gate[t, i]) * ffn("w_", int(idx[t, i]), t)
        for s in range(ns):
            want[t] += ffn("sh_", s, t)
    err = np.abs(y.cpu().numpy() - want).max() / np.abs(want).max()
    assert err <= 2e-3, err
    if T <= 8:
        # without a workspace of the caller's: the same kernels
        y2 = torch.empty_like(y)
        rc = dq.lib.dq_moe_forward_noalloc_ex(desc, r._ref, xd.data_ptr(), 1, T, y2.data_ptr(), None, None, None,
                                              torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0 and np.abs((y2 - y).cpu().numpy()).max() <= 2e-3 * np.abs(want).max()
    # no routing: as before
    a = dq.moe_forward(desc, xd)
    b = dq.moe_forward(desc, xd, routing=dq.MoeRouting())
    torch.cuda.synchronize()
    assert np.abs((a - b).cpu().numpy()).max() <= 2e-3 * np.abs(a.cpu().numpy()).max()


def test_streamed_layer(dq):
    E, k, H, F = 16, 4, 512, 512
    w, dev, desc = layer(dq, E, k, H, F, 0, 77)
    host = {n: torch.from_numpy(w[n]).pin_memory() for n in ("w_gate", "w_up", "w_down")}
    bias = torch.linspace(0.3, -0.3, E).cuda()
    r = dq.MoeRouting("sigmoid", bias, 4, 2, "top2", True, 2.5)
    c = dq.ExpertCache(E, k, H, F, 0, 1, dev["router_W"], host["w_gate"], host["w_up"], host["w_down"], slots=E,
                       max_tokens=6, routing=r)
    x = torch.from_numpy(synth.activations(synth.streams(5, 1)[0], (6, H), 1)).cuda()
    for routing in (r, None, r):
        c.set_routing(routing)
        y = c.forward(x)
        ref = dq.moe_forward(desc, x, routing=routing)
        torch.cuda.synchronize()
        assert ((y - ref).abs().max() <= 2e-3 * ref.abs().max()).item()
    c.close()
