"""dq_moe_route with biases of any size and sign: picks and groups are those of 64 bits (tests/route_ref.py), where the
biases of a group's two best cancel too."""
import numpy as np
import pytest
import torch

from test_gpu_route import NP, check, dq, normal  # noqa: F401  (dq is the fixture)

pytestmark = pytest.mark.gpu

LAST = float(np.finfo(np.float32).max)


def far_biases(E, groups):
    """Logits of which some are out, and biases of fp32's lowest and largest values."""
    g = torch.Generator().manual_seed(E + groups)
    l = torch.randn(120, E, generator=g)
    l[::2][torch.rand(60, E, generator=g) < 0.3] = float("-inf")
    l[40:60, : E // 2] = float("-inf")
    l[60:80, E // 2:] = float("nan")
    rng = np.random.default_rng(E)
    return l.cuda(), (np.full(E, -LAST), np.where(rng.random(E) < 0.7, -LAST, 0.0),
                      np.where(rng.random(E) < 0.5, -LAST, -2e38), np.where(rng.random(E) < 0.5, LAST, -LAST),
                      np.where(rng.random(E) < 0.9, LAST, 2e38), np.where(rng.random(E) < 0.1, 0.0, -LAST))


@pytest.mark.parametrize("E,groups,top,k", [(16, 8, 5, 8), (24, 1, 1, 8), (24, 8, 3, 4), (64, 32, 20, 8), (256, 8, 4, 8),
                                            (256, 32, 16, 8)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_biases_of_the_lowest_and_the_largest_value(dq, E, groups, top, k, scores):  # noqa: F811
    # a bias of fp32's lowest value masks an expert, but not as an infinite logit does: the expert is still a candidate
    l, biases = far_biases(E, groups)
    for b in biases:
        check(dq, l, k, scores=scores, bias=b, n_groups=groups, top_groups=top, group_score="max")


@pytest.mark.parametrize("E,groups,top,k", [(16, 8, 5, 8), (24, 8, 3, 4), (64, 32, 20, 8), (256, 8, 4, 8), (256, 32, 16, 8)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_sums_that_fp32_has_not(dq, E, groups, top, k, scores):  # noqa: F811
    l, biases = far_biases(E, groups)
    for b in biases:
        check(dq, l, k, scores=scores, bias=b, n_groups=groups, top_groups=top, group_score="top2")


@pytest.mark.parametrize("E,groups,top,k", [(64, 32, 8, 8), (96, 32, 9, 6), (128, 32, 8, 8), (256, 32, 8, 8)])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e5, 1e6])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_two_best_that_cancel(dq, E, groups, top, k, size, scores):  # noqa: F811
    # a group's score is s + s' while its values are s + size and s' - size, which fp32 rounds to size * 2^-24
    T, per = 3000, E // groups
    b = np.where(np.arange(E) % per == 0, size, -size)
    b[np.arange(E) % per > 1] = -2 * size
    check(dq, normal(T, E, seed=E + int(np.log10(size))), k, scores=scores, bias=b, n_groups=groups, top_groups=top,
          group_score="top2")


@pytest.mark.parametrize("E,groups,top,k", [(64, 16, 5, 8), (256, 32, 8, 8)])
def test_groups_of_other_sizes_than_the_border(dq, E, groups, top, k):  # noqa: F811
    # biases of every size: what decides is small beside what most groups are
    rng = np.random.default_rng(E)
    b = rng.choice([-1.0, 1.0], E) * 10.0 ** rng.uniform(-3, 6, E)
    per = E // groups
    for g in range(groups):
        b[g * per + 1] = -b[g * per] * (1 + 1e-7 * rng.normal())
        b[g * per + 2:(g + 1) * per] = -1e7
    for scores in ("sigmoid", "softmax"):
        check(dq, normal(1500, E, seed=7), k, scores=scores, bias=b, n_groups=groups, top_groups=top, group_score="top2")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_gates_of_the_least_scores(dq, scores, dtype, renorm):  # noqa: F811
    # scores of e^-88 to e^-100, where fp32 has no full precision left, equal ones among them: the bias takes the picks there
    E, top = 64, 100.0 if scores == "softmax" else 0.0
    g = torch.Generator().manual_seed(3)
    l = top - 88.0 - torch.randint(0, 13, (60, E), generator=g).float()
    l[:, 0] = top
    b = np.zeros(E)
    b[0] = -5.0
    # off by 2^-149 at most before the scale of 2.5, and a gate, a share of a sum of 1e-20 and more, by that over 1e-20
    small = 2.5 * 2.0 ** -148 * (1e20 if renorm else 1.0)
    check(dq, l.to(NP[dtype]).cuda(), 8, small=small, scores=scores, bias=b, renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,top", [(30, 1, 1), (256, 1, 1), (64, 8, 3), (256, 32, 9)])
@pytest.mark.parametrize("bias", [0.0, -1.0, 3.0])
def test_sigmoids_that_64_bits_do_not_tell_apart(dq, E, groups, top, bias):  # noqa: F811
    # above 19 neighbouring logits begin to share 1 / (1 + e^-l), from 37 on it is 1: equal ones go to the lowest index
    g = torch.Generator().manual_seed(E)
    l = 16.0 + 28.0 * torch.rand(150, E, generator=g)
    l[50:100] = 30.0 + 8.0 * torch.rand(50, E, generator=g)
    for x in range(20):                                     # steps of one float
        l[100 + x] = (18.0 + x) * (1 + torch.randint(0, 40, (E,), generator=g) * 2.0 ** -23)
    for gs in ("max", "top2"):
        check(dq, l.cuda(), 6, scores="sigmoid", bias=np.full(E, bias), n_groups=groups, top_groups=top, group_score=gs)
