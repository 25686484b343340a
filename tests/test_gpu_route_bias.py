"""dq_moe_route with biases of any size and sign: picks and groups are those of 64 bits (tests/route_ref.py)."""
import numpy as np
import pytest
import torch

from test_gpu_route import check, dq  # noqa: F401  (dq is the fixture)

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
