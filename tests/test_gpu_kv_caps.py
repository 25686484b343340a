"""A cap's own error.  Every row sees its own position alone, so that the lse is its capped score; a row of q has one value
that is not 0, so that the score is a product and nothing hides the cap behind a sum's roundings.

Bars, in the score's units, x = the capped score.  Relative: the scale of K's group, the call's scale in its units (3) and the
product are 5 roundings of 2^-24, the cap's constant, the logarithm's sum and its ln 2 another 4, tanh 2.5e-7 by its
polynomial: 9e-7.  Absolute: the largest weight is at
most 2^14, so the argument of its exponential and M + log2 of the sum are rounded at up to 14 (2^-24 of it each), log2 is off by
one unit (2^-20) and the exponential by two (2^-22 / ln 2): 3.2e-6 ln 2.  Many rows and caps up to 100
take c - 2c / t, t = 1 + e^2u: e^2u is off by two units (2^-22, times 1 - 1 / t), t by 2^-24, the product of two t by
2^-24, its inverse by 2^-23, its product by 2^-24, all times 2c / t: at most 6e-7 c (t = 1), 4.2e-7 c at t = 2; the argument's
roundings are 2^-23 u / cosh(u)^2 c, 6e-8 c at most: 7e-7 of the cap."""
import numpy as np
import pytest
import torch

import scores_ref
from test_gpu_kv import Case, _i32, dq  # noqa: F401  (dq is the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap", [0.01, 1.0, 30.0, 50.0, 100.0, 100.5, 3000.0, 1e6])
@pytest.mark.parametrize("new,kv,H,n_kv,D,dtype", [([1] * 9, list(range(60, 69)), 32, 8, 128, "fp16"), ([60], [300], 2, 2, 64, "bf16"),
                                                   ([7, 2], [500, 40], 8, 2, 256, "fp16"), ([300], [300], 4, 4, 64, "fp16"),
                                                   ([200, 150], [2000, 150], 8, 2, 128, "bf16"), ([190], [400], 6, 2, 256, "fp16")])
@pytest.mark.parametrize("bias", [False, True])
def test_a_capped_score_by_itself(dq, new, kv, H, n_kv, D, dtype, cap, bias):  # noqa: F811
    c = Case(dq, D + H, new, kv, H, n_kv, D, 16, dtype)
    rng = np.random.default_rng(D + len(new))
    T = sum(new)
    q = np.zeros((T, H, D))
    at = rng.integers(0, D, (T, H))
    np.put_along_axis(q, at[..., None], (rng.choice([-1.0, 1.0], (T, H)) * 10.0 ** rng.uniform(-4, 1, (T, H)))[..., None], 2)
    c.q = torch.tensor(q, dtype=torch.float32).to(c.q.dtype).cuda()
    c.q64 = c.q.double().cpu().numpy()
    first = np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)]).astype(np.int32)
    # a bias is 0 at a row's own position: it selects the kernel that takes both
    slopes = torch.full((H,), 0.25, device="cuda") if bias else None
    _, lse = c.run(max_q_len=max(new), scale=cap, softcap=cap, first_pos=_i32(first), slopes=slopes)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    _, want, _, _, eff = scores_ref.attention(c.host, c.ps, D, c.q64, c.start, c.kv, c.table, cap, n_kv, softcap=cap,
                                              first_pos=first)
    off = np.abs(lse.double().cpu().numpy() - want)
    many = max(new) * (H // n_kv) > 64 and cap <= 100 and not bias
    bar = 9e-7 * np.abs(want) + 3.2e-6 * np.log(2) + (7e-7 * cap if many else 0.0)
    print("cap %g: %.2e of the cap, %.2f of the bar" % (cap, off.max() / cap, (off / bar).max()))
    assert (off <= bar).all()
    # the scores lie on both sides of the form's change at |u| = 1
    u = np.abs(want) / cap
    assert (u < 1e-2).any() and (u > 0.9).any()
