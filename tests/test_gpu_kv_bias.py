"""A distance bias' own error: it is a product and a sum of fp32, whatever the distance and the place in a tile.

Bars, in the score's units.  Rows that see their own position alone have a bias of 0, and their lse is their score, a product as
q has one value that is not 0: test_gpu_kv_caps' bar without a cap, 9e-7 of the score and 3.2e-6 ln 2.  Rows of zeros have
the bias' own sum: a term's bias, M and the sum of both are each rounded at no more than 30 log2 e + 14 where the term
counts (e^-30 below the largest), 3 * 2^-24 of it each, and the slope in units of log 2 by 2^-23 of a bias of 30:
1.1e-5 + 3.6e-6, besides the 3.2e-6 ln 2, where such terms carried the sum; a row's own position carries it, so that a
term e^-b has e^-b of it: (44 b + 14) e^-b with b in nats is below 40: 40 * 2^-24 * 3 and the above."""
import numpy as np
import pytest
import torch

import scores_ref
from test_gpu_kv import Case, _i32, dq  # noqa: F401  (dq is the fixture)

pytestmark = pytest.mark.gpu

SHAPES = [([1] * 9, list(range(60, 69)), 32, 8, 128, "fp16"), ([60], [300], 2, 2, 64, "bf16"), ([300], [300], 4, 4, 64, "fp16"),
          ([200, 150], [2000, 150], 8, 2, 128, "bf16"), ([190], [400], 6, 2, 256, "fp16")]


def slopes_of(H, at):
    return np.array([[30.0, 0.7, 1e-3, -0.013][(h + at) % 4] for h in range(H)], dtype=np.float32)


@pytest.mark.parametrize("new,kv,H,n_kv,D,dtype", SHAPES)
@pytest.mark.parametrize("cap", [0.0, 30.0, 300.0])
@pytest.mark.parametrize("at", range(4))
def test_a_row_s_own_position(dq, new, kv, H, n_kv, D, dtype, cap, at):  # noqa: F811
    c = Case(dq, D + H, new, kv, H, n_kv, D, 16, dtype)
    rng = np.random.default_rng(D + at)
    T = sum(new)
    q = np.zeros((T, H, D))
    where = rng.integers(0, D, (T, H))
    np.put_along_axis(q, where[..., None], (rng.choice([-1.0, 1.0], (T, H)) * 10.0 ** rng.uniform(-3, 1, (T, H)))[..., None], 2)
    c.q = torch.tensor(q, dtype=torch.float32).to(c.q.dtype).cuda()
    c.q64 = c.q.double().cpu().numpy()
    first = np.concatenate([np.arange(L - n, L) for n, L in zip(new, kv)]).astype(np.int32)
    slopes = slopes_of(H, at)
    _, lse = c.run(max_q_len=max(new), scale=1.0, softcap=cap, first_pos=_i32(first), slopes=torch.tensor(slopes).cuda())
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    _, want, _, _, _ = scores_ref.attention(c.host, c.ps, D, c.q64, c.start, c.kv, c.table, 1.0, n_kv, softcap=cap,
                                            slopes=slopes, first_pos=first)
    off = np.abs(lse.double().cpu().numpy() - want)
    bar = 9e-7 * np.abs(want) + 3.2e-6 * np.log(2)
    print("%.2e, %.2f of the bar" % (off.max(), (off / bar).max()))
    assert (off <= bar).all()


@pytest.mark.parametrize("new,kv,H,n_kv,D,dtype", SHAPES)
@pytest.mark.parametrize("prefix", [False, True])
def test_sums_of_the_bias(dq, new, kv, H, n_kv, D, dtype, prefix):  # noqa: F811
    c = Case(dq, D + H, new, kv, H, n_kv, D, 16, dtype)
    c.q.zero_()
    slopes = np.abs(slopes_of(H, 0))
    pre = np.array([L // 3 for L in kv], dtype=np.int32) if prefix else None
    _, lse = c.run(max_q_len=max(new), slopes=torch.tensor(slopes).cuda(), prefix_len=None if pre is None else _i32(pre))
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    _, want, _, _, _ = scores_ref.attention(c.host, c.ps, D, c.q64 * 0, c.start, c.kv, c.table, 1.0, n_kv, slopes=slopes,
                                            prefix_len=pre)
    off = np.abs(lse.double().cpu().numpy() - want)
    bar = 9e-7 * np.abs(want) + 3.2e-6 * np.log(2) + 40 * 3 * 2.0 ** -24
    print("%.2e, %.2f of the bar" % (off.max(), (off / bar).max()))
    assert (off <= bar).all()
