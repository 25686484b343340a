"""dq_kv_attention where its work sharing is at its edges (-m gpu): windowed prompts,
windows as large as an int, lengths as large as a table can list,
rows that a call leaves out, groups of V of very different sizes;
and the binding's refusals.

The bars are test_gpu_kv's.  Where no K is rounded (few rows, or rows that see at
most 1024 tokens) the lse is held to what fp32 sums give: 2^-18 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import kv_ref
from test_gpu_kv import Case, bar_of, dq  # noqa: F401  (dq is the fixture)

pytestmark = pytest.mark.gpu


def definition(c, scale=None, causal=True, window=0):
    return kv_ref.attention(c.host, c.ps, c.D, c.q64, c.start, c.kv, c.table, c.D ** -0.5 if scale is None else scale,
                            causal, window, c.n_kv)


def lse_is_exact(c, lse, **kw):
    ref = definition(c, **kw)[1]
    none = np.isneginf(ref)
    got = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(got), none)
    ref, got = np.where(none, 0, ref), np.where(none, 0, got)
    off = np.abs(got - ref)
    assert (off <= 2.0 ** -18 * (1 + np.abs(ref))).all(), off.max()


@pytest.mark.parametrize("new,kv,H,n_kv,D,window", [
    ([300], [900], 8, 8, 128, 130),                # one head to a K/V head: an item's second row tile starts two tiles
    ([2048], [2048], 8, 8, 128, 512),              # behind its first one
    ([700, 129, 300], [700, 900, 310], 8, 8, 64, 42),
    ([1000], [1500], 6, 6, 64, 1024),              # the widest window of exact scores
    ([1300, 40], [2600, 2000], 5, 5, 64, 1100),    # and one beyond
    ([900], [2500], 3, 3, 128, 2000),
    ([513, 0, 257, 90], [513, 10, 2000, 60], 4, 4, 128, 1),
    ([400, 333], [400, 800], 12, 6, 64, 77),
    ([260, 300], [500, 300], 3, 3, 256, 65),
])
def test_windowed_prompts(dq, new, kv, H, n_kv, D, window):  # noqa: F811
    c = Case(dq, 30, new, kv, H, n_kv, D, 16, "fp16")
    out, lse = c.run(max_q_len=max(new), window=window)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    c.check(out, lse, window=window)
    if window <= 1024:
        lse_is_exact(c, lse, window=window)
    again, lse2 = c.run(max_q_len=max(new), window=window)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new,kv,H,n_kv,D", [
    ([5, 8, 1], [2, 300, 77], 8, 8, 128),          # rows before the cache's first token
    ([6, 6], [0, 3], 8, 2, 256),
    ([300, 200], [90, 700], 4, 4, 64),
    ([150], [20], 8, 2, 128),
])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200])
def test_window_of_any_int(dq, new, kv, H, n_kv, D, window):  # noqa: F811
    c = Case(dq, 31, new, kv, H, n_kv, D, 16, "bf16")
    out, lse = c.run(max_q_len=max(new), window=window)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    c.check(out, lse)
    lse_is_exact(c, lse)
    plain, lse2 = c.run(max_q_len=max(new))
    assert torch.allclose(out.float(), plain.float(), atol=2e-2) and torch.allclose(lse, lse2, atol=1e-4)


@pytest.mark.parametrize("new,kv,H,n_kv,D,ps", [
    ([1], [688], 8, 1, 64, 16),                    # the table's last token
    ([7], [681], 4, 2, 128, 16),
    ([1, 3], [768, 700], 2, 1, 256, 256),
    ([150], [688], 2, 1, 64, 16),
    ([130, 200], [768, 755], 1, 1, 128, 256),
])
def test_the_last_tokens_that_a_table_can_list(dq, new, kv, H, n_kv, D, ps):  # noqa: F811
    # the requests' pages stand at the end of rows that list 2^31 - page_size tokens; the window keeps to them
    c = Case(dq, 32, new, kv, H, n_kv, D, ps, "fp16")
    width = (2 ** 31 - 1) // ps
    pages = -(-max(kv) // ps)
    table = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    table[:, width - pages:] = torch.tensor(c.table[:, :pages], dtype=torch.int32, device="cuda")
    kv_len = torch.tensor([(width - pages) * ps + n for n in kv], dtype=torch.int32, device="cuda")
    start = torch.tensor(c.start, dtype=torch.int32, device="cuda")
    out, lse = dq.kv_attention(c.cache, c.q, start, kv_len, table, window=90, max_q_len=max(new))
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    c.check(out, lse, window=90)
    lse_is_exact(c, lse, window=90)


@pytest.mark.parametrize("most,new,kv,H,n_kv,D", [
    (2, [3, 2, 7], [200, 300, 5], 2, 2, 64),
    (1, [8, 1], [1000, 90], 8, 2, 128),
    (70, [90, 65, 71], [200, 300, 60], 2, 2, 64),
    (130, [400, 130], [500, 130], 4, 1, 128),
    (20, [300, 20], [300, 700], 2, 2, 256),
])
@pytest.mark.parametrize("window", [0, 40])
def test_rows_above_max_q_len_leave_the_others_where_they_stand(dq, most, new, kv, H, n_kv, D, window):  # noqa: F811
    c = Case(dq, 33, new, kv, H, n_kv, D, 16, "fp16")
    T = sum(new)
    behind = 1                                     # and the last row of the last request lies behind T
    q = c.q[:T - behind]
    out, lse = torch.full_like(q, 7.0), torch.full((T - behind, H), 7.0, device="cuda")
    dev = [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (c.start, c.kv, c.table)]
    dq.kv_attention(c.cache, q, *dev, max_q_len=most, window=window, out=out, lse=lse)
    torch.cuda.synchronize()
    assert dq.device_status() == 0
    row = np.concatenate([np.arange(n) for n in new])[:T - behind]
    done = torch.tensor(row < most, device="cuda")
    assert (out[~done] == 7).all() and (lse[~done] == 7).all()
    # the whole result with those rows put in, held to the definition
    full, fl = c.run(max_q_len=max(new), window=window)
    full[:T - behind][done], fl[:T - behind][done] = out[done], lse[done]
    c.check(full, fl, window=window)
    lse_is_exact(c, fl, window=window)


@pytest.mark.parametrize("new,kv,H,n_kv", [
    ([1] * 5, [1, 5, 17, 40, 300], 8, 2),
    ([3, 8], [4, 500], 8, 8),
    ([1], [3000], 4, 1),
    ([1], [20000], 8, 1),                          # over many shares, joined
    ([140, 70], [140, 900], 4, 2),
])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("large", [2.5, 700.0, 8188.0])
def test_v_groups_of_very_different_scales(dq, new, kv, H, n_kv, D, large):  # noqa: F811
    # Values of one group of 32 beside groups whose scales are up to 2^33 as large.  Each group is held to its own
    # size: test_gpu_kv's bar with vmax of the group, and 2^-32 max(1, scale) a token for a product of a weight and
    # a scale that is rounded below fp16's normal range (2^-25 times 8, the row's largest weight being 2^10).
    c = Case(dq, 34, new, kv, H, n_kv, D, 16, "fp16")
    vs = c.host[..., 17 * D:].view(np.float16)
    size = np.array([large, 2.0 ** -17, 2.0 ** -4, 2.0 ** -20, 1.0, 2.0 ** -14, 2.0 ** -9, 2.0 ** -17])
    top = {}
    for g in range(D // 32):
        at = [(kv_ref.v_scale(D, i, g) - 17 * D) // 2 for i in range(16)]
        x = np.clip(vs[..., at].astype(np.float64), -0.6, 0.6) / 0.6 * size[g]
        vs[..., at] = x.astype(np.float16)
        top[g] = np.nanmax(np.abs(vs[..., at].astype(np.float64)))
    c.cache.pages.copy_(torch.from_numpy(c.host))
    out, lse = c.run(max_q_len=max(new), out_dtype=torch.float32)
    ref, rl, mag, big = definition(c)
    lse_is_exact(c, lse)
    scale = np.array([top[x // 32] for x in range(D)])
    n = max(kv)
    bar = bar_of(torch.float32, ref, mag, big, n, 8 * scale) + n * 2.0 ** -32 * np.maximum(1.0, scale)
    off = np.abs(out.double().cpu().numpy() - ref)
    worst = (off / np.maximum(bar, 1e-300)).max((0, 1)).reshape(-1, 32).max(1)
    assert (worst <= 1).all(), worst


def test_binding_refuses_tensors_off_the_device(dq):  # noqa: F811
    # none of these calls launches anything
    c = Case(dq, 35, [1, 2], [20, 40], 4, 2, 64, 16, "fp16")
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    size = dq.kv_attention_workspace_size(c.cache, 4, 2, 3)
    good = dict(q=c.q, q_start=i32(c.start), kv_len=i32(c.kv), block_table=i32(c.table),
                ws=torch.empty(size, dtype=torch.uint8, device="cuda"), out=torch.empty_like(c.q),
                lse=torch.empty(3, 4, device="cuda"))
    for name in good:
        with pytest.raises(ValueError):
            dq.kv_attention(c.cache, **{**good, name: good[name].cpu()})
    with pytest.raises(ValueError):
        dq.kv_attention(c.cache, **{**good, "ws": torch.empty(2 * size, dtype=torch.uint8, device="cuda")[::2]})
    with pytest.raises(dq.DqError):
        dq.kv_attention(c.cache, **{**good, "ws": good["ws"][:size - 1]})
    c.check(*dq.kv_attention(c.cache, **good))
    c.check(*dq.kv_attention(c.cache, **{**good, "ws": torch.empty(-(-size // 4), device="cuda")}))    # bytes count
    k, slots = torch.zeros(3, 2, 64, device="cuda"), torch.full((3,), -1, dtype=torch.int64, device="cuda")
    for a in ((k.cpu(), k, slots), (k, k.cpu(), slots), (k, k, slots.cpu())):
        with pytest.raises(ValueError):
            dq.kv_append(c.cache, *a)
    with pytest.raises(ValueError):
        dq.kv_read(c.cache, slots.cpu())
    with pytest.raises(ValueError):
        dq.kv_read(c.cache, slots, out=(k, k.cpu()))
    with pytest.raises(ValueError):
        dq.KvCache(c.cache.pages.cpu(), 16, 2, 64)
    plan = [i32([3, 4]), i32([1, 1]), i32([[0, 1], [2, 3]]), i32([4, 5]), i32([2])]
    for i in range(5):
        with pytest.raises(ValueError):
            dq.kv_plan(*[t.cpu() if j == i else t for j, t in enumerate(plan)], page_size=16, n_tokens=2)


def test_plan_that_runs_out_counts_no_page_of_the_unserved(dq):  # noqa: F811
    # request 0 needs two pages of the one there is; request 1, behind it, needs none, request 2 one: it is not served
    # either (the needs up to it do not fit), and the page stays on the stack
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = [[3, -1, -1], [5, -1, -1], [6, -1, -1]]
    args = ([16, 4, 16], [32, 2, 1], table, [9, -1, -1, -1], 1)
    ref = kv_ref.plan(*[np.array(a) for a in args[:3]], args[3], 1, 16, 35)
    p = dq.kv_plan(i32(args[0]), i32(args[1]), i32(table), i32(args[3]), i32([1]), page_size=16, n_tokens=35)
    assert p.free_count.item() == ref["free_count"] == 1 and p.unserved.item() == ref["unserved"] == 2
    assert p.kv_len.tolist() == ref["kv_len"] == [16, 6, 16]
    assert p.slots.tolist() == ref["slots"] and p.slots.tolist()[32:34] == [5 * 16 + 4, 5 * 16 + 5]
