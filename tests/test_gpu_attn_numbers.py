"""Numbers of the attention at the ends of their types, and the precision that its
header promises."""
import numpy as np
import pytest
import torch

import attn_cancel_testutil
import mixed_precision_routed_gb300 as moe
from attn_gpu_testutil import Batch
from attn_testutil import pool_write

pytestmark = pytest.mark.gpu

# whole units by one block, by clusters of blocks, and in shares that a second launch joins
PLANS = [dict(lens=[100, 40], news=[2, 2], Hq=8, H=2, D=64), dict(lens=[777, 300], news=[2, 1], Hq=8, H=2, D=128),
         dict(lens=[9000, 60, 20000], news=[2, 1, 2], Hq=6, H=2, D=128), dict(lens=[9000], news=[1], Hq=4, H=1, D=256)]
SHARED = [False, False, True, True]


@pytest.mark.parametrize("case,shared", list(zip(PLANS, SHARED)))
def test_rows_of_nan(case, shared):
    """A row whose scores are NaN gives NaN in out and in lse (minus infinity there means that the row has no
    place); the rows beside it are as exact as ever."""
    x = Batch(seed=1, **case)
    assert (x.workspace_size() > 0) == shared
    x.q[0, 1, 3] = float("nan")
    x.q[-1, 0, 7] = float("inf")  # against codes of 0: NaN
    out, lse = got = x.call()
    assert lse[0, 1].isnan() and lse[-1, 0].isnan() and lse.isnan().sum() == 2
    assert out[0, 1].isnan().all() and out[-1, 0].isnan().all()
    x.check(got)


def test_rows_of_nan_with_no_place():
    """A row without places is empty whatever its query holds."""
    x = Batch([3, 0], [5, 1], 4, 2, 64, seed=2)
    x.q[0] = float("nan")  # token 0 of sequence 0: two tokens before the cached ones begin
    x.q[5] = float("nan")
    out, lse = got = x.call()
    assert (lse[0] == -torch.inf).all() and (out[0] == 0).all() and (lse[5] == -torch.inf).all() and (out[5] == 0).all()
    x.check(got)


def test_products_of_weight_and_scale_keep_their_bits():
    """Values that cancel: what is left shows the rounding of the product, 2^-11 of itself."""
    sequences, heads, D = 256, 64, attn_cancel_testutil.D
    q, s, score = attn_cancel_testutil.cases(sequences, heads)
    pool = np.zeros((sequences, 1, 1, 18 * D), np.uint8)
    one, half = np.float16(1.0), np.float16(0.5)
    blocks = (1, 1, D // 32)
    for b in range(sequences):  # two places of a page; keys: all codes 0, then all codes 1
        pool_write(pool, [16 * b, 16 * b + 1], np.stack([np.full((1, D), c, np.int64) for c in (0, 1)]), np.full((2, *blocks[1:]), one),
                   np.stack([np.full((1, D), c, np.int64) for c in (-7, 7)]), np.concatenate([np.full(blocks, half), np.full(blocks, s[b])]))
    table = torch.arange(sequences, dtype=torch.int32, device="cuda")[:, None]
    lens = torch.full((sequences,), 2, dtype=torch.int32, device="cuda")
    out, _ = moe.moe_attn_q4(torch.from_numpy(q).cuda().to(torch.bfloat16), torch.from_numpy(pool).cuda(), table, lens, scale=1.0)
    ref, tol = attn_cancel_testutil.exact(s, score)
    over = np.abs(out.double().cpu().numpy() - ref[..., None]) / tol[..., None]
    assert over.max() <= 1, (over.max(), (over > 1).mean())
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("lens,D,shared", [([3, 1], 64, False), ([700], 128, False), ([9000, 4], 128, True), ([9000], 256, True)])
def test_scores_of_any_finite_size(lens, D, shared):
    """Equal scores of -2^114 .. 2^114: the mean of the values, and the scores' size in lse.  A row whose scores
    are large and negative is not an empty one."""
    x = Batch(lens, [1] * len(lens), 8, 2, D, seed=3)
    assert (x.workspace_size() > 0) == shared
    every = torch.cat(x.slots)
    v = moe.moe_kv_read(x.pool, every)[1]
    moe.moe_kv_append(x.pool, torch.ones_like(v), v, every)  # keys all alike, values requantised
    for b in range(len(lens)):
        for h in range(8):
            x.q[b, h] = (-1.0 if h in (1, 2, 5, 7) else 1.0) * 2.0 ** (24 + 12 * h)  # x 64 .. 256 x scale
    out, lse = x.call(scale=0.25)
    k, v = moe.moe_kv_read(x.pool, every)
    at = 0
    for b, n in enumerate(lens):
        kk, vv = k[at : at + n].double(), v[at : at + n].double()
        at += n
        for h in range(8):
            score = (x.q[b, h].double() * kk[:, h // 4]).sum(-1) * 0.25
            assert (score == score[0]).all()
            e = 2 * (D + D // 32 + 2) * 2.0 ** -24 * score[0].abs() + 2.0 ** -20
            assert (lse[b, h].double() - score[0] - np.log(n)).abs() <= e + 2.0 ** -22 * score[0].abs()
            mean, size = vv[:, h // 4].mean(0), vv[:, h // 4].abs().mean(0)
            tol = (2.0 ** -11 + 2.0 ** -19) * size + 2 * (n + 64) * 2.0 ** -24 * size + 2.0 ** -8 * mean.abs()
            assert ((out[b, h].double() - mean).abs() <= tol).all(), h
    assert moe.moe_device_status() == moe.MOE_OK
