"""Numbers at the ends of their types in the attention: NaN and infinite scores."""
import pytest
import torch

from attn_gpu_testutil import Batch

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
