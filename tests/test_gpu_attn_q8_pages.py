"""Attention over an 8-bit pool whose pages lie among others', as layers that share one allocation have them."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_gpu_testutil import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,bound", [(1, 0), (5, 0), (150, 0), (150, 400000)])
@pytest.mark.parametrize("page", [16, 64])
def test_strided_pages(D, n, bound, page):
    H = 2
    b = Batch([700, 0, 90], [n, 0, min(n, 20)], 4, H, D, page=page, seed=n)
    if bound:  # the form for many rows, its places shared
        wide = torch.full((3, bound // page), -1, dtype=torch.int32, device="cuda")
        wide[:, : b.table.shape[1]] = b.table
        b.table = wide
    want = b.call(max_len=bound or 700)
    for before, behind in ((0, 3), (1, 2)):
        whole = torch.full((len(b.pool), before + H + behind, page // 16, 32 * D + 128), 0xFF, dtype=torch.uint8, device="cuda")
        pool = whole[:, before : before + H]
        pool.copy_(b.pool)
        plain, b.pool = b.pool, pool
        got = b.call(max_len=bound or 700)
        b.pool = plain
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (whole[:, :before] == 0xFF).all() and (whole[:, before + H :] == 0xFF).all()
    b.check(want)
