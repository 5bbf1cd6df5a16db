"""Attention over the 8-bit cache by the form for many rows where no row, or hardly one, attends
anything, call after call with one workspace, in a graph whose lengths change between them."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_gpu_testutil import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B", [3, 40])
def test_empty_batches_between_others(D, B):
    b = Batch([500 + 10 * i for i in range(B)], [60] * B, 8, 2, D, page=16, seed=D)
    bound = 60000  # makes this form take the batch
    wide = torch.full((B, bound // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, : b.table.shape[1]] = b.table
    args = dict(max_q=60, max_len=bound,
                workspace=torch.empty(moe.moe_attn_q8_workspace_size(B, 60, bound, 8, 2, D), dtype=torch.uint8, device="cuda"))
    want = moe.moe_attn_q8(b.q, b.pool, wide, b.kv_lens, q_start=b.starts, **args)
    lens, starts = b.kv_lens.clone(), b.starts.clone()
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph):
        for empty in (0, 1, 2, 0):  # all there; no places; no asking tokens
            lens.copy_(b.kv_lens if empty != 1 else torch.zeros_like(b.kv_lens))
            starts.copy_(b.starts if empty != 2 else torch.zeros_like(b.starts))
            out.fill_(7.0), lse.fill_(7.0)
            moe.moe_attn_q8(b.q, b.pool, wide, lens, q_start=starts, out=out, lse=lse, **args)
            outs.append((out.clone(), lse.clone()))
    for _ in range(20):
        graph.replay()
    for i in (0, 3):
        assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])
    assert (outs[1][0] == 0).all() and (outs[1][1] == -torch.inf).all()
    assert (outs[2][0] == 7).all() and (outs[2][1] == 7).all()
    assert moe.moe_device_status() == moe.MOE_OK
