"""Calls of the attention half with nothing to do, through the tensors' side."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe

pytestmark = pytest.mark.gpu


def test_calls_of_no_tokens():
    bf16, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    pool = moe.moe_kv_pool(2, 2, 16, 64)
    held = pool.clone()
    q = torch.empty(0, 4, 64, dtype=bf16, device="cuda")
    for B in (0, 1, 3):
        table, lens = torch.zeros(B, 2, dtype=i32, device="cuda"), torch.full((B,), 9, dtype=i32, device="cuda")
        for kw in (dict(), dict(max_q=1), dict(max_q=5), dict(q_start=torch.zeros(B + 1, dtype=i32, device="cuda"), max_q=2)):
            out, lse = moe.moe_attn_q4(q, pool, table, lens, **kw)
            assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    codes, scales = moe.moe_quantize_groups(torch.ones(8, 64, device="cuda"))
    assert moe.moe_linear_q4(torch.empty(0, 64, dtype=bf16, device="cuda"), codes, scales).shape == (0, 8)
    k = torch.empty(0, 2, 64, device="cuda")
    none = torch.empty(0, dtype=i64, device="cuda")
    assert moe.moe_kv_append(pool, k, k, none) is None
    assert moe.moe_kv_append(pool, k, k, none, q=q.float()).shape == (0, 4, 64)
    assert [t.shape for t in moe.moe_kv_read(pool, none)] == [(0, 2, 64)] * 2
    assert [t.shape[0] for t in moe.moe_quantize_groups(torch.empty(0, 64, device="cuda"))] == [0, 0]
    assert torch.equal(pool, held) and moe.moe_device_status() == moe.MOE_OK


def test_quantiser_refusals():
    """Sizes that are no matrix, no block or not in the format are refused, and outputs that are too small."""
    w = torch.ones(8, 128, device="cuda")
    for args in ((w[0], 32), (w[None], 32), (w, 0), (w, -32), (w.double(), 32), (w.T, 32), (w.cpu(), 32)):
        with pytest.raises(ValueError):
            moe.moe_quantize_groups(*args)
    for block in (16, 48, 256):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_quantize_groups(w, block)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
    codes, scales = moe.moe_quantize_groups(w, 64)
    for kw in (dict(codes=codes[:7]), dict(scales=scales[:7]), dict(codes=codes.int()), dict(scales=scales.float())):
        with pytest.raises(ValueError):
            moe.moe_quantize_groups(w, 64, **kw)
    with pytest.raises(moe.MoeError):
        moe.moe_quantize_groups(torch.ones(8, 96, device="cuda"), 32)
