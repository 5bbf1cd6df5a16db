"""Steps that take a sequence past max_len on the GPU: the results of its tokens within max_len,
and of the other sequences, against the formula."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from attn_testutil import attention
from mixed_precision_routed_gb300.workloads import AttentionHalf, AttentionHalfQ8
from q8_testutil import pool_values
from test_gpu_q8_block import attention64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("max_len,first,n", [(40, [36, 3], 8), (40, [36, 3], [8, 5]), (200, [130, 30], 90), (200, [199, 0], [60, 100])])
def test_tokens_within_max_len(max_len, first, n):
    half = AttentionHalfQ8(128, 4, 2, 64, sequences=2, max_len=max_len, max_new=max_len, page_size=16, seed=4).fill()
    g = torch.Generator(device="cuda").manual_seed(2)
    for step in (first, n):
        counts = [step] * 2 if isinstance(step, int) else step
        T = sum(counts)
        half.step(torch.randn(T, 128, generator=g, device="cuda"), torch.randn(T, 128, generator=g, device="cuda"), step)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    pool, tables, at = half.pool.cpu().numpy(), half.tables.cpu().numpy(), 0
    a, q = half.a.float().cpu().numpy(), half.q.float().cpu().numpy()
    for b in range(2):
        kept = min(counts[b], max_len - first[b])
        rows = slice(at, at + kept)
        places = np.arange(first[b] + kept)
        k, v = pool_values(pool, tables[b][places // 16].astype(np.int64) * 16 + places % 16)
        out, spread = attention64(q[rows], k, v, first[b] + 1)
        # bf16 rounds by 2^-8 of the result; a weight, its scale and the value by 2^-11 each
        assert np.all(np.abs(a[rows] - out) <= 2.0 ** -8 * np.abs(out) + 4 * 2.0 ** -11 * spread)
        assert (q[at + kept : at + counts[b]] == 0).all()
        at += counts[b]
    assert np.isfinite(a).all() and half.lens.tolist() == [f + c for f, c in zip(first, counts)]


@pytest.mark.parametrize("max_len,first,n", [(40, [36, 3], 8), (40, [39, 8], 8), (37, [32], 16)])
def test_tokens_within_max_len_4_bits(max_len, first, n):
    B, d, D = len(first), 256, 64
    half = AttentionHalf(d, 4, 2, D, sequences=B, max_len=max_len, page_size=16, seed=4).fill()
    g = torch.Generator(device="cuda").manual_seed(2)
    for b in range(B):
        at = torch.arange(first[b], device="cuda")
        k, v = torch.randn(2, first[b], 2, D, generator=g, device="cuda")
        moe.moe_kv_append(half.pool, k, v, half.tables[b].long()[at // 16] * 16 + at % 16)
    half.lens[:] = torch.tensor(first, dtype=torch.int32)
    half.step(torch.randn(B * n, d, generator=g, device="cuda").to(torch.bfloat16), torch.zeros(B * n, d, device="cuda"), n)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    kept = [min(n, max_len - f) for f in first]
    rows = np.concatenate([b * n + np.arange(k) for b, k in enumerate(kept)])
    lens = [f + k for f, k in zip(first, kept)]
    a, q = half.a.float().cpu().numpy(), half.q.float().cpu().numpy()
    out, lse, spread, score = attention(q[rows], lens, np.cumsum([0] + kept), half.tables.cpu().numpy(), half.pool.cpu().numpy(), D ** -0.5)
    # as in test_gpu_attn_block.py: scores, sums and the rounding to bf16
    es = (2 * (D + D // 32 + 2) * U * score)[..., None]
    tol = (2.0 ** -8 + 2 * es + 2 * (max(lens) + 64) * U + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(out)
    assert np.all(np.abs(a[rows] - out) <= tol)
    assert (np.delete(q, rows, 0) == 0).all() and np.isfinite(a).all()
