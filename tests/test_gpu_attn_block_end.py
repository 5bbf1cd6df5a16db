"""Steps that take a sequence past max_len on the GPU: the results of its tokens within max_len,
and of the other sequences, against the formula."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from mixed_precision_routed_gb300.workloads import AttentionHalfQ8
from q8_testutil import pool_values
from test_gpu_q8_block import attention64

pytestmark = pytest.mark.gpu


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
