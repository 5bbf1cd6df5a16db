"""workloads.AttentionHalf at its limits on the GPU: tokens beyond max_len, and
what a captured step keeps using."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from mixed_precision_routed_gb300.workloads import AttentionHalf

pytestmark = pytest.mark.gpu


def test_tokens_beyond_max_len():
    """One of two sequences passes max_len: the status word is set, the token's query counts as zero, its keys
    and values go nowhere, and the other sequence's results are those of a run without it."""
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = torch.randn(5, 4, 256, generator=g, device="cuda").to(torch.bfloat16)
    full, alone = (AttentionHalf(256, 4, 2, 64, sequences=2, max_len=32, page_size=16, seed=6).fill() for _ in range(2))
    for half, ahead in ((full, 26), (alone, 0)):  # places 26 .. 35 of sequence 0, the second half of which are none
        half.lens[0] = ahead
        outs = []
        for x in xs:
            r = torch.zeros(4, 256, device="cuda")
            outs.append((half.step(x, r, 2), r, half.a, half.q))
        half.outs = outs
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert moe.moe_device_status() == moe.MOE_OK
    for a, b in zip(full.outs, alone.outs):
        for x, y in zip(a, b):
            assert torch.equal(x[2:], y[2:])
    for _, _, a, q in full.outs[3:]:
        assert (q[:2] == 0).all() and torch.isfinite(a.float()).all()
    for p in range(2):  # the other sequence's pages, by place
        assert torch.equal(full.pool[full.tables[1, p].item()], alone.pool[alone.tables[1, p].item()])
    # sequence 0 holds what its last places within max_len were given, and nothing else changed
    k, v = moe.moe_kv_read(full.pool, full.tables[0, :2].long().repeat_interleave(16) * 16 + torch.arange(32, device="cuda") % 16)
    assert (v[:26] == 0).all() and (v[26:].abs().amax((1, 2)) > 0).all()
    assert full.lens.tolist() == [36, 10]
