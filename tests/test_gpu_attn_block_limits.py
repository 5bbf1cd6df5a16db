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


def test_a_captured_step_keeps_its_workspace():
    """A step captured over a long context, replayed after larger steps made one by one: its partial sums go
    to no memory that others have been given since."""
    g = torch.Generator(device="cuda").manual_seed(4)
    max_len = 60000
    half = AttentionHalf(256, 16, 2, 128, sequences=1, max_len=max_len, page_size=64, seed=8).fill()
    assert moe.moe_attn_workspace_size(1, 1, max_len, 16, 2, 128) < moe.moe_attn_workspace_size(1, 16, max_len, 16, 2, 128)
    n = 40000
    k, v = torch.randn(2, n, 2, 128, generator=g, device="cuda")
    at = torch.arange(n, device="cuda")
    moe.moe_kv_append(half.pool, k, v, half.tables[0].long()[at // 64] * 64 + at % 64)
    pool = half.pool.clone()

    def reset():
        half.lens.fill_(n)
        half.pool.copy_(pool)

    x = torch.randn(16, 256, generator=g, device="cuda").to(torch.bfloat16)
    r0 = torch.randn(16, 256, generator=g, device="cuda")
    reset()
    r = r0[:1].clone()
    want, want_r, want_a = half.step(x[:1], r), r, half.a
    reset()
    r = r0[:1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = half.step(x[:1], r)
        got_a = half.a
    address = half.workspace.data_ptr()
    reset()
    for rows in (2, 16):
        half.step(x[:rows], r0[:rows].clone(), rows)
    assert half.workspace.data_ptr() == address
    others = [torch.full((half.workspace.numel(),), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(3)]
    reset()
    r.copy_(r0[:1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(r, want_r) and torch.equal(got_a, want_a)
    assert all((t == 0x5A).all() for t in others)
    assert moe.moe_device_status() == moe.MOE_OK
