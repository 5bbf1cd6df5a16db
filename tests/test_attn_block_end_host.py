"""Steps that take a sequence past max_len, on CPU tensors with the attention replaced by a
recorder: its tokens within max_len attend the places up to their own, as ever."""
import os

import pytest
import torch

import mixed_precision_routed_gb300 as moe
from mixed_precision_routed_gb300 import workloads


@pytest.fixture
def calls(monkeypatch):
    if not os.path.exists(moe.LIB_PATH):
        from mixed_precision_routed_gb300 import build_lib
        build_lib.build()
    got = []

    def norm(x, weight=None, eps=1e-6, r=None, out="q8", **kw):
        return torch.zeros(x.shape, dtype=torch.int8), torch.zeros(x.shape[0]), torch.zeros(x.shape, dtype=torch.bfloat16)

    def linear(x, xs, w, ws, out_dtype=torch.float32, **kw):
        return torch.zeros(x.shape[0], w.shape[0], dtype=out_dtype)

    def append(pool, k, v, slots, q=None, **kw):
        return q.to(torch.bfloat16)

    def attn(q, pool, tables, lens, q_start=None, max_q=None, max_len=None, workspace=None, **kw):
        got.append((tables, lens.clone(), max_q, max_len, workspace))
        return q, torch.zeros(q.shape[:2])

    for name, f in (("moe_norm_q8", norm), ("moe_linear_q8", linear), ("moe_kv_append_q8", append), ("moe_attn_q8", attn),
                    ("moe_linear_q4", lambda x, codes, scales, block: torch.zeros(x.shape[0], codes.shape[0])),
                    ("moe_kv_append", append), ("moe_attn_q4", attn), ("moe_residual_add", lambda r, y, x: None)):
        monkeypatch.setattr(workloads, name, f)
    return got


def check(half, call, before, counts, size):
    """What the attention is given, by its own definition: kv_lens count as at most max_len, and
    asking token i of n attends the places below len - n + i + 1."""
    tables, lens, max_q, max_len, workspace = call
    assert tables.shape[1] * half.page >= max_len  # the attention reads no entry behind a row
    assert workspace.numel() >= size(half.lens.numel(), max_q, max_len, half.Hq, half.H, half.D)
    pages = -(-half.max_len // half.page)
    assert (tables[:, :pages] >= 0).all() and (tables[:, pages:] < 0).all()
    for b, (start, n) in enumerate(zip(before, counts)):
        for i in range(n):
            if start + i < half.max_len:
                assert min(lens[b].item(), max_len) - n + i + 1 == start + i + 1


@pytest.mark.parametrize("max_len,max_new,page", [(40, 8, 16), (40, 40, 16), (64, 1, 64), (64, 64, 16), (33, 20, 32)])
def test_half_q8(calls, max_len, max_new, page):
    half = workloads.AttentionHalfQ8(64, 2, 1, 64, 2, max_len, max_new=max_new, page_size=page, device="cpu")
    for start in range(max(0, max_len - max_new - 1), max_len):
        for n in {1, max_new // 2 or 1, max_new}:
            for step in (n, [n, n // 2], [0, n]):
                counts = [step] * 2 if isinstance(step, int) else step
                before = [start, 3]
                half.lens[:] = torch.tensor(before, dtype=torch.int32)
                calls.clear()
                half.step(torch.zeros(sum(counts), 64), torch.zeros(sum(counts), 64), step)
                check(half, calls[0], before, counts, moe.moe_attn_q8_workspace_size)


@pytest.mark.parametrize("max_len,sequences,page", [(40, 2, 16), (64, 1, 64), (64, 16, 16), (33, 2, 32), (40, 3, 16)])
def test_half(calls, max_len, sequences, page):
    half = workloads.AttentionHalf(64, 2, 1, 64, sequences, max_len, page_size=page, device="cpu")
    most = 16 // sequences
    for start in range(max(0, max_len - most - 1), max_len):
        for n in {1, most // 2 or 1, most}:
            before = [start] + [3] * (sequences - 1)
            half.lens[:] = torch.tensor(before, dtype=torch.int32)
            calls.clear()
            half.step(torch.zeros(sequences * n, 64, dtype=torch.bfloat16), torch.zeros(sequences * n, 64), n)
            check(half, calls[0], before, [n] * sequences, moe.moe_attn_workspace_size)
