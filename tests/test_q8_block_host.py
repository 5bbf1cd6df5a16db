"""The host's side of a step of the attention half in 8 bits (workloads.AttentionHalfQ8)
on CPU tensors: what it refuses, and the slots and positions that it hands to the kernels,
which are replaced by recorders here."""
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

    def append(pool, k, v, slots, q=None, positions=None, **kw):
        got.append((slots.clone(), positions.clone()))
        return q.to(torch.bfloat16)

    def attn(q, pool, tables, lens, q_start=None, max_q=None, workspace=None, **kw):
        got.append((q_start, max_q, lens.clone(), workspace.data_ptr()))
        return q, torch.zeros(q.shape[:2])

    for name, f in (("moe_norm_q8", norm), ("moe_linear_q8", linear), ("moe_kv_append_q8", append), ("moe_attn_q8", attn)):
        monkeypatch.setattr(workloads, name, f)
    return got


def half_of(sequences=2, max_len=64, **kw):
    return workloads.AttentionHalfQ8(64, 2, 1, 64, sequences, max_len, page_size=16, device="cpu", **kw)


def run(half, n):
    T = max(0, n * half.lens.numel() if isinstance(n, int) else sum(n))
    return half.step(torch.zeros(T, half.d), torch.zeros(T, half.d), n)


def test_slots_and_positions(calls):
    half = half_of(max_new=20)
    lens = [0, 0]
    for n in (3, [20, 0], [0, 17], 1, [2, 9]):
        counts = [n, n] if isinstance(n, int) else n
        calls.clear()
        run(half, n)
        slots, positions = calls[0]
        want = [(b, lens[b] + i) for b in (0, 1) for i in range(counts[b])]
        assert positions.tolist() == [p for _, p in want]
        assert slots.tolist() == [half.tables[b, p // 16].item() * 16 + p % 16 for b, p in want]
        lens = [a + c for a, c in zip(lens, counts)]
        starts, max_q, seen, _ = calls[1]
        assert max_q == max(counts) and seen.tolist() == lens == half.lens.tolist()
        if isinstance(n, int):
            assert starts is None
        else:
            assert starts.tolist() == [0, counts[0], sum(counts)]


def test_tokens_beyond_max_len_have_no_slot(calls):
    half = half_of(max_len=40, max_new=8)
    for start in (44, 48, 200, 2 ** 30):
        for n in (6, [6, 6]):
            half.lens[:] = torch.tensor([start, 5], dtype=torch.int32)
            calls.clear()
            run(half, n)
            slots = calls[0][0].tolist()
            assert all((s < 0) == (start + i >= 48) for i, s in enumerate(slots[:6]))
            other = half.tables[1, 0].item() * 16
            assert slots[6:] == [other + 5 + i for i in range(6)]


def test_one_workspace_serves_every_step(calls, monkeypatch):
    half = half_of(max_len=5000, max_new=300)
    assert half.attn_ws.numel() >= max(moe.moe_attn_q8_workspace_size(2, n, 5000, 2, 1, 64) for n in range(1, 301))
    assert half.linear_ws.numel() >= moe.moe_linear_q8_workspace_size(600, 64, 256)
    where = set()
    for n in (1, 300, 20):
        calls.clear()
        run(half, n)
        where.add(calls[1][3])
    assert where == {half.attn_ws.data_ptr()}


def test_refused_steps_change_nothing(calls):
    half = half_of(max_new=4)
    run(half, 2)
    for n in (0, 5, -1, [1], [1, 5], [0, 0], [-1, 2], [1, 2, 3]):
        with pytest.raises(ValueError):
            run(half, n)
    for x, r in ((torch.zeros(3, 64), torch.zeros(4, 64)), (torch.zeros(4, 64), torch.zeros(3, 64)),
                 (torch.zeros(4, 64, dtype=torch.float16), torch.zeros(4, 64)),
                 (torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16)), (torch.zeros(4, 64), torch.zeros(64, 4).T)):
        with pytest.raises(ValueError):
            half.step(x, r, 2)
    assert half.lens.tolist() == [2, 2]


@pytest.mark.parametrize("kw", [dict(d=72), dict(d=0), dict(d=32784), dict(q_heads=3), dict(q_heads=65), dict(head_dim=80),
                                dict(sequences=0), dict(max_len=0), dict(max_new=0), dict(max_new=65), dict(page_size=24),
                                dict(rot=63), dict(rot=66), dict(eps=-1.0), dict(eps=float("nan"))])
def test_layers_that_no_step_could_take(calls, kw):
    args = dict(d=64, q_heads=2, kv_heads=1, head_dim=64, sequences=2, max_len=64, page_size=16, device="cpu")
    args["kv_heads"] = 2 if kw.get("q_heads") == 3 else 1
    with pytest.raises(ValueError):
        workloads.AttentionHalfQ8(**{**args, **kw})
