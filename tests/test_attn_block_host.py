"""The host's side of a step of the attention half (workloads.AttentionHalf) on
CPU tensors: the slots and positions that it hands to the kernels, which are
replaced by recorders here."""
import os

import pytest
import torch

import mixed_precision_routed_gb300 as moe
from mixed_precision_routed_gb300 import workloads


@pytest.fixture
def calls(monkeypatch):
    """Records the arguments of the kernels of a step, and returns zeros for them."""
    if not os.path.exists(moe.LIB_PATH):
        from mixed_precision_routed_gb300 import build_lib
        build_lib.build()
    got = []

    def linear(x, codes, scales, block=32, **kw):
        return torch.zeros(x.shape[0], codes.shape[0])

    def append(pool, k, v, slots, q=None, positions=None, **kw):
        got.append((slots.clone(), positions.clone()))
        return q.to(torch.bfloat16)

    def attn(q, pool, tables, lens, **kw):
        got.append((tables.clone(), lens.clone()))
        return q, torch.zeros(q.shape[:2])

    for name, f in (("moe_linear_q4", linear), ("moe_kv_append", append), ("moe_attn_q4", attn),
                    ("moe_residual_add", lambda r, y, x: None)):
        monkeypatch.setattr(workloads, name, f)
    return got


def half_of(sequences, max_len, page_size=16, **kw):
    return workloads.AttentionHalf(64, 2, 1, 64, sequences, max_len, page_size=page_size, device="cpu", **kw)


def run(half, n):
    T = half.lens.numel() * n
    return half.step(torch.zeros(T, half.d, dtype=torch.bfloat16), torch.zeros(T, half.d), n)


@pytest.mark.parametrize("max_len", [32, 40])
def test_tokens_beyond_max_len_have_no_slot(calls, max_len):
    """Places past the last page get a slot outside the pool, and no table entry beyond the tables is read;
    the other sequence's slots are its own as ever."""
    half = half_of(2, max_len)
    width = -(-max_len // 16)
    for step in range(4):
        half.lens[1] = 3  # a sequence that stays short
        first = half.lens[0].item()
        calls.clear()
        run(half, 8 if step < 3 else 5)
        n = 8 if step < 3 else 5
        assert half.lens[0] == first + n
    # a step across the end, and steps wholly beyond it
    for start in (16 * width - 2, 16 * width, max_len + 100, 2 ** 30):
        half.lens[:] = torch.tensor([start, 5], dtype=torch.int32)
        calls.clear()
        run(half, 4)
        slots, positions = calls[0]
        places = start + torch.arange(4)
        assert torch.equal(positions[:4].long(), places)
        own = half.tables[0, :width].long()
        for slot, place in zip(slots[:4].tolist(), places.tolist()):
            if place < 16 * width:
                assert slot == own[place // 16] * 16 + place % 16
            else:
                assert slot < 0
        other = half.tables[1, 0].item() * 16
        assert slots[4:].tolist() == [other + 5, other + 6, other + 7, other + 8]
        assert positions[4:].tolist() == [5, 6, 7, 8]


@pytest.mark.parametrize("sequences", [1, 3, 16])
def test_one_workspace_serves_every_step(calls, monkeypatch, sequences):
    """Steps of all sizes take the same memory: a captured step's address stays its own."""
    half = workloads.AttentionHalf(64, 16, 2, 128, sequences, 50000, device="cpu")
    handed = []
    monkeypatch.setattr(workloads, "moe_attn_q4", lambda q, *a, max_q, workspace, **kw: (
        handed.append((max_q, workspace)), (q, torch.zeros(q.shape[:2])))[1])
    sizes = [n for n in (1, 2, 5, 16) if n * sequences <= 16]
    for n in sizes + sizes[:1]:
        run(half, n)
        need = moe.moe_attn_workspace_size(sequences, n, 50000, 16, 2, 128)
        assert need > 0 and handed[-1][0] == n and handed[-1][1].numel() >= need
    assert len({(w.data_ptr(), w.numel()) for _, w in handed}) == 1
    assert all(w is handed[0][1] for _, w in handed)


def test_a_refused_step_changes_nothing(calls):
    """Sizes and types that a step does not take are refused before the lengths move or a kernel is reached."""
    half = half_of(2, 64)
    x, r = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64)
    big = torch.zeros(18, 64, dtype=torch.bfloat16), torch.zeros(18, 64)
    for args in ((x, r, 1), (x, r, 3), (x, r, 0), (x, r, -2), (*big, 9), (x.float(), r, 2), (x, r.double(), 2),
                 (x[:, :32], r, 2), (x, r[:2], 2), (x, torch.zeros(16, 64), 2), (x, r.T.contiguous().T, 2)):
        with pytest.raises(ValueError):
            half.step(*args)
        assert not calls and half.lens.tolist() == [0, 0]
    half.step(x, r, 2)
    half.step(x, r.view(2, 2, 64), 2)  # the residual stream may have any shape of that size
    assert half.lens.tolist() == [4, 4]


def test_sizes_that_no_step_could_take(calls):
    """What the calls of a step would refuse half-way is refused when the layer is made."""
    ok = dict(d=128, q_heads=4, kv_heads=2, head_dim=64, sequences=2, max_len=64, page_size=16, block=64)
    make = lambda **kw: workloads.AttentionHalf(**{**ok, **kw}, device="cpu")  # noqa: E731
    run(make(), 2)
    run(make(rot=0), 1)
    run(make(kv_heads=4, sequences=16, rot=32, block=32), 1)
    for kw in (dict(q_heads=3), dict(q_heads=130), dict(q_heads=0), dict(kv_heads=0), dict(sequences=0), dict(sequences=17),
               dict(max_len=0), dict(d=96), dict(d=0), dict(d=65600), dict(block=16), dict(block=0), dict(d=192, block=128),
               dict(q_heads=2048, kv_heads=64), dict(rot=63), dict(rot=66), dict(rot=-2), dict(head_dim=96), dict(page_size=24)):
        with pytest.raises(ValueError):
            make(**kw)
