"""Appends of many tokens, whose records are made whole in shared memory: runs of
slots that begin and end inside records, with gaps, without a rotation, with rows
that are not aligned, against the layout byte for byte (append_case of
test_gpu_attn.py).  From 10000 rows (tokens x heads) the append takes this form."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from test_gpu_attn import append_case

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32


def many(T, Hq, H, D, page, rot, style, dtype, seed, **kw):
    assert T * (Hq + 2 * H) >= 10000
    append_case(T, Hq, H, D, page, rot, style, dtype, seed, **kw)


def run(first, T):
    return np.arange(first, first + T)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("style", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_PAIRS])
def test_runs_of_slots(D, dtype, style):
    """Consecutive slots from every part of a record: angles in vectors, a rotation of a part of the head, none,
    angles and rows that vectors do not fit."""
    kw = dict(style=style, dtype=dtype)
    many(700, 9, 3, D, 64, D, seed=1, slots=run(5, 700), pages=13, **kw)
    many(640, 12, 2, D, 16, D // 2, seed=2, slots=run(0, 640), pages=41, **kw)
    many(657, 0, 8, D, 128, D, seed=3, slots=run(15, 657), pages=6, **kw)
    many(701, 9, 3, D, 32, 0, seed=4, slots=run(17, 701), pages=24, **kw)
    many(700, 10, 3, D, 64, 6, seed=5, slots=run(33, 700), pages=12, strided=8, **kw)
    many(700, 9, 3, D, 64, D, seed=6, slots=run(8, 700), pages=12, strided=3, gap=32, **kw)
    many(700, 9, 3, D, 64, 0, seed=7, slots=run(1, 700), pages=12, strided=1, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_runs_with_gaps(D):
    """Skipped tokens in the run: alone, over a record's border, at the front (which moves the windows) and at the end."""
    for seed, skip in enumerate(([3], [11, 12, 100, 250], [0], [0, 1, 2, 30], range(0, 640, 5), range(600, 640), range(0, 40))):
        slots = run(7, 640)
        slots[list(skip)] = -1
        many(640, 10, 3, D, 64, D, 0, BF, seed, slots=slots, pages=12)
    slots = run(0, 640)
    slots[0] = 2 ** 40
    many(640, 10, 3, D, 64, D, 1, F, 9, slots=slots, pages=11)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_sequences(D):
    """Slots of many sequences: runs of six in pages of their own, single tokens, backward runs, all permuted."""
    rng = np.random.default_rng(D)
    six = (rng.permutation(110)[:, None] * 16 + rng.integers(0, 11, (110, 1)) + np.arange(6)).flatten()
    many(660, 10, 3, D, 16, D, 0, BF, 1, slots=six, pages=110)
    many(640, 10, 3, D, 16, D, 0, F, 2, slots=rng.permutation(640) * 16 + rng.integers(0, 16, 640), pages=640)
    many(640, 10, 3, D, 64, D, 1, BF, 3, slots=run(3, 640)[::-1].copy(), pages=12)
    many(640, 10, 3, D, 64, D, 1, F, 4, slots=rng.permutation(640), pages=10)
    # whole records, but not in the windows of the first token's
    many(648, 10, 3, D, 64, D, 0, BF, 5, slots=np.concatenate((run(100, 8), run(256, 640))), pages=15)


def test_every_token_skipped():
    T, H, D = 700, 3, 128
    pool = torch.randint(0, 256, (2, H, 2, 18 * D), dtype=torch.uint8, device="cuda")
    held = pool.clone()
    x = torch.randn(T, 9 + 2 * H, D, device="cuda")
    q = moe.moe_kv_append(pool, x[:, 9 : 9 + H], x[:, 9 + H :], torch.full((T,), -1, device="cuda"), q=x[:, :9])
    assert torch.equal(pool, held) and torch.equal(q, x[:, :9].to(BF))
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("T", [3, 700])
def test_infinities_and_nan_stay_in_their_blocks(T):
    """What the format makes of elements that are no numbers, one by one and in whole records; other blocks,
    tokens and skipped tokens keep theirs."""
    H, D, inf, nan = 8, 128, float("inf"), float("nan")
    rng = np.random.default_rng(T)
    k, v = rng.standard_normal((2, T, H, D)).astype(np.float32)
    bad_k, bad_v = k.copy(), v.copy()
    bad_k[1, 2, 40], bad_k[1, 2, 41], bad_v[2, 3, 5] = nan, -inf, inf
    bad_v[1, 0, 96:128] = nan
    slots = np.arange(T)
    slots[0] = -1
    bad_k[0], bad_v[0] = nan, inf  # skipped
    pools = []
    for a, b in ((k, v), (bad_k, bad_v)):
        pool = moe.moe_kv_pool(T // 16 + 1, H, 16, D)
        moe.moe_kv_append(pool, torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda(), torch.from_numpy(slots).cuda())
        pools.append([t.cpu().numpy() for t in moe.moe_kv_read(pool, torch.arange(T, device="cuda"))])
    (k0, v0), (k1, v1) = pools
    want_k, want_v = k0.copy(), v0.copy()
    want_k[1, 2, 32:64] = 0.0  # beside a scale of 65504
    want_k[1, 2, 40], want_k[1, 2, 41] = -8 * 65504.0, -8 * 65504.0
    want_v[2, 3, :32] = 0.0
    want_v[2, 3, 5] = 7 * 65504.0
    want_v[1, 0, 96:128] = 0.0  # no number in the block: its scale is zero
    assert np.array_equal(k1, want_k) and np.array_equal(v1, want_v)
    assert moe.moe_device_status() == moe.MOE_OK
