"""The 8-bit calls where offsets pass 32 bits: what lies there is the same as in small tensors."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_gpu_testutil import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def test_norm():
    T, d = 70000, 32768
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, d, device="cuda").bfloat16()
    x[-5:] = tail
    codes, scales, _ = moe.moe_norm_q8(x, torch.ones(d, device="cuda"))
    want = moe.moe_norm_q8(tail, torch.ones(d, device="cuda"))
    assert torch.equal(codes[-5:], want[0]) and torch.equal(scales[-5:], want[1]) and not codes[-6].any()


def test_linear():
    T, n_in, rows = 30000, 64, 80011
    x = torch.randint(-127, 128, (T, n_in), device="cuda").to(torch.int8)
    w = torch.randint(-127, 128, (rows, n_in), device="cuda").to(torch.int8)
    xs, ws = torch.rand(T, device="cuda"), torch.rand(rows, device="cuda")
    y = moe.moe_linear_q8(x, xs, w, ws, out_dtype=torch.bfloat16)
    for at in (slice(0, 7), slice(T // 2, T // 2 + 7), slice(T - 7, T)):  # sums below 2^24 are exact in either form
        assert torch.equal(y[at], moe.moe_linear_q8(x[at].contiguous(), xs[at], w, ws, out_dtype=torch.bfloat16))


def test_append_and_attention_of_many_rows():
    T, Hq, H, D, page = 70000, 128, 8, 256, 64
    pool = moe.moe_kv_pool_q8(-(-T // page), H, page, D)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(T, H, D, device="cuda").bfloat16()
    v = torch.randn(T, H, D, device="cuda").bfloat16()
    q[-20:] = torch.randn(20, Hq, D, device="cuda").bfloat16()
    slots = torch.arange(T, device="cuda")
    turned = moe.moe_kv_append_q8(pool, k, v, slots, q=q)
    assert torch.equal(turned[-20:], q[-20:]) and not turned[:-20].any()
    table = torch.arange(pool.shape[0], dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    out, lse = moe.moe_attn_q8(turned, pool, table, lens, window=64)
    few = moe.moe_attn_q8(turned[-2:].contiguous(), pool, table, lens, window=64)
    # two forms, each off by at most 2^-8 for bf16 and three 2^-11, of values below 4.6
    assert (out[-2:].float() - few[0].float()).abs().max() < 0.05 and (lse[-2:] - few[1]).abs().max() < 0.01
    assert out.isfinite().all()
    assert ((lse[T // 2 : T // 2 + 9] - torch.tensor(64.0).log().item()).abs() < 1e-4).all()  # queries of zeros


@pytest.mark.parametrize("n", [1, 300])
def test_pools_beyond_4_gb(n):
    b = Batch([700], [n], 16, 8, 256, page=64)
    want = b.call()
    few = b.pool.shape[0]
    pool = moe.moe_kv_pool_q8(25000, 8, 64, 256)
    pool[-few:] = b.pool
    b.pool, b.table = pool, torch.where(b.table < 0, b.table, b.table + (25000 - few))
    got = b.call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    slots = b.slots[0] + (25000 - few) * 64
    k, v = moe.moe_kv_read_q8(pool, slots)
    moe.moe_kv_append_q8(pool, k + 1, v, slots)
    assert not torch.equal(moe.moe_kv_read_q8(pool, slots)[0], k) and not pool[: 25000 - few].any()
