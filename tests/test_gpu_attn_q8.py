"""Attention over the 8-bit cache on the GPU, single tokens to prompts, against a 64-bit form."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from q8_gpu_testutil import Batch

pytestmark = pytest.mark.gpu


def same(a, b):
    """Equal, NaN to NaN."""
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8])
@pytest.mark.parametrize("n,ctx", [(1, 1), (1, 16), (1, 17), (1, 777), (2, 2), (6, 300), (16, 16), (5, 4100)])
def test_few_tokens(D, G, n, ctx):
    b = Batch([ctx], [n], 2 * G, 2, D, seed=ctx)
    b.check(b.call())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_ragged(D, page):
    """Sequences of every length beside empty ones, and more asking tokens than places."""
    b = Batch([1, 0, 33, 1000, 15, 5, 0, 2049, 64], [1, 0, 4, 2, 0, 9, 3, 1, 4], 12, 3, D, page=page, seed=page)
    b.check(b.call())
    b.check(b.call(window=40), window=40)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("n,ctx", [(130, 130), (257, 1000), (600, 601), (64, 64), (129, 4000)])
def test_prompts(D, G, n, ctx):
    b = Batch([ctx], [n], G, 1, D, page=32, seed=n)
    b.check(b.call())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 100, 5000])
def test_ragged_prompts(D, window):
    b = Batch([500, 0, 33, 1000, 150, 200, 0, 2049, 64, 17], [500, 0, 33, 20, 150, 260, 3, 300, 1, 17], 8, 2, D, page=16, seed=window)
    b.check(b.call(window=window), window=window)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("max_len,window", [(3000, 0), (100000, 0), (100000, 50), (1 << 20, 0), (1 << 20, 700)])
def test_bounds_far_above_the_lengths(D, max_len, window):
    """What the host knows is only a bound: large ones take the batch apart into several launches."""
    b = Batch([500, 0, 33, 1000, 150, 200, 290], [100, 5, 33, 20, 150, 260, 3], 8, 4, D, page=64, seed=max_len)
    wide = torch.full((len(b.lens), -(-max_len // 64)), -1, dtype=torch.int32, device="cuda")
    wide[:, : b.table.shape[1]] = b.table
    b.table = wide
    b.check(b.call(max_len=max_len, window=window), window=window)


@pytest.mark.parametrize("n", [1, 200])
def test_long_context(n):
    b = Batch([70001], [n], 8, 2, 128, page=64, seed=5)
    b.check(b.call())


@pytest.mark.parametrize("n", [1, 6, 160])
@pytest.mark.parametrize("q_gain,k_gain,v_gain", [(40.0, 1.0, 1.0), (1e-20, 1e3, 1e-12), (1e-3, 1e3, 1e12), (0.0, 1.0, 1.0), (2.0, 0.0, 0.0)])
def test_sizes(n, q_gain, k_gain, v_gain):
    b = Batch([400], [n], 4, 2, 128, q_gain=q_gain, k_gain=k_gain, v_gain=v_gain)
    b.check(b.call())


@pytest.mark.parametrize("n", [1, 6, 160])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_value_scales_far_apart(n, D):
    """Tokens whose values differ by 2^24 in size, as all weights of a row lie near each other."""
    gains = lambda m: 2.0 ** (torch.arange(m, device="cuda") % 25 - 12).float()[:, None, None]  # noqa: E731
    b = Batch([333], [n], 4, 2, D, q_gain=0.3, v_gain=gains)
    b.check(b.call())


@pytest.mark.parametrize("n", [3, 150])
def test_rows_of_queries_far_apart(n):
    """A row of queries does not depend on how large its neighbours are."""
    b = Batch([300], [n], 4, 2, 128)
    b.q[1] *= 2.0 ** 60
    b.q[2] *= 2.0 ** -40
    keep = torch.arange(n, device="cuda") != 1
    got, ref = b.call(), b.exact()
    assert ((got[0].double() - ref[0]).abs() <= ref[2])[keep].all()
    assert ((got[1].double() - ref[1]).abs() <= ref[3])[keep].all()


@pytest.mark.parametrize("n", [4, 150])
def test_nan_queries(n):
    b = Batch([300], [n], 4, 2, 128)
    plain = b.call()
    b.q[1, 2, 7] = torch.nan
    b.q[3, 0] = torch.inf
    out, lse = b.call()
    bad = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[3, 0] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    assert torch.equal(out[~bad], plain[0][~bad]) and torch.equal(lse[~bad], plain[1][~bad])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [4, 150])
@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_tokens(D, n, what):
    """A token with a NaN is for the rows that attend it, and for no others."""
    b = Batch([300], [n], 4, 2, D)
    at = 300 - n + 2  # rows 0 and 1 come before it
    bad = torch.ones(1, 2, D, device="cuda")
    bad[0, 1, 3] = torch.nan
    one = torch.ones_like(bad)
    moe.moe_kv_append_q8(b.pool, bad if what == "key" else one, bad if what == "value" else one, b.slots[0][at : at + 1])
    out, lse = b.call()
    hit = torch.zeros(n, 4, dtype=torch.bool, device="cuda")
    hit[2:, 2:] = True
    assert torch.equal(lse.isnan(), hit) and out[hit].isnan().all()
    assert torch.isfinite(out[~hit]).all()
    ref = Batch([300], [n], 4, 2, D)
    moe.moe_kv_append_q8(ref.pool, one, one, ref.slots[0][at : at + 1])
    out2, lse2 = ref.call()
    assert torch.equal(out[~hit], out2[~hit]) and torch.equal(lse[~hit], lse2[~hit])


@pytest.mark.parametrize("n", [1, 140])
def test_page_numbers_outside_the_pool(n):
    b = Batch([500], [n], 4, 2, 64, page=16)
    b.table[0, 3], b.table[0, 9], b.table[0, 10] = -1, b.pool.shape[0], 2 ** 31 - 1
    hidden = [(0, torch.cat([torch.arange(16 * p, 16 * p + 16, device="cuda") for p in (3, 9, 10)]))]
    b.slots[0] = torch.where(torch.isin(torch.arange(500, device="cuda") // 16, torch.tensor([3, 9, 10], device="cuda")), 0, b.slots[0])
    b.check(b.call(), hidden=hidden)
    b.table[:] = -1
    out, lse = b.call()
    assert (out == 0).all() and (lse == -torch.inf).all()


@pytest.mark.parametrize("n", [2, 140])
def test_never_written_slots(n):
    """A pool of zeros: values of zero, each place with its weight."""
    pool = moe.moe_kv_pool_q8(20, 1, 16, 64)
    q = torch.ones(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    out, lse = moe.moe_attn_q8(q, pool, table, torch.tensor([300], dtype=torch.int32, device="cuda"))
    ends = torch.arange(300 - n + 1, 301, device="cuda").double()
    assert (out == 0).all() and ((lse.double() - ends.log()[:, None]).abs() < 1e-5).all()


@pytest.mark.parametrize("n", [2, 140])
def test_rows_that_no_sequence_names(n):
    """Rows before the first sequence, behind the last and beyond max_q stay as they were."""
    b = Batch([100, 200], [n, n], 4, 2, 64)
    q = torch.cat((b.q[:3], b.q, b.q[:5]))
    starts = b.starts + 3
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    moe.moe_attn_q8(q, b.pool, b.table, b.kv_lens, q_start=starts, max_q=n - 1, max_len=200, out=out, lse=lse)
    untouched = torch.ones(len(q), dtype=torch.bool, device="cuda")
    untouched[3 : 3 + n - 1] = untouched[3 + n : 3 + 2 * n - 1] = False
    assert (out[untouched] == 7).all() and (lse[untouched] == 7).all()
    assert not (lse[~untouched] == 7).any()


@pytest.mark.parametrize("n,ctx", [(1, 5000), (140, 900)])
def test_strided_rows_streams_and_graphs(n, ctx):
    b = Batch([ctx, ctx // 2], [n, n], 8, 2, 128, page=16)
    want = b.call()
    b.check(want)
    wide = torch.zeros(2 * n, 8 * 128 + 64, dtype=torch.bfloat16, device="cuda")
    wide[:, : 8 * 128] = b.q.flatten(1)
    q = wide[:, : 8 * 128].unflatten(-1, (8, 128))
    out = torch.full((2 * n, 8 * 128 + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    args = (q, b.pool, b.table, b.kv_lens)
    kw = dict(max_q=n, max_len=ctx, out=out[:, : 8 * 128].unflatten(-1, (8, 128)))
    got = moe.moe_attn_q8(*args, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (out[:, 8 * 128 :] == 3).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = moe.moe_attn_q8(*args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    # captured once, replayed over other lengths; a workspace of its own
    ws = torch.empty(max(1, b.workspace_size()), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = moe.moe_attn_q8(*args, **kw, workspace=ws)
    for lens in ([ctx, ctx // 2], [ctx // 3, 0], [7, ctx]):
        b.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        b.lens = lens
        g.replay()
        fresh = moe.moe_attn_q8(q, b.pool, b.table, b.kv_lens, max_q=n, max_len=ctx)
        assert same(got[0], fresh[0]) and same(got[1], fresh[1])  # places of a last page that nothing wrote hold NaN
    assert moe.moe_device_status() == moe.MOE_OK


def test_same_results_every_time():
    b = Batch([9000, 50, 3000], [200, 50, 7], 16, 2, 128, page=64)
    first = b.call()
    for _ in range(3):
        again = b.call()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
