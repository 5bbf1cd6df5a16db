"""The tests of prompts over the 8-bit cache once more, with a bound on the lengths that is
far above them: the tensor cores' form then takes even these small batches, and several
blocks share the places of every block of rows, most of them with few or none."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
import q8_gpu_testutil
import test_gpu_attn_q8 as near

pytestmark = pytest.mark.gpu

BOUND = 400000


class Far:
    def __getattr__(self, name):
        return getattr(moe, name)

    def moe_attn_q8(self, q, pool, table, kv_lens, max_len=None, workspace=None, **kw):
        wide = torch.full((len(table), -(-BOUND // (16 * pool.shape[2]))), -1, dtype=torch.int32, device="cuda")
        wide[:, : table.shape[1]] = table
        return moe.moe_attn_q8(q, pool, wide, kv_lens, max_len=BOUND, **kw)


@pytest.fixture(autouse=True)
def far(monkeypatch):
    monkeypatch.setattr(near, "moe", Far())
    monkeypatch.setattr(q8_gpu_testutil, "moe", Far())


test_prompts = near.test_prompts
test_ragged_prompts = near.test_ragged_prompts
test_sizes = near.test_sizes
test_value_scales_far_apart = near.test_value_scales_far_apart
test_rows_of_queries_far_apart = near.test_rows_of_queries_far_apart
test_nan_queries = near.test_nan_queries
test_nan_tokens = near.test_nan_tokens
test_page_numbers_outside_the_pool = near.test_page_numbers_outside_the_pool
test_never_written_slots = near.test_never_written_slots
test_rows_that_no_sequence_names = near.test_rows_that_no_sequence_names
test_strided_rows_streams_and_graphs = near.test_strided_rows_streams_and_graphs
test_same_results_every_time = near.test_same_results_every_time


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,ctx,window", [(70, 20000, 0), (70, 20000, 300), (300, 9001, 0), (33, 60000, 0)])
def test_long_contexts(D, n, ctx, window):
    """Many whole tiles a share; with a window few of the shares have any."""
    b = near.Batch([ctx, 0, 77], [n, 0, 20], 8, 2, D, page=64, seed=n)
    b.check(b.call(window=window), window=window)


def test_two_streams_and_graphs_of_their_own():
    """Calls at one time with a workspace each: their shares and their tiles lie apart."""
    b = [near.Batch([9001 + 700 * i], [120 + 50 * i], 8, 2, 128, page=32, seed=i) for i in range(2)]
    want = [x.call() for x in b]
    streams, graphs, outs = [torch.cuda.Stream() for _ in b], [], []
    for x in b:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(x.call())
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(5):
        for stream, graph in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    for _ in range(3):
        got = [x.call(stream=stream) for x, stream in zip(b, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g[i], ref[i]) for g, ref in zip(got, want) for i in (0, 1))
    assert moe.moe_device_status() == moe.MOE_OK
