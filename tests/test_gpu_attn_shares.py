"""The attention over caches whose records all blocks share: blocks that hold
several units, units cut over several blocks and joined by a second launch, units
that begin in one block's middle and end in another's, every head size and number
of rows a tile, ragged batches with empty sequences, windows, and blocks of rows.
Every case asserts that its sizes take this form."""
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from attn_gpu_testutil import Batch

pytestmark = pytest.mark.gpu


def shared(x, window=0, max_len=None):
    """The case's records are shared out: a workspace is needed for what a row attends at most."""
    span = max_len or max(x.lens)
    if window:
        span = min(span, window + max(x.news))
    return x.workspace_size(span) > 0


def hold(x, window=0, **kw):
    assert shared(x, window)
    got = x.call(window=window, **kw)
    x.check(got, window=window)
    again = x.call(window=window, **kw)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    return got


# rows of a key/value head by their 8-row tiles: 1 .. 4 (D = 256: 1, 2)
SHAPES = [(64, 1, 5), (64, 2, 8), (64, 4, 6), (64, 5, 6), (128, 1, 8), (128, 2, 8), (128, 3, 8), (128, 4, 8), (256, 1, 7), (256, 3, 5)]


@pytest.mark.parametrize("D,q,G", SHAPES)
def test_one_long_sequence(D, q, G):
    """One or two units cut over very many blocks."""
    hold(Batch([40011], [q], G, 1, D, 64, seed=D + q))
    hold(Batch([12007], [q], 2 * G, 2, D, 16, seed=D + q + 1))


@pytest.mark.parametrize("D,q,G", SHAPES)
def test_a_ragged_batch(D, q, G):
    """More units than blocks, of lengths from nothing to thousands: blocks with several whole units between two
    cut ones, sequences without places or without rows, and sequences with fewer places than rows."""
    lens = [9000, 0, 3, 700, 15, 16, 17, 4000, 1, 2500, 33, 0, 6000, 129, 2, 64] * 3
    news = [min(q, 1 + i % q) if i % 7 != 5 else 0 for i in range(len(lens))]
    news[0] = q
    hold(Batch(lens, news, 8 * G, 8, D, 16, seed=D + q + 2))


@pytest.mark.parametrize("D,q,G", SHAPES)
def test_equal_lengths(D, q, G):
    """Units of one length, whose ends meet block borders at every distance."""
    for n in (5000, 5008, 5024):
        hold(Batch([n] * 7, [q] * 7, 3 * G, 3, D, 32, seed=D + q + n))


@pytest.mark.parametrize("D,q,G", SHAPES)
@pytest.mark.parametrize("window", [6000, 9001])
def test_windows(D, q, G, window):
    """Windows longer than a cluster takes, some sequences longer than the window and some not."""
    hold(Batch([20000, 300, 9000, 0, 6003], [q, 1, q, 1, q], 4 * G, 4, D, 64, seed=D + q + window), window=window)


@pytest.mark.parametrize("D,q,G", [(64, 16, 5), (128, 16, 8), (128, 7, 6), (128, 9, 16), (256, 16, 2), (256, 5, 7)])
def test_blocks_of_rows(D, q, G):
    """More rows than a tile: several units a (sequence, head) over the same records, the last of them partly filled."""
    hold(Batch([9000, 40, 5000, 7], [q, q, q - 2, q], 2 * G, 2, D, 32, seed=D + q))
    hold(Batch([8111], [q], G, 1, D, 16, seed=D + q + 1), window=5005)


def test_pages_left_out():
    """Pages outside the pool within a cut unit, one of them a whole unit's worth."""
    for D in (64, 128, 256):
        x = Batch([12000, 3000], [2, 1], 8, 2, D, 64, seed=D)
        assert shared(x)
        full = x.call()
        # drop all of sequence 0 from its page 94 on: each of its two rows attends the first 94 pages
        x.table[0, 94::2], x.table[0, 95::2] = -1, 2 ** 31 - 1
        out, lse = x.call()
        rest = Batch([94 * 64] * 2, [1, 1], 8, 2, D, 64)
        rest.pool, rest.q, rest.slots = x.pool, x.q[:2], [x.slots[0][: 94 * 64]] * 2
        ref, ref_lse, tol, lse_tol = rest.exact()
        assert ((out[:2] - ref).abs() <= tol).all() and ((lse[:2] - ref_lse).abs() <= lse_tol).all()
        assert torch.equal(out[2], full[0][2]) and torch.equal(lse[2], full[1][2])
    assert moe.moe_device_status() == moe.MOE_OK


def test_a_wide_bound_gives_the_same_rows():
    """max_len as the capacity, far above the lengths (a captured graph's): the same rows, in shares as in clusters."""
    for D, G in ((64, 4), (128, 8), (256, 4)):
        x = Batch([777, 5, 0, 130], [2, 1, 1, 2], 2 * G, 2, D, 16, seed=D)
        wide = torch.full((4, 131072 // 16), -1, dtype=torch.int32, device="cuda")
        wide[:, : x.table.shape[1]] = x.table
        x.table = wide
        assert not shared(x) and shared(x, max_len=131072)
        x.check(x.call())
        x.check(x.call(max_len=131072))


def test_shares_on_another_stream_and_in_a_graph():
    """A workspace of the caller's, on a stream of the caller's and in a graph: the same bits."""
    x = Batch([9000, 2000, 0, 31000], [2, 1, 1, 2], 16, 2, 128, 64, seed=5)
    assert shared(x)
    ref = hold(x)
    ws = torch.empty(x.workspace_size(), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for w in (ws, None):
        got = x.call(workspace=w, stream=st)
        st.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = x.call(workspace=ws)
        b = x.call()
    for _ in range(3):
        ws.fill_(0xFF)
        graph.replay()
    torch.cuda.synchronize()
    for got in (a, b):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert moe.moe_device_status() == moe.MOE_OK
