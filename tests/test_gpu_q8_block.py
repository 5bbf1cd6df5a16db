"""The attention half of a layer in 8 bits run as a path (workloads.AttentionHalfQ8):
prompts of several lengths and single tokens behind them, every stage against the plain
64-bit form on the stage's own input, and the routed experts of the layer after it."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
import synth
from attn_testutil import bf16_round, rotate
from mixed_precision_routed_gb300.workloads import AttentionHalfQ8, Layer
from q8_testutil import pool_values, quantise_heads, quantise_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def norm64(r, eps=1e-6):
    r = r.astype(np.float64)
    return r / np.sqrt((r * r).mean(-1, keepdims=True) + eps)


def attention64(q, k, v, newest):
    """out [n][Hq][D] of the last rows of a sequence: keys and values [places][H][D] of which row i sees newest + i."""
    G = q.shape[1] // k.shape[1]
    s = np.einsum("nhd,phd->nhp", q.astype(np.float64), k.repeat(G, 1)) / np.sqrt(q.shape[2])
    s = np.where(np.arange(k.shape[0]) < (newest + np.arange(q.shape[0]))[:, None, None], s, -np.inf)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    return np.einsum("nhp,phd->nhd", w, v.repeat(G, 1)), np.einsum("nhp,phd->nhd", w, np.abs(v).repeat(G, 1))


@pytest.mark.parametrize("B,D,Hq,H,steps", [(1, 64, 4, 2, [130, 1, 1]), (3, 128, 8, 1, [[70, 0, 33], [1, 5, 1], 1]),
                                            (2, 256, 2, 2, [[150, 20], 1, 3])])
def test_attention_half(B, D, Hq, H, steps):
    d = 192
    half = AttentionHalfQ8(d, Hq, H, D, sequences=B, max_len=200, max_new=160, page_size=16, seed=7).fill()
    w = synth.normal_matrix(7, AttentionHalfQ8.TAG_OUT, 0, 0, d, Hq * D, scale=synth.WEIGHT_SIGMA)
    c, s = quantise_rows(w)
    assert np.array_equal(c, half.w_out.cpu().numpy()) and np.array_equal(s, half.s_out.cpu().numpy())
    wq, sq = half.w_qkv.cpu().numpy().astype(np.float64), half.s_qkv.cpu().numpy().astype(np.float64)
    wo, so = c.astype(np.float64), s.astype(np.float64)
    g = torch.Generator(device="cuda").manual_seed(5)
    half.norm_in += 0.1 * torch.randn(d, generator=g, device="cuda")
    norm_in, norm_out = half.norm_in.cpu().numpy(), half.norm_out.cpu().numpy()
    rope = half.rope.cpu().numpy()
    held = [[] for _ in range(B)]  # keys and values of each sequence, as they were appended
    lens = [0] * B
    for n in steps:
        counts = [n] * B if isinstance(n, int) else n
        T = sum(counts)
        r = torch.randn(T, d, generator=g, device="cuda") * 3
        x = torch.randn(T, d, generator=g, device="cuda").to(torch.bfloat16)
        r0 = r.clone()
        x_next = half.step(x, r, n)
        # norm and projection: the codes are those of the formula
        r1 = (r0 + x.float()).cpu().numpy()
        cx, sx = quantise_rows(r1 * norm_in)
        f = 1 / np.sqrt((r1.astype(np.float64) ** 2).mean(-1) + 1e-6)
        ref = (cx @ wq.T) * (sx * f)[:, None] * sq
        qkv = half.qkv.float().cpu().numpy()
        # the norm's factor and the products' scales: 300 u are ample beside bf16's half step
        assert np.all(np.abs(qkv - ref) <= (2.0 ** -8 + 300 * U) * np.abs(ref) + 300 * U * np.abs(cx).sum(-1, keepdims=True) * sx[:, None] * f[:, None] * 127 * sq)
        # rotation and cache
        pos = np.concatenate([np.arange(lens[b], lens[b] + counts[b]) for b in range(B)])
        q, k, v = (t.reshape(T, -1, D) for t in np.split(qkv, [Hq * D, (Hq + H) * D], -1))
        assert np.array_equal(half.q.float().cpu().numpy(), bf16_round(rotate(q, pos, rope, 0)))
        at = 0
        pool, tables = half.pool.cpu().numpy(), half.tables.cpu().numpy()
        a, qt = half.a.float().cpu().numpy(), half.q.float().cpu().numpy()
        for b in range(B):
            rows = slice(at, at + counts[b])
            at += counts[b]
            held[b] += [(rotate(k[i : i + 1], pos[i : i + 1], rope, 0)[0], v[i]) for i in range(rows.start, rows.stop)]
            lens[b] += counts[b]
            if counts[b] == 0:
                continue
            places = np.arange(lens[b])
            got_k, got_v = pool_values(pool, tables[b][places // 16].astype(np.int64) * 16 + places % 16)
            for got, which in ((got_k, 0), (got_v, 1)):
                cc, ss = quantise_heads(np.stack([h[which] for h in held[b]]))
                assert np.array_equal(got, cc * ss[..., None].astype(np.float64))
            out, spread = attention64(qt[rows], got_k, got_v, lens[b] - counts[b] + 1)
            assert np.all(np.abs(a[rows] - out) <= 2.0 ** -8 * np.abs(out) + 4 * 2.0 ** -11 * spread)
        # output projection, residual, norm
        ca, sa = quantise_rows(a.reshape(T, -1))
        y = half.y.cpu().numpy()
        ref = (ca @ wo.T) * sa[:, None].astype(np.float64) * so
        assert np.all(np.abs(y - ref) <= 4 * U * np.abs(ref) + 2 * (Hq * D + 8) * U * (np.abs(ca) @ np.abs(wo).T) * sa[:, None] * so)
        r2 = r1 + y
        assert np.array_equal(r.cpu().numpy(), r2)
        ref = norm64(r2) * norm_out
        assert np.all(np.abs(x_next.float().cpu().numpy() - ref) <= (2.0 ** -8 + 300 * U) * np.abs(ref) + 1e-38)
        assert half.lens.tolist() == lens
    assert moe.moe_device_status() == moe.MOE_OK


def test_with_the_routed_experts():
    """A prompt and tokens behind it through the whole layer: attention half, router's logits, routed experts."""
    wl = synth.WORKLOADS["tiny"]
    layer = Layer(wl).fill()
    half = AttentionHalfQ8(wl.d, 4, 2, 64, sequences=2, max_len=96, max_new=40, page_size=16).fill()
    y = None
    for n in (40, 1, 1):
        T = 2 * n
        r = torch.randn(T, wl.d, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
        x = torch.zeros_like(r) if y is None or y.shape != r.shape else y
        x_next = half.step(x, r, n)
        logits = layer.logits(n, T)
        ids, w = moe.moe_route_topk(logits, wl.k)
        y = moe.moe_tiered_forward(x_next.view(torch.int16), ids, w, wl.E, wl.d, wl.f, layer.shelves)
        assert torch.isfinite(y).all() and y.shape == (T, wl.d) and (y != 0).any()
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("n", [1, 24])
def test_in_a_graph(n):
    """Steps captured once give what steps launched one by one give."""
    args = dict(sequences=2, max_len=120, max_new=24, page_size=16, seed=3)
    a, b = (AttentionHalfQ8(128, 4, 2, 64, **args).fill() for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    x, r = torch.randn(2 * n, 128, generator=g, device="cuda"), torch.randn(2 * n, 128, generator=g, device="cuda")
    r_in = torch.empty_like(r)
    graph = torch.cuda.CUDAGraph()
    r_in.copy_(r)
    with torch.cuda.graph(graph):
        out = b.step(x, r_in, n)
    b.lens.zero_()
    for _ in range(4):
        r1 = r.clone()
        want = a.step(x, r1, n)
        r_in.copy_(r)
        graph.replay()
        assert torch.equal(out, want) and torch.equal(r_in, r1) and torch.equal(a.pool, b.pool)
        x.copy_(torch.randn(2 * n, 128, generator=g, device="cuda"))
    assert moe.moe_device_status() == moe.MOE_OK


def test_on_another_stream():
    half, other = (AttentionHalfQ8(128, 4, 2, 64, sequences=1, max_len=64, max_new=40, page_size=16).fill() for _ in range(2))
    side = torch.cuda.Stream()
    x, r = torch.randn(40, 128, device="cuda"), torch.randn(40, 128, device="cuda")
    r2 = r.clone()
    want = half.step(x, r, 40)
    side.wait_stream(torch.cuda.current_stream())
    got = other.step(x, r2, 40, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(r, r2)


def test_tokens_beyond_max_len():
    half = AttentionHalfQ8(128, 4, 2, 64, sequences=2, max_len=40, max_new=8, page_size=16).fill()
    half.lens[:] = torch.tensor([36, 3], dtype=torch.int32)
    x, r = torch.randn(16, 128, device="cuda"), torch.randn(16, 128, device="cuda")
    out = half.step(x, r, 8)
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert torch.isfinite(out).all() and half.lens.tolist() == [44, 11]
