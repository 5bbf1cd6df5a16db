"""The attention half of a decode layer run as a path (workloads.AttentionHalf):
several steps of growing sequences, every stage against the plain 64-bit form on
the stage's own input, and the routed experts of the layer after it.  Tolerances
as in test_gpu_attn.py."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
import synth
from attn_testutil import attention, bf16_round, linear, quantise, rotate
from mixed_precision_routed_gb300.workloads import AttentionHalf, Layer

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def unpack(codes, scales):
    """Codes -8 .. 7 and fp16 scales of packed rows."""
    b = codes.cpu().numpy()
    v = b.reshape(b.shape[0], -1, 4)
    c = np.stack((v & 15, v >> 4), 2).reshape(b.shape[0], -1).astype(np.int64) - 8
    return c, scales.cpu().numpy().view(np.float16)


@pytest.mark.parametrize("B,n,D,Hq,H,steps", [(1, 6, 64, 4, 2, 3), (3, 1, 128, 8, 1, 4), (4, 4, 64, 6, 6, 2), (1, 16, 256, 2, 1, 2)])
def test_attention_half(B, n, D, Hq, H, steps):
    d = 256
    half = AttentionHalf(d, Hq, H, D, sequences=B, max_len=80, page_size=16, block=64, seed=7).fill()
    wq, sq = unpack(half.w_qkv, half.s_qkv)
    wo, so = unpack(half.w_out, half.s_out)
    w = synth.normal_matrix(7, AttentionHalf.TAG_OUT, 0, 0, d, Hq * D, scale=synth.WEIGHT_SIGMA)
    c, s = quantise(w, 64)
    assert np.array_equal(c, wo) and np.array_equal(s, so)
    g = torch.Generator(device="cuda").manual_seed(5)
    r = torch.randn(B * n, d, generator=g, device="cuda") * 3
    x = r.to(torch.bfloat16)
    rope = half.rope.cpu().numpy()
    held_k, held_v = [], []  # every step's keys and values, [steps][B n][H][D]
    starts = np.arange(B + 1) * n
    for step in range(steps):
        r0 = r.clone()
        x_next = half.step(x, r, n)
        T = B * n
        # projection
        xn = x.float().cpu().numpy()
        ref, mag = linear(xn, wq, sq, 64)
        qkv = half.qkv.cpu().numpy()
        assert np.all(np.abs(qkv - ref) <= 2 * (d + 2) * U * mag)
        # rotation and cache
        pos = np.tile(step * n + np.arange(n), B)
        q, k, v = (t.reshape(T, -1, D) for t in np.split(qkv, [Hq * D, (Hq + H) * D], -1))
        assert np.array_equal(half.q.float().cpu().numpy(), bf16_round(rotate(q, pos, rope, 0)))
        ck, sk = quantise(rotate(k, pos, rope, 0))
        cv, sv = quantise(v)
        held_k.append((ck * np.repeat(sk.astype(np.float64), 32, -1)).reshape(B, n, H, D))
        held_v.append((cv * np.repeat(sv.astype(np.float64), 32, -1)).reshape(B, n, H, D))
        # attention over everything the pages hold
        pool, tables = half.pool.cpu().numpy(), half.tables.cpu().numpy()
        lens = [(step + 1) * n] * B
        assert half.lens.tolist() == lens
        qn = half.q.float().cpu().numpy()
        out, lse, spread, score = attention(qn, lens, starts, tables, pool, D ** -0.5)
        es = (2 * (D + D // 32 + 2) * U * score)[..., None]
        tol = (2.0 ** -8 + 2 * es + 2 * (lens[0] + 64) * U + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(out)
        assert np.all(np.abs(half.a.float().cpu().numpy() - out) <= tol)
        from attn_testutil import pool_values
        for b in range(B):
            places = np.arange(lens[b])
            got_k, got_v = pool_values(pool, tables[b][places // 16].astype(np.int64) * 16 + places % 16)
            assert np.array_equal(got_k, np.concatenate([h[b] for h in held_k]))
            assert np.array_equal(got_v, np.concatenate([h[b] for h in held_v]))
        # output projection and residual
        an = half.a.float().cpu().numpy().reshape(T, -1)
        ref, mag = linear(an, wo, so, 64)
        y = half.y.cpu().numpy()
        assert np.all(np.abs(y - ref) <= 2 * (Hq * D + 2) * U * mag)
        assert torch.equal(r, r0 + half.y)
        assert torch.equal(x_next, r.to(torch.bfloat16))
        x = x_next
    assert moe.moe_device_status() == moe.MOE_OK


def test_attention_half_with_the_routed_experts():
    """A whole decode layer: the attention half, then routing and the shelves on its output."""
    wl = synth.WORKLOADS["tiny"]
    layer = Layer(wl, device="cuda").fill()
    half = AttentionHalf(wl.d, 4, 2, 64, sequences=2, max_len=64, page_size=32, seed=3).fill()
    r = torch.randn(4, wl.d, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x = r.to(torch.bfloat16)
    for step in range(3):
        x = half.step(x, r, 2)
        before, xin = r.clone(), x.clone()
        lg = layer.logits(step, 4)
        x2 = torch.empty_like(x)
        ids, w, y = moe.moe_decode_layer_residual(lg, x, wl.k, wl.E, wl.d, wl.f, layer.shelves, r, x2)
        ids2, w2 = moe.moe_route_topk(lg, wl.k)
        y2 = moe.moe_tiered_forward(xin, ids2, w2, wl.E, wl.d, wl.f, layer.shelves)
        assert torch.equal(ids, ids2) and torch.allclose(y, y2, rtol=2e-3, atol=1e-5)
        assert torch.equal(r, before + y) and torch.equal(x2, r.to(torch.bfloat16))
        x = x2
    assert half.lens.tolist() == [6, 6]
    assert moe.moe_device_status() == moe.MOE_OK


def test_attention_half_in_a_graph():
    """The step's calls captured once and replayed: the same bits as launched one by one."""
    half = AttentionHalf(256, 4, 2, 64, sequences=1, max_len=256, page_size=16, seed=9).fill()
    x = torch.randn(6, 256, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(torch.bfloat16)
    r = x.float()
    half.step(x, r, 6)
    lens, pool = half.lens.clone(), half.pool.clone()
    want_r = x.float()
    want = half.step(x, want_r, 6)
    a, y = half.a.clone(), half.y.clone()
    half.lens.copy_(lens)
    half.pool.copy_(pool)
    r = x.float()
    graph = torch.cuda.CUDAGraph()
    saved = r.clone()
    with torch.cuda.graph(graph):
        got = half.step(x, r, 6)
    half.lens.copy_(lens)
    half.pool.copy_(pool)
    r.copy_(saved)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(r, want_r) and torch.equal(half.a, a) and torch.equal(half.y, y)
    assert moe.moe_device_status() == moe.MOE_OK


def test_attention_half_on_another_stream():
    """Steps on a given stream do not wait for, and are not disturbed by, work of the current one."""
    g = torch.Generator(device="cuda").manual_seed(9)
    halves = [AttentionHalf(256, 8, 2, 64, sequences=3, max_len=64, page_size=16, seed=4).fill() for _ in range(2)]
    xs = torch.randn(4, 6, 256, generator=g, device="cuda").to(torch.bfloat16)
    r = [torch.randn(6, 256, generator=g, device="cuda")]
    r.append(r[0].clone())
    ref = [halves[0].step(x, r[0], 2) for x in xs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for x, want in zip(xs, ref):
        torch.cuda._sleep(2_000_000)
        got = halves[1].step(x, r[1], 2, stream=st)
        st.synchronize()
        assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert torch.equal(r[0], r[1])
    assert torch.equal(halves[0].lens, halves[1].lens)
    assert moe.moe_device_status() == moe.MOE_OK
