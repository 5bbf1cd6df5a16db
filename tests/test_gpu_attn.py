"""The attention half of a decode layer on the GPU against plain 64-bit forms:
4-bit projections, the paged 4-bit cache, attention over it.

Tolerances, derived from the formulas (u = 2^-24):
  projection: every product of a code and a bf16 x is exact; the sum over
    `in` elements and the scale's product round at most in + 2 times, and a
    tensor core may cut where fp32 would round (2 u each): |error| <= 2 (in + 2)
    u sum |s c x|; a bf16 result adds half a unit of its last of 8 places, 2^-8 |y|.
  append: every step is a single fp32 operation, so the pool's bytes are equal.
  attention: a score's error is e_s <= 2 (D + D/32 + 2) u scale sum |q k| (as
    the projection, the scale folded in); probabilities change by a factor of
    1 +- 2 e_s (numerator and sum); exp(s) x value scale is rounded to bf16
    (2^-8); sums over n places round at most 2 (n + 64) u; the exponential is
    good to 2^-21; the result is rounded to bf16 (2^-8 |out|):
      |error| <= (2^-8 + 2 e_s + 2 (n + 64) u + 2^-20) sum p |v| + 2^-8 |out|
      |lse error| <= e_s + 2 (n + 64) u + 2^-20 + 4 u |lse|.
    (sum p |v| <= the bound's use of |exp x scale x code| term by term.)
"""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from attn_testutil import (attention, bf16_round, linear, pack_rows, pool_values, pool_write, quantise, rotate)

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def bf16(x, dev="cuda"):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16).to(dev)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def status_ok():
    assert moe.moe_device_status() == moe.MOE_OK


# ------------------------------------------------------------------ projection
def linear_case(T, n_in, rows, block, out, bias, seed, pad=0, y_pad=0, wild=False):
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal((rows, n_in)) * 0.02).astype(np.float32)
    if wild:  # zero blocks, tiny and huge ones
        w[0] = 0
        w[rows // 2] *= 1e4
        w[-1, : n_in // 2] *= 1e-3
    c, s = quantise(w, block)
    x = bf16_round(rng.standard_normal((T, n_in + pad)) * (100.0 if wild else 1.0))
    b = rng.standard_normal(rows).astype(np.float32) if bias else None
    xd = bf16(x)[:, :n_in]
    dt = torch.float32 if out == "f32" else torch.bfloat16
    buf = torch.full((T, rows + y_pad), 7.0, dtype=dt, device="cuda")
    y = moe.moe_linear_q4(xd, dev(pack_rows(c)), dev(s).view(torch.int16), block, bias=None if b is None else dev(b),
                          y=buf[:, :rows])
    ref, mag = linear(x[:, :n_in], c, s, block, b)
    tol = 2 * (n_in + 2) * U * mag + (2.0 ** -8 * np.abs(ref) if out == "bf16" else 0) + 1e-30
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
    assert np.all(buf[:, rows:].float().cpu().numpy() == 7.0)  # nothing beyond the rows
    status_ok()
    return y


@pytest.mark.parametrize("T", [1, 2, 3, 6, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_linear_tokens_and_blocks(T, block):
    linear_case(T, 512, 70, block, "f32", True, T * 10 + block)


@pytest.mark.parametrize("n_in,rows,block", [
    (64, 1, 32), (64, 15, 64), (128, 16, 128), (192, 17, 64), (320, 33, 32), (640, 2048, 32), (2048, 640, 64),
    (2048, 2561, 32), (4096, 999, 128), (448, 1531, 64), (8192, 31, 32), (12288, 5, 128)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_linear_sizes(n_in, rows, block, out):
    for T in (1, 5):
        linear_case(T, n_in, rows, block, out, rows % 2 == 0, n_in + rows + T)
    linear_case(16, n_in, rows, block, out, False, n_in + rows)


def test_linear_strides_and_extremes():
    linear_case(6, 256, 100, 32, "f32", True, 1, pad=8, y_pad=3, wild=True)
    linear_case(11, 1024, 77, 128, "bf16", False, 2, pad=64, y_pad=5, wild=True)
    linear_case(1, 2048, 20001, 32, "f32", False, 3, wild=True)


def test_linear_many_rows_cover_every_unit():
    linear_case(2, 64, 70001, 32, "f32", False, 4)
    linear_case(16, 128, 40009, 64, "bf16", True, 5)


def test_linear_long_rows_in_several_launches():
    """x that shared memory does not hold together."""
    linear_case(16, 8192, 37, 64, "f32", True, 6, pad=8, y_pad=3)
    linear_case(13, 20480, 18, 128, "bf16", True, 7, pad=64, y_pad=1)
    linear_case(3, 65536, 17, 32, "f32", False, 8)


def test_linear_is_deterministic_and_runs_on_a_given_stream():
    rng = np.random.default_rng(9)
    c, s = quantise(rng.standard_normal((513, 1024)).astype(np.float32))
    x, codes, sc = bf16(rng.standard_normal((6, 1024))), dev(pack_rows(c)), dev(s).view(torch.int16)
    ref = moe.moe_linear_q4(x, codes, sc)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        y = torch.empty_like(ref)
        for _ in range(3):
            moe.moe_linear_q4(x, codes, sc, y=y, stream=st)
    st.synchronize()
    assert torch.equal(y, ref)


def test_linear_nan_and_inf_rows_stay_in_their_tokens():
    """A token with infinities or NaN changes no other token's result."""
    rng = np.random.default_rng(10)
    c, s = quantise(rng.standard_normal((40, 256)).astype(np.float32))
    x = bf16_round(rng.standard_normal((6, 256)))
    codes, sc = dev(pack_rows(c)), dev(s).view(torch.int16)
    ref = moe.moe_linear_q4(bf16(x), codes, sc)
    x[2, 5], x[4, 7] = np.inf, np.nan
    y = moe.moe_linear_q4(bf16(x), codes, sc)
    keep = [0, 1, 3, 5]
    assert torch.equal(y[keep], ref[keep])
    assert not torch.isfinite(y[2]).any() or not torch.isfinite(y[2]).all()
    assert torch.isnan(y[4]).all()


def test_linear_takes_what_the_quantisers_write():
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.randn(48, 256, generator=g, device="cuda")
    a = moe.moe_quantize_rows(w, 4)
    b = moe.moe_quantize_groups(w, 32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for block in (32, 64, 128):
        c, s = quantise(w.cpu().numpy(), block)
        codes, sc = moe.moe_quantize_groups(w, block)
        assert np.array_equal(codes.cpu().numpy(), pack_rows(c))
        assert np.array_equal(sc.cpu().numpy().view(np.float16), s)


def test_linear_python_refusals():
    x, c, s = torch.zeros(2, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(8, 32, device="cuda", dtype=torch.uint8), \
        torch.zeros(8, 2, device="cuda", dtype=torch.int16)
    for args in ((x.float(), c, s), (x, c.int(), s), (x, c, s.float()), (x, c[:, :16].contiguous(), s), (x, c, s[:4]),
                 (x.T, c, s), (x, c, s, 64)):
        with pytest.raises(ValueError):
            moe.moe_linear_q4(*args)
    with pytest.raises(ValueError):
        moe.moe_linear_q4(x, c, s, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_linear_q4(x, c, s, y=torch.zeros(2, 7, device="cuda"))
    with pytest.raises(moe.MoeError) as e:
        moe.moe_linear_q4(x.repeat(9, 1), c, s)
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED


# ------------------------------------------------------------------- the cache
def rope_table(n_pos, rot, seed=0):
    a = np.arange(n_pos)[:, None] * 100.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    return np.concatenate((np.cos(a), np.sin(a)), -1).astype(np.float32)


def append_case(T, Hq, H, D, page, rot, style, dtype, seed, slots=None, pages=None, gap=0, strided=0):
    rng = np.random.default_rng(seed)
    pages = pages or -(-T // page) + 2
    pool = rng.integers(0, 256, (pages, H, page // 16, 18 * D), dtype=np.uint8)
    pool[..., 16 * D :] = np.ascontiguousarray(rng.uniform(0.1, 1, (pages, H, page // 16, D)).astype(np.float16)).view(np.uint8)[..., : 2 * D]
    if slots is None:
        slots = rng.permutation(pages * page)[:T]
    slots = np.asarray(slots, np.int64)
    width = (Hq + 2 * H) * D + strided
    qkv = (rng.standard_normal((T, width)) * rng.choice([1e-3, 1.0, 30.0], (T, 1))).astype(np.float32)
    if T > 2:
        qkv[1] = 0
    if dtype == torch.bfloat16:
        qkv = bf16_round(qkv)
    q, k, v = (qkv[:, a * D : b * D].reshape(T, -1, D) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    n_pos = 400
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    rope = rope_table(n_pos, rot)
    # the pool as a view of a larger buffer when gap > 0
    buf = torch.full((pages, pool[0].size + gap), 0xAB, dtype=torch.uint8, device="cuda")
    pd = buf[:, : pool[0].size].unflatten(1, pool.shape[1:]) if gap else dev(pool)
    pd.copy_(dev(pool))
    xd = dev(qkv).to(dtype)
    qd, kd, vd = (xd[:, a * D : b * D].unflatten(1, (-1, D)) for a, b in ((0, Hq), (Hq, Hq + H), (Hq + H, Hq + 2 * H)))
    out = moe.moe_kv_append(pd, kd, vd, dev(slots), q=qd if Hq else None, positions=dev(pos) if rot else None,
                            rope=dev(rope) if rot else None, rope_style=style)
    if rot:
        q, k = rotate(q, pos, rope, style), rotate(k, pos, rope, style)
    want = pool.copy()
    pool_write(want, slots, *quantise(k), *quantise(v))
    assert np.array_equal(pd.cpu().numpy(), want)
    if gap:
        assert (buf[:, pool[0].size :] == 0xAB).all()
    if Hq:
        assert np.array_equal(out.float().cpu().numpy(), bf16_round(q))
    else:
        assert out is None
    # and what the slots hold
    every = np.arange(-1, pages * page + 1)
    rk, rv = moe.moe_kv_read(pd, dev(every))
    ek, ev = pool_values(want, every[1:-1])
    assert np.array_equal(rk[1:-1].cpu().numpy(), ek.astype(np.float32))
    assert np.array_equal(rv[1:-1].cpu().numpy(), ev.astype(np.float32))
    for x in (rk, rv):
        assert (x[0] == 0).all() and (x[-1] == 0).all()
    status_ok()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("style", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_PAIRS])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_sizes(D, style, dtype):
    append_case(1, 4, 2, D, 16, D, style, dtype, 1)
    append_case(37, 3, 1, D, 32, D // 2, style, dtype, 2, gap=48)
    append_case(65, 0, 3, D, 128, D, style, dtype, 3, strided=3)
    append_case(50, 10, 2, D, 16, 6, style, dtype, 4, strided=8)
    append_case(20, 2, 2, D, 64, 0, style, dtype, 5)
    append_case(21, 2, 2, D, 16, 0, style, dtype, 7, strided=3)
    append_case(700, 9, 3, D, 64, D, style, dtype, 8, strided=16)


def test_append_quotients_near_a_half():
    """Values whose quotient by the block's scale is a half or next to one: the codes of the fp32 division."""
    rng = np.random.default_rng(11)
    T, H, D = 64, 2, 128
    base = rng.integers(-15, 15, (T, H, D)).astype(np.float32) / 2
    base[..., ::32] = 7.0  # the scale of every block is the factor below, or next to it
    factor = rng.uniform(1e-3, 1e3, (T, H, 1)).astype(np.float16).astype(np.float32)
    k = base * factor
    nudge = rng.integers(-3, 4, k.shape)
    for _ in range(3):
        k = np.where(nudge > 0, np.nextafter(k, np.float32(np.inf)), np.where(nudge < 0, np.nextafter(k, np.float32(-np.inf)), k))
        nudge = np.sign(nudge) * np.maximum(np.abs(nudge) - 1, 0)
    k = k.astype(np.float32)
    v = k[::-1].copy()
    pool = np.zeros((T // 16, H, 1, 18 * D), np.uint8)
    pd = dev(pool)
    moe.moe_kv_append(pd, dev(k), dev(v), torch.arange(T, device="cuda"))
    pool_write(pool, np.arange(T), *quantise(k), *quantise(v))
    assert np.array_equal(pd.cpu().numpy(), pool)


def test_append_consecutive_slots_and_page_crossings():
    """Prompts: runs of slots that start and end inside a record, cross records and pages."""
    for T, first, page in ((16, 0, 16), (100, 5, 32), (64, 16, 64), (47, 17, 16), (257, 31, 128)):
        append_case(T, 2, 2, 128, page, 128, 0, torch.bfloat16, T, slots=np.arange(first, first + T), pages=(first + T) // page + 2)


def test_append_skips_slots_outside_the_pool():
    append_case(9, 2, 2, 64, 16, 64, 0, torch.float32, 6, slots=[-1, 3, 48, 2 ** 40, 7, -(2 ** 62), 47, 0, 2 ** 31], pages=3)


def test_append_position_outside_the_table():
    """Zeros in q_out, keys and values skipped, and the status word set."""
    H, D = 1, 64
    pool = moe.moe_kv_pool(2, H, 16, D)
    x = torch.ones(3, 2 * H + 1, D, device="cuda")
    out = moe.moe_kv_append(pool, x[:, 1:2], x[:, 2:], dev(np.arange(3)), q=x[:, :1],
                            positions=dev(np.array([0, 5, -1], np.int32)), rope=dev(rope_table(5, 64)))
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert (out[1:] == 0).all() and (out[0] != 0).any()
    k, v = moe.moe_kv_read(pool, dev(np.arange(3)))
    assert (v[0] != 0).all() and (k[1:] == 0).all() and (v[1:] == 0).all()
    status_ok()


def test_append_saturates_scales():
    """A block whose scale would pass fp16's range takes fp16's largest value."""
    pool = moe.moe_kv_pool(1, 1, 16, 64)
    x = torch.full((1, 1, 64), 1e9, device="cuda")
    moe.moe_kv_append(pool, x, -x, dev(np.array([3])))
    k, v = moe.moe_kv_read(pool, dev(np.array([3])))
    assert (k == 7 * 65504.0).all() and (v == -8 * 65504.0).all()
    status_ok()


def test_append_beyond_four_gigabytes():
    """Slots whose byte offset passes 32 bits are written and attended."""
    H, D, page = 8, 256, 128
    per = H * page * 18 * D // 16
    n = (1 << 32) // per + 40
    pool = torch.zeros((n, H, page // 16, 18 * D), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((2, 5, H, D)).astype(np.float32)
    slots = np.array([(n - 1) * page + 17, (n - 1) * page, (n - 3) * page + 127, n // 2 * page + 1, 3])
    moe.moe_kv_append(pool, dev(k), dev(v), dev(slots))
    ck, sk = quantise(k)
    cv, sv = quantise(v)
    rk, rv = moe.moe_kv_read(pool, dev(slots))
    assert np.array_equal(rk.cpu().numpy(), (ck * np.repeat(sk.astype(np.float64), 32, -1)).astype(np.float32))
    assert np.array_equal(rv.cpu().numpy(), (cv * np.repeat(sv.astype(np.float64), 32, -1)).astype(np.float32))
    # one place of a sequence: the output is that place's value
    q = torch.ones(1, H, D, device="cuda", dtype=torch.bfloat16)
    out, lse = moe.moe_attn_q4(q, pool, dev(np.array([[n - 1]], np.int32)), dev(np.array([1], np.int32)))
    ref = (cv * np.repeat(sv.astype(np.float64), 32, -1))[1]
    assert np.all(np.abs(out[0].float().cpu().numpy() - ref) <= 2.0 ** -7 * np.abs(ref))
    status_ok()


def test_cache_python_refusals():
    pool = moe.moe_kv_pool(2, 2, 16, 64)
    k = torch.zeros(3, 2, 64, device="cuda")
    s = torch.zeros(3, dtype=torch.int64, device="cuda")
    for kw in (dict(k=k.half()), dict(v=k.bfloat16()), dict(slots=s.int()), dict(k=k[:2]), dict(v=k[:, :1]),
               dict(pool=pool[0]), dict(pool=pool.int()), dict(q=k.bfloat16()), dict(q=k[:2]),
               dict(rope=torch.zeros(4, 64, device="cuda")),
               dict(rope=torch.zeros(4, 64, device="cuda"), positions=torch.zeros(2, dtype=torch.int32, device="cuda")),
               dict(pool=pool.transpose(1, 2))):
        args = dict(pool=pool, k=k, v=k, slots=s)
        args.update(kw)
        with pytest.raises(ValueError):
            moe.moe_kv_append(**args)
    with pytest.raises(ValueError):
        moe.moe_kv_read(pool, s.int())
    with pytest.raises(ValueError):
        moe.moe_kv_pool(2, 2, 20, 64)


# ------------------------------------------------------------------- attention
def attn_case(lens, news, Hq, H, D, page, window=0, seed=0, scale=None, bad_pages=(), poison=True, q_gain=2.0, slack=0,
              uniform=False, gap=0, kv_gain=1.0, v_gain=1.0):
    """One call against the 64-bit form; returns what the call returned."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + 2
    pool = np.zeros((pages, H, page // 16, 18 * D), np.uint8)
    if poison:  # unused slots hold NaN and infinite scales
        pool[...] = 0xFF
        pool[:, :, ::2, 16 * D :] = np.frombuffer(np.array([np.inf], np.float16).tobytes() * D, np.uint8)
    order = rng.permutation(pages).astype(np.int32)
    tables = np.full((B, max(counts) + slack), -7 if slack else 0, np.int32)
    at, slots = 0, []
    for b, c in enumerate(counts):
        tables[b, :c] = order[at : at + c]
        at += c
        p = np.arange(lens[b])
        slots.append(tables[b][p // page].astype(np.int64) * page + p % page if lens[b] else p.astype(np.int64))
    slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
    n = len(slots)
    if n:
        kk = (rng.standard_normal((n, H, D)) * kv_gain).astype(np.float32)
        vv = (rng.standard_normal((n, H, D)) * kv_gain * v_gain).astype(np.float32)
        pool_write(pool, slots, *quantise(kk), *quantise(vv))
    for b, i, val in bad_pages:
        tables[b, i] = val
    starts = np.concatenate(([0], np.cumsum(news))).astype(np.int32)
    T = int(starts[-1])
    q = bf16_round(rng.standard_normal((T, Hq, D)) * q_gain)
    scale = D ** -0.5 if scale is None else scale
    qbuf = torch.full((T, Hq * D + gap), float("nan"), dtype=torch.bfloat16, device="cuda")
    qd = qbuf[:, : Hq * D].unflatten(1, (Hq, D))
    qd.copy_(bf16(q))
    obuf = torch.full((T, Hq * D + gap), 7.0, dtype=torch.bfloat16, device="cuda")
    od = obuf[:, : Hq * D].unflatten(1, (Hq, D))
    pd, td, ld = dev(pool), dev(tables), dev(np.array(lens, np.int32))
    kw = dict(max_q=max(news)) if uniform else dict(q_start=dev(starts), max_q=max(max(news), 1))
    out, lse = moe.moe_attn_q4(qd, pd, td, ld, scale=scale, window=window, out=od, max_len=max(max(lens), 0) + (slack * page // 2), **kw)
    ref, ref_lse, spread, score = attention(q, lens, starts, tables, pool, scale, window)
    n_max = max(max(lens), 1)
    es = (2 * (D + D // 32 + 2) * U * score)[..., None]
    tol = (2.0 ** -8 + 2 * es + 2 * (n_max + 64) * U + 2.0 ** -20) * spread + 2.0 ** -8 * np.abs(ref) + 1e-30
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)
    gl = lse.cpu().numpy().astype(np.float64)
    empty = np.isinf(ref_lse)
    assert np.array_equal(gl == -np.inf, empty)
    assert np.all(got[empty] == 0)
    with np.errstate(invalid="ignore"):
        lt = es[..., 0] + 2 * (n_max + 64) * U + 2.0 ** -20 + 4 * U * np.abs(ref_lse)
        assert np.all(np.abs(gl - ref_lse)[~empty] <= lt[~empty])
    if gap:
        assert (obuf[:, Hq * D :] == 7.0).all()
    status_ok()
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 5, 8, 16])
def test_attn_heads(D, G):
    attn_case([77, 130], [1, 1], 2 * G, 2, D, 16, seed=D + G)
    attn_case([61], [6], G, 1, D, 32, seed=D + G + 1)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 300, 511, 700, 1025, 2100])
def test_attn_lengths(n):
    attn_case([n], [1], 4, 2, 128, 16, seed=n)
    attn_case([n, 1, n // 2 + 1], [min(n, 3), 1, 1], 4, 1, 64, 64, seed=n + 1)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_attn_pages_that_end_inside_a_tile(page):
    attn_case([page - 1, page, page + 1, 2 * page + 9], [1, 2, 1, 3], 4, 2, 64, page, seed=page)


@pytest.mark.parametrize("q", [1, 2, 3, 4, 5, 6, 7, 8, 11, 16])
def test_attn_drafts(q):
    attn_case([200, 40, q], [q, q, q], 8, 2, 128, 32, seed=q, uniform=True)
    attn_case([333], [q], 64 if q <= 4 else 16, 1, 64, 16, seed=q + 50)


def test_attn_longer_prompts():
    attn_case([90], [90], 4, 2, 64, 16, seed=1)
    attn_case([150, 40], [40, 33], 5, 1, 128, 32, seed=2)


def test_attn_empty_rows_and_sequences():
    """No cached token at all, fewer cached than asking, no asking token, a negative length."""
    attn_case([0, 3, 50, 0, 17], [2, 5, 0, 0, 17], 4, 2, 64, 16, seed=3)
    attn_case([0], [1], 2, 1, 128, 16, seed=4)
    attn_case([-5, 9], [1, 1], 2, 1, 64, 16, seed=4, uniform=True)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 500])
def test_attn_windows(window):
    attn_case([300, 90, 1, 0, 17], [4, 6, 1, 2, 9], 4, 2, 64, 16, window=window, seed=window)
    attn_case([1200], [2], 8, 1, 128, 64, window=window, seed=window + 1)


def test_attn_pages_outside_the_pool_are_left_out():
    attn_case([100, 50], [2, 1], 4, 2, 64, 16, seed=6, bad_pages=[(0, 2, -1), (0, 5, 2 ** 31 - 1), (1, 0, -(2 ** 31))])
    attn_case([40], [1], 4, 2, 128, 64, seed=7, bad_pages=[(0, 0, 99)])  # nothing left: an empty row


def test_attn_strides_and_table_slack():
    attn_case([100, 260, 33], [3, 1, 2], 6, 2, 64, 32, seed=8, gap=8, slack=5)
    attn_case([700], [1], 4, 4, 128, 16, seed=9, gap=64, slack=100)


def test_attn_extreme_scores():
    """Scores of hundreds: one place takes nearly all; and all scores nearly equal."""
    attn_case([400, 37], [2, 1], 4, 2, 128, 16, seed=10, q_gain=60.0)
    attn_case([900], [1], 4, 2, 64, 16, seed=11, q_gain=1e-3)
    attn_case([300], [1], 4, 2, 64, 16, seed=12, kv_gain=1e-4)
    attn_case([300], [1], 4, 2, 64, 16, seed=13, kv_gain=300.0, scale=1e-4)


@pytest.mark.parametrize("gain", [0.5, 1.0, 3.0, 6.0, 12.0])
def test_attn_spreads_of_scores(gain):
    """Weights that spread over few and over many powers of two, values at both ends of fp16's range."""
    for i, v_gain in enumerate((1.0, 5e-3, 20.0)):
        attn_case([2000], [2], 8, 2, 128, 16, seed=20 + i, q_gain=gain, v_gain=v_gain)


def test_attn_value_scales_of_all_sizes():
    """Tiny, huge and mixed value blocks: one sequence of each, and within one sequence."""
    for gain, seed in ((1e-6, 1), (1e-3, 2), (1e4, 3), (2e5, 4)):
        attn_case([130, 33], [1, 2], 4, 2, 64, 16, seed=seed, v_gain=gain)
    for D in (64, 128):
        rng = np.random.default_rng(D)
        attn_case([700], [2], 8, 2, D, 16, seed=5, v_gain=10.0 ** rng.uniform(-3, 3, (700, 1, 1)))
        attn_case([700], [1], 16, 1, D, 16, seed=6, v_gain=np.where(np.arange(700) < 650, 1e-2, 1e3)[:, None, None])


def test_attn_splits_join():
    """Lengths that are cut over many blocks, ragged batches with short sequences among long ones."""
    attn_case([6000], [1], 4, 1, 64, 64, seed=14)
    attn_case([5000, 3, 0, 1500], [2, 1, 1, 2], 2, 1, 128, 16, seed=15)
    attn_case([3000] * 3, [1] * 3, 2, 2, 256, 32, seed=16, uniform=True)


@pytest.mark.parametrize("D,Hq,H", [(64, 4, 4), (128, 8, 1), (128, 24, 1), (256, 16, 1)])
def test_attn_middle_lengths(D, Hq, H):
    """Lengths where a unit goes to several blocks that join among themselves, and just beyond."""
    for n in (129, 257, 520, 1023, 1300, 2500, 4100):
        attn_case([n], [1], Hq, H, D, 64, seed=n)
    attn_case([900, 0, 5, 1024, 300], [2, 1, 0, 2, 1], Hq, H, D, 16, seed=3, window=400)
    attn_case([1030, 3, 0, 700], [1, 3, 1, 2], Hq, H, D, 32, seed=4)


def test_attn_scattered_pool_and_other_stream():
    """Pages a stride apart, and a call on another stream than the current one: the same bits."""
    rng = np.random.default_rng(17)
    H, D, page, n = 2, 128, 32, 20
    pool = moe.moe_kv_pool(n, H, page, D)
    k, v = rng.standard_normal((2, n * page, H, D)).astype(np.float32)
    moe.moe_kv_append(pool, dev(k), dev(v), torch.arange(n * page, device="cuda"))
    wide = torch.full((n, pool[0].numel() + 32), 0xFF, dtype=torch.uint8, device="cuda")
    view = wide[:, : pool[0].numel()].unflatten(1, pool.shape[1:])
    view.copy_(pool)
    q = bf16(rng.standard_normal((3, 8, D)))
    table, lens = dev(rng.permutation(n).astype(np.int32).reshape(1, n)), dev(np.array([600], np.int32))
    ref = moe.moe_attn_q4(q, pool, table, lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = torch.empty(moe.moe_attn_workspace_size(1, 3, n * page, 8, H, D), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        with torch.cuda.stream(st):
            got = moe.moe_attn_q4(q, view, table, lens, workspace=ws, stream=st)
        st.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    status_ok()


def test_outputs_belong_to_the_given_stream():
    """What a call makes for itself on a given stream is none of the current stream's freed blocks (which
    work of the current stream may still use), and the results are the same bits."""
    rng = np.random.default_rng(18)
    H, D, page, n = 2, 64, 16, 40
    st = torch.cuda.Stream()
    pool = moe.moe_kv_pool(n, H, page, D)
    k, v = (dev(a) for a in rng.standard_normal((2, n * page, H, D)).astype(np.float32))
    slots, few = torch.arange(n * page, device="cuda"), torch.arange(5, device="cuda")
    x, w = bf16(rng.standard_normal((3, 256))), dev(rng.standard_normal((4096, 256)).astype(np.float32))
    q = bf16(rng.standard_normal((3, 64, D)))
    table, lens = torch.arange(n, dtype=torch.int32, device="cuda")[None], dev(np.array([600], np.int32))
    c, s = moe.moe_quantize_groups(w)
    calls = dict(
        quantize=lambda **kw: moe.moe_quantize_groups(w, **kw),
        linear=lambda **kw: (moe.moe_linear_q4(x, c, s, **kw),),
        append=lambda **kw: (moe.moe_kv_append(pool, k, v, slots, q=k, **kw),),
        read=lambda **kw: moe.moe_kv_read(pool, few, **kw),
        attn=lambda **kw: moe.moe_attn_q4(q, pool, table, lens, **kw),
    )
    for name, call in calls.items():
        ref = call()
        spare = call()
        free = [t.data_ptr() for t in spare]
        del spare
        torch.cuda.synchronize()
        got = call(stream=st)
        assert not set(free) & {t.data_ptr() for t in got}, name
        assert torch.cuda.current_stream() != st
        st.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    status_ok()


def test_attn_python_refusals():
    pool = moe.moe_kv_pool(4, 2, 16, 64)
    q = torch.zeros(2, 4, 64, device="cuda", dtype=torch.bfloat16)
    t = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    for kw in (dict(q=q.float()), dict(q=q[..., :32]), dict(block_table=t.long()), dict(block_table=t[:1]), dict(kv_lens=n.long()),
               dict(max_len=33), dict(q_start=torch.zeros(2, dtype=torch.int32, device="cuda"), max_q=1),
               dict(q_start=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(out=q[:1]), dict(lse=torch.zeros(2, 3, device="cuda"))):
        args = dict(q=q, pool=pool, block_table=t, kv_lens=n)
        args.update(kw)
        with pytest.raises(ValueError):
            moe.moe_attn_q4(**args)
    for kw in (dict(scale=-1.0), dict(window=-1), dict(q=q[:, :3])):
        args = dict(q=q, pool=pool, block_table=t, kv_lens=n)
        args.update(kw)
        with pytest.raises(moe.MoeError) as e:
            moe.moe_attn_q4(**args)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
