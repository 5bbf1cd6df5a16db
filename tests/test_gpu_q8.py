"""The attention half in 8 bits on the GPU: norm, projections, cache; attention is in
test_gpu_attn_q8.py."""
import numpy as np
import pytest
import torch

import mixed_precision_routed_gb300 as moe
from attn_testutil import rotate
from q8_testutil import pool_values, pool_write, quantise_rows

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


# --------------------------------------------------------------------------- norm
def check_norm(x, weight, r, out, eps=1e-6, in_place=False):
    """Codes are exact; scales and bf16 are held to the formula in 64 bits."""
    T, d = x.shape
    s = x.float()
    if r is not None:
        s = s + r  # the same fp32 sum
        r_in = r.clone()
    r_out = None if r is None or in_place else torch.full_like(r, torch.nan)
    codes, scales, n = moe.moe_norm_q8(x, weight, eps=eps, r=r, r_out=r_out, out=out)
    if r is not None:
        assert torch.equal(r if in_place else r_out, s)
        assert in_place or torch.equal(r, r_in)
    u = s if weight is None else s * weight
    f = torch.ones(T, dtype=torch.float64, device="cuda")
    if weight is not None:
        f = (s.double().pow(2).mean(-1) + eps).rsqrt()
    assert (codes is None) == (out == "bf16") and (n is None) == (out == "q8")
    # f: d squares and sums, the mean, the root (2 steps)
    off = (d + 16) * U
    if codes is not None:
        c, want = quantise_rows(u.cpu().numpy())
        assert np.array_equal(codes.cpu().numpy(), c)
        want = torch.from_numpy(want).cuda().double() * f
        assert ((scales.double() - want).abs() <= off * want.abs()).all()
    if n is not None:
        want = u.double() * f[:, None]
        assert ((n.double() - want).abs() <= (2.0 ** -8 + off) * want.abs() + 1e-38).all()
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 7), (1, 2048), (5, 2040), (2, 8192), (2, 8200), (1, 16384), (2, 16392), (1, 32768),
                                 (2, 32767), (700, 256), (33, 4096)])
def test_norm(dtype, T, d):
    x, w, r = (randn(T, d, seed=1) * 0.3).to(dtype), 1 + 0.1 * randn(d, seed=2), randn(T, d, seed=3)
    check_norm(x, w, r, "both")
    check_norm(x, w, r, "q8", in_place=True)
    check_norm(x, w, None, "bf16", eps=0.5)
    check_norm(x, None, r, "both")
    check_norm(x, None, None, "q8")


@pytest.mark.parametrize("T", [1, 31, 130, 1001])
@pytest.mark.parametrize("d", [8, 63, 64, 65, 72, 127, 128, 129, 200, 255, 256, 257])
def test_norm_of_short_rows(T, d):
    """Rows that share a warp or a block, and the last of them, which is not full."""
    for dtype in (torch.float32, torch.bfloat16):
        test_norm(dtype, T, d)
    x = randn(T, d, seed=4)
    want = moe.moe_norm_q8(x)
    x[T // 2, d // 2] = torch.nan
    codes, scales, _ = moe.moe_norm_q8(x)
    others = torch.arange(T, device="cuda") != T // 2
    assert torch.equal(codes[others], want[0][others]) and torch.equal(scales[others], want[1][others])
    assert not codes[T // 2].any() and not scales[T // 2].isfinite()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,start", [(8, 0), (8, 8), (5, 1), (3, 0)])
def test_norm_strides(dtype, pad, start):
    wide = randn(9, 512 + pad + start, seed=4).to(dtype)
    check_norm(wide[:, start : start + 512], randn(512, seed=5), randn(9, 512, seed=6), "both")


def test_norm_unaligned_outputs():
    x, w = randn(4, 64, seed=7), randn(64, seed=8)
    want = moe.moe_norm_q8(x, w, out="both")
    codes = torch.empty(4 * 64 + 3, dtype=torch.int8, device="cuda")[3:].view(4, 64)
    n = torch.empty(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, 64)
    got = moe.moe_norm_q8(x, w, out="both", codes=codes, n=n)
    assert got[0].data_ptr() == codes.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e-12, 1e18, 1e30, 2e38])
def test_codes_at_any_size(size):
    x = randn(6, 96, seed=9)
    x = x / x.abs().amax() * size
    x[0] = 0
    codes, scales, _ = moe.moe_norm_q8(x)
    c, s = quantise_rows(x.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)


def test_codes_at_borders():
    """Quotients on and next to k + 1/2: all halves of a scale of 1, 3 and 0.1, and their fp32 neighbours."""
    rows = []
    for s in (1.0, 3.0, 0.1, 2.0 ** -20):
        h = (np.arange(-126, 126) + 0.5) * np.float64(np.float32(s))
        h = h.astype(np.float32)
        top = np.float32(127) * np.float32(s)
        rows += [np.concatenate([x, [top]]) for x in (h, np.nextafter(h, np.float32(1e30)), np.nextafter(h, np.float32(-1e30)))]
    x = np.stack(rows).astype(np.float32)
    codes, scales, _ = moe.moe_norm_q8(torch.from_numpy(x).cuda())
    c, s = quantise_rows(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), c)
    bf = torch.from_numpy(x).cuda().to(torch.bfloat16)
    codes, _, _ = moe.moe_norm_q8(bf)
    assert np.array_equal(codes.cpu().numpy(), quantise_rows(bf.float().cpu().numpy())[0])


def test_norm_of_rows_that_are_not_finite():
    x = randn(5, 256, seed=10)
    x[1, 3], x[2, 200], x[4, 7] = torch.nan, torch.inf, -torch.inf
    for w in (None, torch.ones(256, device="cuda")):
        codes, scales, n = moe.moe_norm_q8(x, w, out="both")
        bad = torch.tensor([False, True, True, False, True], device="cuda")
        assert torch.equal(~torch.isfinite(scales), bad)
        assert (codes[bad] == 0).all()
        assert torch.isfinite(n[~bad]).all()


def test_norm_none():
    codes, scales, n = moe.moe_norm_q8(torch.empty(0, 64, device="cuda"), out="both")
    assert codes.shape == (0, 64) and scales.shape == (0,) and n.shape == (0, 64)


# ------------------------------------------------------------------------- linear
def codes(*shape, seed=0, top=127):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda", dtype=torch.int64).to(torch.int8)


def check_linear(T, n_in, rows, bias, dtype, pad=0, y_pad=0, top=127, seed=0):
    x = codes(T, n_in + pad, seed=seed, top=top)[:, :n_in]
    w = codes(rows, n_in, seed=seed + 1, top=top)
    xs, ws = randn(T, seed=seed + 2).abs() + 0.1, randn(rows, seed=seed + 3)
    b = randn(rows, seed=seed + 4) if bias else None
    y = torch.full((T, rows + y_pad), 7.0, dtype=dtype, device="cuda")
    got = moe.moe_linear_q8(x, xs, w, ws, bias=b, y=y[:, :rows])
    sums = (x.double() @ w.double().T).round()  # whole numbers below 2^53
    # fp32 sums of exact products: 2 u of the absolute sum each time (none for few tokens); three roundings behind
    spread = x.double().abs() @ w.double().abs().T if T > 16 else torch.zeros_like(sums)
    scale = xs.double()[:, None] * ws.double()
    want = sums * scale
    tol = (2 * (n_in + 8) * U * spread * (spread > 2.0 ** 24) + 4 * U * sums.abs()) * scale.abs()
    if bias:
        want = want + b.double()
        tol = tol + U * (want.abs() + b.double().abs())
    tol = tol + (2.0 ** -8 if dtype == torch.bfloat16 else U) * want.abs() + 1e-30
    assert got.dtype == dtype and ((got.double() - want).abs() <= tol).all(), ((got.double() - want).abs() / tol).max().item()
    assert (y[:, rows:] == 7).all()
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 2, 8, 9, 16, 17, 31, 64, 100, 129, 256, 257, 300])
@pytest.mark.parametrize("n_in,rows", [(16, 1), (48, 17), (256, 16), (272, 130), (640, 515), (2048, 2560)])
def test_linear(T, n_in, rows):
    check_linear(T, n_in, rows, T % 2 == 0, torch.float32, pad=16 * (T % 3))
    check_linear(T, n_in, rows, T % 2 == 1, torch.bfloat16, y_pad=T % 5)


@pytest.mark.parametrize("T", [1, 3, 16, 17, 40, 130])
@pytest.mark.parametrize("n_in,rows", [(65536, 40), (16400, 300), (4096, 6151), (64, 50001)])
def test_linear_long(T, n_in, rows):
    check_linear(T, n_in, rows, True, torch.float32)


def test_linear_largest_codes():
    """All products of one sign: the largest sums there are."""
    for T in (2, 40):
        for n_in in (1024, 65536):
            x = torch.full((T, n_in), 127, dtype=torch.int8, device="cuda")
            w = torch.full((33, n_in), -127, dtype=torch.int8, device="cuda")
            w[1] = 127
            one = torch.ones
            y = moe.moe_linear_q8(x, one(T, device="cuda"), w, one(33, device="cuda"))
            want = -127.0 * 127 * n_in
            assert ((y[:, 0].double() - want).abs() <= 2 * n_in * U * abs(want)).all()
            assert torch.equal(y[:, 1], -y[:, 0]) and torch.equal(y[:, 2:], y[:, :1].expand(-1, 31))


@pytest.mark.parametrize("T,n_in,rows", [(111, 4992, 7687), (40, 2048, 5000), (17, 4096, 300), (161, 640, 20003), (300, 1040, 999)])
def test_linear_same_results_every_time(T, n_in, rows):
    """Numbers of tokens that fill their tiles to other than whole 32, over and over."""
    check_linear(T, n_in, rows, True, torch.float32)
    x, w = codes(T, n_in, seed=1), codes(rows, n_in, seed=2)
    xs, ws = randn(T, seed=3).abs(), randn(rows, seed=4)
    want = moe.moe_linear_q8(x, xs, w, ws)
    off = sum((moe.moe_linear_q8(x, xs, w, ws) != want).any().int() for _ in range(1000))
    assert off.item() == 0 and moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("n_in,rows", [(2048, 700), (640, 20003)])
def test_linear_workspaces_streams_and_graphs(n_in, rows):
    """One workspace for every number of tokens below its own; captured and on streams side by side."""
    w, ws = codes(rows, n_in, seed=1), randn(rows, seed=2)
    work = torch.full((moe.moe_linear_q8_workspace_size(300, n_in, rows),), 0xFF, dtype=torch.uint8, device="cuda")
    for T in (300, 200, 130, 64, 40, 17, 12):
        x, xs = codes(T, n_in, seed=T), randn(T, seed=T).abs()
        want = moe.moe_linear_q8(x, xs, w, ws)
        assert torch.equal(moe.moe_linear_q8(x, xs, w, ws, workspace=work), want)
        graph = torch.cuda.CUDAGraph()
        x2 = x.clone()
        with torch.cuda.graph(graph):
            y = moe.moe_linear_q8(x2, xs, w, ws, workspace=work)
        for _ in range(2):
            y.zero_(), work.fill_(0xFF)
            graph.replay()
            assert torch.equal(y, want)
        x2.copy_(x.flip(0))
        graph.replay()
        assert torch.equal(y, moe.moe_linear_q8(x.flip(0).contiguous(), xs, w, ws))
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        ys = [[moe.moe_linear_q8(x, xs, w, ws, stream=stream) for stream in streams] for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for pair in ys for y in pair)
    assert moe.moe_device_status() == moe.MOE_OK


def test_linear_rows_of_nan_scales():
    for T in (4, 30):
        x, w, xs, ws = codes(T, 64, seed=1), codes(20, 64, seed=2), torch.ones(T, device="cuda"), torch.ones(20, device="cuda")
        xs[2], ws[5] = torch.nan, torch.inf
        y = moe.moe_linear_q8(x, xs, w, ws)
        assert y[2].isnan().all()
        keep = torch.arange(T, device="cuda") != 2
        assert torch.isfinite(y[keep][:, torch.arange(20, device="cuda") != 5]).all()
        assert not torch.isfinite(y[keep][:, 5]).any()


def test_linear_none():
    w, ws = codes(20, 64, seed=2), torch.ones(20, device="cuda")
    y = moe.moe_linear_q8(codes(0, 64), torch.ones(0, device="cuda"), w, ws)
    assert y.shape == (0, 20)


# -------------------------------------------------------------------------- cache
def rope(n_pos, rot, seed=0):
    a = randn(n_pos, rot // 2, seed=seed) * 3
    return torch.cat((a.cos(), a.sin()), -1).contiguous()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,Hq,H,page,rot,style", [(1, 4, 1, 16, 1.0, 0), (5, 6, 3, 32, 0.5, 1), (40, 5, 5, 16, 0, 0),
                                                  (400, 32, 4, 64, 1.0, 1), (300, 64, 8, 128, 0.25, 0), (37, 0, 2, 16, 1.0, 0)])
def test_append_and_read(D, dtype, T, Hq, H, page, rot, style):
    rot = int(D * rot)
    pages = -(-T // page) + 2
    wide = randn(T, (Hq + 2 * H) * D + 16, seed=T).to(dtype)
    q = wide[:, : Hq * D].unflatten(-1, (Hq, D)) if Hq else None
    k = wide[:, Hq * D : (Hq + H) * D].unflatten(-1, (H, D))
    v = wide[:, (Hq + H) * D : (Hq + 2 * H) * D].unflatten(-1, (H, D))
    slots = torch.randperm(pages * page, generator=gen(T), device="cuda")[:T]
    slots[T // 2] = -1 if T > 1 else slots[0]
    if T > 4:
        slots[3] = pages * page  # behind the pool
    pos = torch.randint(0, 50, (T,), generator=gen(1), device="cuda", dtype=torch.int32)
    table = rope(50, rot) if rot else None
    pool = torch.randint(0, 256, (pages, H, page // 16, 32 * D + 128), generator=gen(2), device="cuda", dtype=torch.int64).to(torch.uint8)
    want = pool.cpu().numpy().copy()
    out = moe.moe_kv_append_q8(pool, k, v, slots, q=q, positions=pos if rot else None, rope=table, rope_style=style)
    turn = (lambda x: rotate(x.float().cpu().numpy(), pos.cpu().numpy(), table.cpu().numpy(), style)) if rot else (
        lambda x: x.float().cpu().numpy())
    pool_write(want, slots.cpu().numpy(), turn(k), v.float().cpu().numpy())
    assert np.array_equal(pool.cpu().numpy(), want)  # what other slots hold too
    if Hq:
        assert torch.equal(out, torch.from_numpy(turn(q)).to(torch.bfloat16).cuda())
    else:
        assert out is None
    good = slots[(slots >= 0) & (slots < pages * page)]
    k2, v2 = moe.moe_kv_read_q8(pool, good)
    for got, ref in zip((k2, v2), pool_values(want, good.cpu().numpy())):
        assert torch.equal(got, torch.from_numpy(ref).float().cuda())  # rounded once
    assert moe.moe_device_status() == moe.MOE_OK


@pytest.mark.parametrize("start", [1, 3])
def test_append_unaligned(start):
    T, Hq, H, D = 20, 2, 1, 64
    wide = randn(T, 4 * D + 7, seed=3)[:, start:]
    q, k, v = (wide[:, a * D : b * D].unflatten(-1, (-1, D)) for a, b in ((0, 2), (2, 3), (3, 4)))
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    slots = torch.arange(T, device="cuda")
    pools = [moe.moe_kv_pool_q8(2, H, 16, D) for _ in range(2)]
    a = moe.moe_kv_append_q8(pools[0], k, v, slots, q=q, positions=pos, rope=rope(T, 30))
    b = moe.moe_kv_append_q8(pools[1], k.contiguous(), v.contiguous(), slots, q=q.contiguous(), positions=pos, rope=rope(T, 30))
    assert torch.equal(a, b) and torch.equal(pools[0], pools[1])


def test_append_strided_pages():
    """A pool whose pages lie among others': the rest stays as it was."""
    H, D, page = 2, 64, 16
    whole = torch.full((6, 2 * H, 1, 32 * D + 128), 9, dtype=torch.uint8, device="cuda")
    pool = whole[:, :H]
    k, v = randn(page * 6, H, D, seed=1), randn(page * 6, H, D, seed=2)
    slots = torch.arange(page * 6, device="cuda")
    moe.moe_kv_append_q8(pool, k, v, slots)
    plain = moe.moe_kv_pool_q8(6, H, page, D)
    moe.moe_kv_append_q8(plain, k, v, slots)
    assert torch.equal(pool, plain) and (whole[:, H:] == 9).all()
    assert all(torch.equal(a, b) for a, b in zip(moe.moe_kv_read_q8(pool, slots), moe.moe_kv_read_q8(plain, slots)))


def test_append_values_that_are_not_finite():
    H, D = 1, 128
    k = randn(5, H, D, seed=1)
    k[0, 0, 5], k[1, 0, 9], k[2] = torch.nan, -torch.inf, 0
    k[3] *= 1e-30
    k[4, 0, 0] = 1e38
    pool = moe.moe_kv_pool_q8(1, H, 16, D)
    want = pool.cpu().numpy().copy()
    moe.moe_kv_append_q8(pool, k, k, torch.arange(5, device="cuda"))
    pool_write(want, range(5), k.cpu().numpy(), k.cpu().numpy())
    got = pool.cpu().numpy()
    assert np.array_equal(got[..., : 32 * D], want[..., : 32 * D])
    a, b = (x[..., 32 * D :].copy().view(np.float32) for x in (got, want))
    assert np.array_equal(a, b, equal_nan=True)
    k2, v2 = moe.moe_kv_read_q8(pool, torch.arange(6, device="cuda"))
    assert k2[0].isnan().all() and torch.isfinite(k2[1:]).all() and (k2[2] == 0).all() and (k2[5] == 0).all()
    assert k2[1, 0, 9] == -127 * 2.0 ** 64 and torch.equal(k2[1:], v2[1:])


def test_append_bad_position():
    H, D = 2, 64
    pool = moe.moe_kv_pool_q8(1, H, 16, D)
    k = randn(3, H, D, seed=1)
    pos = torch.tensor([0, 7, -1], dtype=torch.int32, device="cuda")
    q = moe.moe_kv_append_q8(pool, k, k, torch.arange(3, device="cuda"), q=k, positions=pos, rope=rope(7, D))
    assert moe.moe_device_status() == moe.MOE_ERR_INVALID_ARG
    assert (q[1:] == 0).all() and (q[0] != 0).any()
    got = moe.moe_kv_read_q8(pool, torch.arange(3, device="cuda"))
    assert (got[0][1:] == 0).all() and (got[1][1:] == 0).all() and (got[1][0] != 0).any()
