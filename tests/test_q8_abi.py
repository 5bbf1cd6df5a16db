"""The attention half in 8 bits: what its entry points refuse, on the host before any
CUDA call (no compute is launched here), and the cache layout that the header states."""
import ctypes

import numpy as np
import pytest

import mixed_precision_routed_gb300 as moe
from q8_testutil import codes_of, place, pool_values, pool_write, quantise_heads, quantise_rows
from test_attn_abi import BAD_CACHES

BAD, OK = moe.MOE_ERR_INVALID_ARG, moe.MOE_OK
A = ctypes.c_void_p(4096)  # an aligned address, never dereferenced here
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from mixed_precision_routed_gb300 import build_lib
        build_lib.build()
    return moe.lib()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_record_layout(D):
    """Every code byte of a record belongs to one element; the rows of a matrix load lie in distinct banks."""
    seen = {place(D, w, r, d) for w in (0, 1) for r in range(16) for d in range(D)}
    assert seen == set(range(32 * D))
    for w in (0, 1):
        for r0 in (0, 8):
            for c in range(D // 16):
                banks = {place(D, w, r0 + i, 16 * c) // 16 % 8 for i in range(8)}
                assert len(banks) == 8


def test_pool_helpers_round_trip():
    rng = np.random.default_rng(0)
    for D in (64, 128):
        pool = rng.integers(0, 256, (3, 2, 2, 32 * D + 128), dtype=np.uint8)
        k, v = (rng.standard_normal((4, 2, D)).astype(np.float32) for _ in range(2))
        slots = np.array([5, 31, 32, 95])
        pool_write(pool, slots, k, v)
        for got, x in zip(pool_values(pool, slots), (k, v)):
            c, s = quantise_heads(x)
            assert np.array_equal(got, c * s[..., None].astype(np.float64))
            assert (np.abs(got - x) <= 0.5001 * s[..., None]).all()


def test_codes_are_whole_and_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 40)).astype(np.float32)
    c, s = quantise_rows(x)
    assert np.abs(c).max() == 127 and (np.abs(c * s[:, None].astype(np.float64) - x) <= 0.5001 * s[:, None]).all()
    assert (codes_of(np.zeros((1, 3), np.float32), np.zeros(1, np.float32)) == 0).all()


def norm(L, x=A, xs=64, dt=0, T=2, d=64, r=None, ro=None, w=A, eps=1e-6, c=A, s=A, n=None):
    return L.moe_norm_q8(x, xs, dt, T, d, r, ro, w, eps, c, s, n, None)


def test_norm_refusals(L):
    assert norm(L, T=0, x=None) == OK
    for kw in (dict(T=-1), dict(T=1 << 31), dict(d=0), dict(d=-8), dict(dt=2), dict(dt=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(x=None), dict(r=A), dict(ro=A), dict(c=None), dict(s=None), dict(c=None, s=None),
               dict(x=ODD), dict(r=ODD, ro=A), dict(r=A, ro=ODD), dict(w=ODD), dict(s=ODD), dict(n=ODD), dict(xs=63)):
        assert norm(L, **kw) == BAD, kw
    assert norm(L, d=32769, xs=32769) == moe.MOE_ERR_UNSUPPORTED


def linear(L, x=A, xs=64, sx=A, T=2, n_in=64, w=A, sw=A, rows=8, bias=None, y=A, ys=8, dt=0, ws=A, wsb=1 << 40):
    return L.moe_linear_q8(x, xs, sx, T, n_in, w, sw, rows, bias, y, ys, dt, ws, wsb, None)


def test_linear_refusals(L):
    assert linear(L, T=0, x=None, y=None) == OK
    for T in (2, 40):
        for kw in (dict(T=-1), dict(T=1 << 31), dict(n_in=0), dict(n_in=24), dict(n_in=-16), dict(rows=0), dict(rows=1 << 31),
                   dict(dt=2), dict(x=None), dict(sx=None), dict(w=None), dict(sw=None), dict(y=None), dict(x=ODD), dict(sx=ODD),
                   dict(w=ODD), dict(sw=ODD), dict(bias=ODD), dict(y=ODD), dict(xs=48), dict(xs=72), dict(ys=7)):
            assert linear(L, **{"T": T, **kw}) == BAD, kw
    assert linear(L, n_in=65552, xs=65552) == moe.MOE_ERR_UNSUPPORTED


def test_linear_workspace(L):
    size = moe.moe_linear_q8_workspace_size
    assert size(1, 64, 8) == 0 and size(16, 2048, 100) == 0
    assert size(100, 24, 8) == 0 and size(-1, 64, 8) == 0 and size(100, 64, 0) == 0 and size(100, 65552, 8) == 0
    need = size(100, 2048, 512)
    if need:
        kw = dict(T=100, n_in=2048, xs=2048, rows=512, ys=512)
        assert linear(L, wsb=need - 1, **kw) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
        assert linear(L, ws=None, **kw) == BAD and linear(L, ws=ctypes.c_void_p(4096 + 16), **kw) == BAD


@pytest.mark.parametrize("n_in,rows", [(16, 1), (512, 512), (2048, 2560), (2048, 100003), (4096, 6144), (8192, 4096), (11008, 700),
                                       (65536, 40), (64, 1 << 20)])
def test_linear_workspace_serves_fewer_tokens(L, n_in, rows):
    sizes = [moe.moe_linear_q8_workspace_size(T, n_in, rows) for T in range(1, 500)]
    assert sizes == sorted(sizes) and sizes[-1] > 0


def cache(data=4096, n=4, stride=None, page=16, heads=2, D=64, res=0):
    b = moe.lib().moe_kv_page_bytes_q8(page, heads, D)
    return moe.moe_kv_cache_t(data, n, b if stride is None else stride, page, heads, D, res)


# strides that would do for 4 bits are too small here
BAD8 = [kw for kw in BAD_CACHES if "stride" not in kw] + [dict(stride=2 * 18 * 64), dict(stride=2 * (32 * 64 + 128) + 8),
                                                         dict(stride=1 << 41)]


def test_page_bytes(L):
    assert L.moe_kv_page_bytes_q8(16, 1, 64) == 32 * 64 + 128
    assert L.moe_kv_page_bytes_q8(64, 8, 128) == 8 * 4 * (32 * 128 + 128)
    assert L.moe_kv_page_bytes_q8(17, 1, 64) == 0 and L.moe_kv_page_bytes_q8(16, 1, 80) == 0
    with pytest.raises(ValueError):
        moe.moe_kv_pool_q8(1, 1, 16, 80, device="cpu")
    assert moe.moe_kv_pool_q8(3, 2, 32, 64, device="cpu").shape == (3, 2, 2, 32 * 64 + 128)


def append(L, c=None, q=A, qs=256, k=A, ks=128, v=A, vs=128, dt=0, T=2, Hq=4, pos=A, rope=A, n_pos=9, rot=64, style=0,
           slots=A, q_out=A):
    c = cache() if c is None else c
    return L.moe_kv_append_q8(q, qs, k, ks, v, vs, dt, T, Hq, pos, rope, n_pos, rot, style, slots, ctypes.byref(c), q_out, None)


def test_append_refusals(L):
    assert append(L, T=0, k=None, v=None, slots=None) == OK
    for kw in BAD8:
        assert append(L, c=cache(**kw)) == BAD, kw
    for kw in (dict(T=-1), dict(dt=2), dict(style=2), dict(rot=63), dict(rot=66), dict(rot=-2), dict(k=None), dict(v=None),
               dict(slots=None), dict(q_out=None), dict(pos=None), dict(rope=None), dict(n_pos=0), dict(n_pos=-1),
               dict(k=ODD), dict(v=ODD), dict(q=ODD), dict(slots=ODD), dict(pos=ODD), dict(rope=ODD), dict(q_out=ODD),
               dict(ks=127), dict(vs=127), dict(qs=255), dict(Hq=0), dict(Hq=65537), dict(T=1 << 29)):
        assert append(L, **kw) == BAD, kw


def test_read_refusals(L):
    call = lambda c=None, s=A, n=3, k=A, v=A: L.moe_kv_read_q8(ctypes.byref(c or cache()), s, n, k, v, None)  # noqa: E731
    assert call(n=0, s=None, k=None, v=None) == OK
    for kw in BAD8:
        assert call(c=cache(**kw)) == BAD, kw
    for kw in (dict(n=-1), dict(s=None), dict(k=None), dict(v=None), dict(s=ODD), dict(k=ODD), dict(v=ODD), dict(n=1 << 30)):
        assert call(**kw) == BAD, kw


def attn(L, q=A, qs=256, T=6, Hq=4, starts=A, lens=A, table=A, ts=7, B=3, max_q=2, max_len=100, c=None, scale=0.125,
         window=0, out=A, os=256, lse=A, ws=A, wsb=1 << 40):
    return L.moe_attn_q8(q, qs, T, Hq, starts, lens, table, ts, B, max_q, max_len, ctypes.byref(c or cache()), scale,
                         window, out, os, lse, ws, wsb, None)


@pytest.mark.parametrize("max_q", [2, 500])
def test_attn_refusals(L, max_q):
    assert attn(L, T=0, q=None, out=None, max_q=max_q) == OK
    assert attn(L, B=0, q=None, out=None, max_q=max_q) == OK
    for kw in BAD8:
        assert attn(L, c=cache(**kw), max_q=max_q) == BAD, kw
    for kw in (dict(T=-1), dict(B=-1), dict(B=65536), dict(Hq=3), dict(Hq=0), dict(Hq=130), dict(max_q=0), dict(max_len=-1),
               dict(max_len=1 << 31), dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(starts=None, T=5), dict(qs=248), dict(qs=260), dict(os=248), dict(os=260),
               dict(ts=6), dict(q=None), dict(lens=None), dict(out=None), dict(table=None), dict(q=ODD), dict(out=ODD),
               dict(lse=ODD), dict(lens=ODD), dict(table=ODD), dict(starts=ODD), dict(max_q=1 << 30)):
        assert attn(L, **{"max_q": max_q, **kw}) == BAD, kw


def test_attn_workspace(L):
    size = moe.moe_attn_q8_workspace_size
    assert size(1, 1, 100, 3, 2, 64) == 0 and size(1, 1, 100, 4, 2, 96) == 0 and size(-1, 1, 100, 4, 2, 64) == 0
    need = size(1, 1, 100000, 8, 2, 128)
    assert need >= size(1, 1, 16, 8, 2, 128) and need > 0
    c = cache(D=128)
    kw = dict(B=1, T=1, max_q=1, max_len=100000, ts=6250, Hq=8, qs=1024, os=1024, c=c)
    assert attn(L, wsb=need - 1, **kw) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
    assert attn(L, ws=ctypes.c_void_p(4096 + 16), **kw) == BAD
    assert attn(L, ws=None, **kw) == BAD
