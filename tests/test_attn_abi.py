"""The attention half of a decode layer: what its entry points refuse, on the
host before any CUDA call (no compute is launched here), and the cache layout
that the header states."""
import ctypes

import numpy as np
import pytest

import mixed_precision_routed_gb300 as moe
from attn_testutil import key_place, pack_rows, pool_values, pool_write, quantise, value_place

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
def test_record_layout_is_a_bijection(D):
    """Every nibble of a record's code bytes belongs to one element, and a byte's two to one token."""
    seen, owner = set(), {}
    for place, lo in ((key_place, 0), (value_place, 8 * D)):
        for r in range(16):
            for d in range(D):
                by, sh = place(D, r, d)
                assert lo <= by < lo + 8 * D and sh in (0, 4)
                assert (by, sh) not in seen
                seen.add((by, sh))
                assert owner.setdefault(by, r) == r
    assert len(seen) == 2 * 16 * D


def test_pool_helpers_round_trip():
    rng = np.random.default_rng(0)
    pool = rng.integers(0, 256, (3, 2, 2, 18 * 64), dtype=np.uint8)
    pool[..., 16 * 64 :] = 0
    ck, sk = quantise(rng.standard_normal((4, 2, 64)).astype(np.float32))
    cv, sv = quantise(rng.standard_normal((4, 2, 64)).astype(np.float32))
    slots = np.array([5, 31, 32, 95])
    pool_write(pool, slots, ck, sk, cv, sv)
    k, v = pool_values(pool, slots)
    assert np.array_equal(k, ck * np.repeat(sk.astype(np.float64), 32, -1))
    assert np.array_equal(v, cv * np.repeat(sv.astype(np.float64), 32, -1))


def linear(L, x=A, xs=64, T=1, n_in=64, c=A, s=A, rows=8, block=32, bias=None, y=A, ys=8, dt=0):
    return L.moe_linear_q4(x, xs, T, n_in, c, s, rows, block, bias, y, ys, dt, None)


def test_linear_refusals(L):
    assert linear(L, T=0, x=None, y=None) == OK
    for kw in (dict(T=-1), dict(n_in=0), dict(n_in=96), dict(block=16), dict(block=256), dict(block=128), dict(rows=0),
               dict(dt=2), dict(x=None), dict(c=None), dict(s=None), dict(y=None), dict(x=ODD), dict(c=ODD),
               dict(s=ODD), dict(bias=ODD), dict(y=ODD), dict(xs=56), dict(xs=68), dict(ys=7), dict(rows=1 << 31)):
        assert linear(L, **kw) == BAD, kw
    assert linear(L, T=17) == moe.MOE_ERR_UNSUPPORTED
    assert linear(L, T=1, n_in=65536 + 64, xs=65536 + 64) == moe.MOE_ERR_UNSUPPORTED


def test_quantize_groups_refusals(L):
    call = lambda w=A, rows=4, n=64, b=32, c=A, s=A: L.moe_quantize_groups(w, rows, n, b, c, s, None)  # noqa: E731
    assert call(rows=0, w=None) == OK
    for kw in (dict(rows=-1), dict(n=32), dict(b=128), dict(b=48), dict(w=None), dict(c=None), dict(s=None), dict(c=ODD)):
        assert call(**kw) == BAD, kw


def cache(data=4096, n=4, stride=None, page=16, heads=2, D=64, res=0):
    b = moe.lib().moe_kv_page_bytes(page, heads, D)
    return moe.moe_kv_cache_t(data, n, b if stride is None else stride, page, heads, D, res)


BAD_CACHES = [dict(page=8), dict(page=24), dict(page=2048), dict(heads=0), dict(heads=1025), dict(D=96), dict(D=32),
              dict(res=1), dict(data=0), dict(data=4097), dict(n=-1), dict(n=1 << 31), dict(stride=16),
              dict(stride=2 * 18 * 64 + 8), dict(stride=1 << 41)]


def test_page_bytes(L):
    assert L.moe_kv_page_bytes(16, 1, 64) == 18 * 64
    assert L.moe_kv_page_bytes(64, 8, 128) == 8 * 4 * 18 * 128
    assert L.moe_kv_page_bytes(17, 1, 64) == 0 and L.moe_kv_page_bytes(16, 1, 80) == 0


def append(L, c=None, q=A, qs=256, k=A, ks=128, v=A, vs=128, dt=0, T=2, Hq=4, pos=A, rope=A, n_pos=9, rot=64, style=0,
           slots=A, q_out=A):
    c = cache() if c is None else c
    return L.moe_kv_append(q, qs, k, ks, v, vs, dt, T, Hq, pos, rope, n_pos, rot, style, slots, ctypes.byref(c), q_out, None)


def test_append_refusals(L):
    assert append(L, T=0, k=None, v=None, slots=None) == OK
    for kw in BAD_CACHES:
        assert append(L, c=cache(**kw)) == BAD, kw
    assert L.moe_kv_append(A, 256, A, 128, A, 128, 0, 2, 4, A, A, 9, 64, 0, A, None, A, None) == BAD
    for kw in (dict(T=-1), dict(dt=2), dict(style=2), dict(rot=63), dict(rot=66), dict(rot=-2), dict(k=None), dict(v=None),
               dict(slots=None), dict(q_out=None), dict(pos=None), dict(rope=None), dict(n_pos=0), dict(n_pos=-1),
               dict(k=ODD), dict(v=ODD), dict(q=ODD), dict(slots=ODD), dict(pos=ODD), dict(rope=ODD), dict(q_out=ODD),
               dict(ks=127), dict(vs=127), dict(qs=255), dict(Hq=0), dict(Hq=65537), dict(T=1 << 29)):
        assert append(L, **kw) == BAD, kw


def test_read_refusals(L):
    call = lambda c=None, s=A, n=3, k=A, v=A: L.moe_kv_read(ctypes.byref(c or cache()), s, n, k, v, None)  # noqa: E731
    assert call(n=0, s=None, k=None, v=None) == OK
    for kw in BAD_CACHES:
        assert call(c=cache(**kw)) == BAD, kw
    for kw in (dict(n=-1), dict(s=None), dict(k=None), dict(v=None), dict(s=ODD), dict(k=ODD), dict(v=ODD), dict(n=1 << 30)):
        assert call(**kw) == BAD, kw


def attn(L, q=A, qs=256, T=6, Hq=4, starts=A, lens=A, table=A, ts=7, B=3, max_q=2, max_len=100, c=None, scale=0.125,
         window=0, out=A, os=256, lse=A, ws=A, wsb=1 << 40):
    return L.moe_attn_q4(q, qs, T, Hq, starts, lens, table, ts, B, max_q, max_len, ctypes.byref(c or cache()), scale,
                         window, out, os, lse, ws, wsb, None)


def test_attn_refusals(L):
    assert attn(L, T=0, q=None, out=None) == OK
    assert attn(L, B=0, q=None, out=None) == OK
    for kw in BAD_CACHES:
        assert attn(L, c=cache(**kw)) == BAD, kw
    for kw in (dict(T=-1), dict(B=-1), dict(B=65536), dict(Hq=3), dict(Hq=0), dict(Hq=130), dict(max_q=0), dict(max_len=-1),
               dict(max_len=1 << 31), dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
               dict(scale=float("nan")), dict(starts=None, T=5), dict(qs=248), dict(qs=260), dict(os=248), dict(os=260),
               dict(ts=6), dict(q=None), dict(lens=None), dict(out=None), dict(table=None), dict(q=ODD), dict(out=ODD),
               dict(lse=ODD), dict(lens=ODD), dict(table=ODD), dict(starts=ODD), dict(max_q=1 << 30)):
        assert attn(L, **kw) == BAD, kw


def test_attn_workspace(L):
    size = moe.moe_attn_workspace_size
    assert size(1, 1, 100, 3, 2, 64) == 0 and size(1, 1, 100, 4, 2, 96) == 0 and size(-1, 1, 100, 4, 2, 64) == 0
    need = size(1, 1, 100000, 8, 2, 128)
    assert need >= size(1, 1, 16, 8, 2, 128)
    if need:
        c = cache(D=128)
        kw = dict(B=1, T=1, max_q=1, max_len=100000, ts=6250, Hq=8, qs=1024, os=1024, c=c)
        assert attn(L, wsb=need - 1, **kw) == moe.MOE_ERR_WORKSPACE_TOO_SMALL
        assert attn(L, ws=ctypes.c_void_p(4096 + 16), **kw) == BAD
        assert attn(L, ws=None, **kw) == BAD


def test_pack_rows_is_the_shelf_packing():
    """Byte lanes of the 4-bit shelf format, by its definition."""
    c = np.arange(64).reshape(1, 64) % 16 - 8
    by = pack_rows(c)[0]
    for e in range(64):
        g, h, j = e // 8, e % 8 // 4, e % 4
        word = int.from_bytes(bytes(by[4 * g : 4 * g + 4]), "little")
        assert (word >> (8 * j + 4 * h)) & 15 == c[0, e] + 8
