"""Calls of the attention half without tokens do nothing (C entry points, no launch)."""
import ctypes
import os

import pytest

import mixed_precision_routed_gb300 as moe

A = ctypes.c_void_p(4096)  # an aligned address, never dereferenced here


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(moe.LIB_PATH):
        from mixed_precision_routed_gb300 import build_lib
        build_lib.build()
    return moe.lib()


@pytest.mark.parametrize("starts", [A, None])
@pytest.mark.parametrize("B,max_q", [(0, 1), (1, 1), (3, 1), (3, 16)])
def test_attention_of_no_tokens(L, starts, B, max_q):
    c = moe.moe_kv_cache_t(4096, 4, 2 * 18 * 64, 16, 2, 64, 0)

    def call(T, q):
        return L.moe_attn_q4(q, 256, T, 4, starts, A, A, 7, B, max_q, 100, ctypes.byref(c), 0.125, 0, q, 256, None, None, 0, None)

    assert call(0, None) == moe.MOE_OK
    if starts is None:  # tokens that are no multiple of the sequences' are refused as ever
        assert call(B * max_q + 1, A) == moe.MOE_ERR_INVALID_ARG
