"""Host-side checks of the attention and scored-routing entry points (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from mxfp4_routed_expert_03_gb300 import build
    build.build()
    import mxfp4_routed_expert_03_gb300 as m
    return m


def test_cache_sizes(L):
    d = L.moe_attn_desc(32, 4, 128, 64, 1000)
    assert L.moe_kv_code_bytes(d) == 1000 * 4 * 64 * 64
    assert L.moe_kv_scale_bytes(d) == 1000 * 4 * 64 * 4
    d = L.moe_attn_desc(16, 16, 64, 16, 100_000_000)
    assert L.moe_kv_code_bytes(d) == 100_000_000 * 16 * 16 * 32  # past 32 bits


@pytest.mark.parametrize("fields", [(0, 1, 64, 16, 1), (4, 0, 64, 16, 1), (4, 3, 64, 16, 1),
                                    (4, 2, 64, 16, 0), (4, 2, 64, 0, 1), (4, 2, -64, 16, 1)])
def test_create_rejects_bad_fields(L, fields):
    h = ctypes.c_void_p()
    d, c = L.moe_attn_desc(*fields), L.moe_kv_cache(16, 16, 16, 16)
    assert L.lib().moe_attn_create(ctypes.byref(d), ctypes.byref(c), ctypes.byref(h)) == L.MOE_ERR_INVALID_ARG
    assert h.value is None and L.moe_kv_code_bytes(d) == -1


@pytest.mark.parametrize("fields", [(4, 2, 96, 16, 1), (4, 2, 256, 16, 1), (4, 2, 64, 48, 1),
                                    (4, 2, 64, 512, 1), (2048, 2, 64, 16, 1), (4, 2, 64, 16, 1 << 27)])
def test_create_rejects_unsupported_shapes(L, fields):
    h = ctypes.c_void_p()
    d, c = L.moe_attn_desc(*fields), L.moe_kv_cache(16, 16, 16, 16)
    assert L.lib().moe_attn_create(ctypes.byref(d), ctypes.byref(c), ctypes.byref(h)) == L.MOE_ERR_UNSUPPORTED
    assert L.moe_kv_scale_bytes(d) == -1


def test_create_rejects_bad_cache_pointers(L):
    d = L.moe_attn_desc(4, 2, 64, 16, 1)
    for c in (L.moe_kv_cache(16, 16, 16, None), L.moe_kv_cache(16, 8, 16, 16)):
        with pytest.raises(L.MoeError):
            L.moe_attn_create(d, c)
    assert L.lib().moe_attn_create(None, None, None) == L.MOE_ERR_INVALID_ARG


def test_null_handles_are_rejected(L):
    bad = L.MOE_ERR_INVALID_ARG
    assert L.moe_attn_forward(None, L.moe_attn_batch(), None, 0, None, 0, None, None, 0) == bad
    assert L.moe_kv_append(None, 1, None, 0, None, 0, None) == bad
    assert L.moe_kv_read(None, 1, None, None, 0, None, 0) == bad
    assert L.moe_qk_norm_rope(None, 1, L.moe_rope_desc(), None, None, 0, None, 0, None, 0, None, 0) == bad
    assert L.moe_attn_status(None) == bad
    assert L.moe_attn_workspace_bytes(None, 1, 1, 1, 1) == 0
    assert L.moe_plan_scored(None, 1, None, None, L.moe_route_desc(), None, L.moe_plan_buf(), None, 0) == bad
    L.moe_attn_destroy(None)
