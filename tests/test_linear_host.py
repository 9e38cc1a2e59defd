"""Host-side checks of the norm, the dense product and the rotation into the cache (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from mxfp4_routed_expert_03_gb300 import build
    build.build()
    import mxfp4_routed_expert_03_gb300 as m
    return m


@pytest.mark.parametrize("d,eps,weight,code", [
    (0, 1e-6, None, -1), (-8, 1e-6, None, -1), (100, 1e-6, None, -1), (128, -1.0, None, -1), (128, float("nan"), None, -1),
    (128, float("inf"), None, -1), (128, 1e-6, 8, -1), (16392, 1e-6, None, -2)])
def test_norm_create_rejects(L, d, eps, weight, code):
    h, desc = ctypes.c_void_p(), L.moe_norm_desc(d, eps, weight)
    assert L.lib().moe_norm_create(ctypes.byref(desc), ctypes.byref(h)) == code
    assert h.value is None


@pytest.mark.parametrize("d_in,d_out,wq,ws,code", [
    (0, 8, 16, 16, -1), (24, 8, 16, 16, -1), (16, 4, 16, 16, -1), (16, 0, 16, 16, -1), (-16, 8, 16, 16, -1),
    (16, 8, None, 16, -1), (16, 8, 8, 16, -1), (16, 8, 16, None, -1), (16, 8, 16, 2, -1), (65552, 8, 16, 16, -2),
    (16, (1 << 20) + 8, 16, 16, -2)])
def test_linear_create_rejects(L, d_in, d_out, wq, ws, code):
    h, desc = ctypes.c_void_p(), L.moe_linear_desc(d_in, d_out)
    assert L.lib().moe_linear_create(ctypes.byref(desc), wq, ws, ctypes.byref(h)) == code
    assert h.value is None


def test_null_handles_are_rejected(L):
    bad = L.MOE_ERR_INVALID_ARG
    assert L.lib().moe_norm_create(None, None) == bad and L.lib().moe_linear_create(None, 16, 16, None) == bad
    h = ctypes.c_void_p()
    assert L.lib().moe_norm_create(None, ctypes.byref(h)) == bad
    assert L.lib().moe_linear_create(None, 16, 16, ctypes.byref(h)) == bad
    assert L.moe_add_norm(None, 1, None, 0, None, 0, None, 0, None, 0, None) == bad
    assert L.moe_linear_forward(None, 1, L.moe_fp8_rows(), None, 0, 0) == bad
    assert L.moe_linear_status(None) == bad
    assert L.moe_linear_set_fault_injection(None, 0, 0) == bad
    assert L.moe_rope_append(None, 1, L.moe_rope_desc(), None, None, 0, None, 0, None, 0, None, None, 0) == bad
    L.moe_norm_destroy(None)
    L.moe_linear_destroy(None)


def test_rows_of_codes_are_checked():
    import torch
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    rows = Fp8Rows(q, s)  # (its device is checked by the call)
    assert rows.desc.q_stride == 256 and rows.desc.s_stride == 2
    rows.check(4, 256, -1)
    for T, width, device in ((5, 256, -1), (4, 272, -1), (4, 256, 0)):
        with pytest.raises(ValueError):
            rows.check(T, width, device)
    assert Fp8Rows(q[:, :144], s).width == 144
    for bad in ((q[0], s), (q.float(), s), (q.t(), s), (q, s[0]), (q, s.double()), (q, s[:3]), (q, s[:, :1]), (q, s.t())):
        with pytest.raises(ValueError):
            Fp8Rows(*bad)


def test_weights_of_another_layout_are_refused():
    """A matrix [rows][columns] by its shape: a transposed one has as many elements and would be read as another."""
    import torch
    from mxfp4_routed_expert_03_gb300.checks import matrix
    bits = (torch.uint8, torch.int8)
    w = torch.zeros(384, 256, dtype=torch.uint8)
    for ok in (w, w.view(3, 128, 256), w.flatten(), torch.zeros(500, 256, dtype=torch.int8), w.view(3, 1, 128, 256)):
        matrix(ok, 384, 256, bits, "w_q")
    for bad in (w.t(), w.t().contiguous(), torch.zeros(256, 384, dtype=torch.uint8), w.view(768, 128), w[:383], w.float(), w[:, ::2], w.flatten()[:-1]):
        with pytest.raises(ValueError):
            matrix(bad, 384, 256, bits, "w_q")
    s = torch.zeros(3, 2)
    for ok in (s, s[:, None, :, None], s.flatten(), torch.zeros(4, 2)):
        matrix(ok, 3, 2, (torch.float32,), "w_s")
    for bad in (s.t(), s.t().contiguous(), s.t().contiguous()[:, None, :, None], s.double(), s[:2]):
        with pytest.raises(ValueError):
            matrix(bad, 3, 2, (torch.float32,), "w_s")
    matrix(torch.zeros(3, 1), 3, 1, (torch.float32,), "w_s")
    matrix(torch.zeros(1, 5), 1, 5, (torch.float32,), "w_s")
