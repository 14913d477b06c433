"""What the operators around the FP4 product refuse (no GPU needed: no call
below reaches a launch)."""
import ctypes
import os

import pytest

P = 0x1000  # a well-aligned fake device pointer
NULL = 1


@pytest.fixture(scope="module")
def fp4():
    import torch
    if torch.cuda.device_count() > 0:
        pytest.skip("host-only ABI checks run without a GPU")
    import fp4_fully_quantized_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.skip("libfp4.so not built")
    m.lib()
    return m


def test_norm_amax_without_y(fp4):
    """amax is that of y or y8: of a norm that stores neither there is none."""
    q = fp4.fp4_mx8(P, P, 4, 40, 64, 2)
    for outputs in ({"h": P, "ld_h": 40}, {"h8": ctypes.pointer(q)}, {"h": P, "ld_h": 40, "h8": ctypes.pointer(q)}):
        n = fp4.fp4_rmsnorm_fwd(rows=4, cols=40, dtype=0, gamma_t=0, x=P, ld_x=40, gamma=P, amax=P, eps=1e-5, **outputs)
        assert fp4.lib().fp4_rmsnorm(ctypes.byref(n), None) == NULL, outputs


def test_widths_past_every_product(fp4):
    """2^25 columns are taken (as wide as a product goes), more are not."""
    L, n = fp4.lib(), (1 << 25) + 1
    assert L.fp4_mx8_quantize(P, 0, n, ctypes.byref(fp4.fp4_mx8(P, P, 1, n, n + 31, n // 32 + 1)), None) == 2
    assert fp4.fp4_act_backward_workspace_bytes(2000, n) == 0 < fp4.fp4_act_backward_workspace_bytes(2000, n - 1)
    assert fp4.fp4_rmsnorm_backward_workspace_bytes(2, n) == 0 < fp4.fp4_rmsnorm_backward_workspace_bytes(2, n - 1)


def test_outputs_over_inputs_lie_as_they_do(fp4):
    """An output in an input's buffer has its leading dimension (and type): rows elsewhere would be overwritten before
    they are read."""
    L, Q, unsupported = fp4.lib(), 0x2000, 4
    for over in ({"y": P, "ld_y": 41}, {"y": P, "ld_y": 40, "h": P, "ld_h": 48}, {"residual": Q, "ld_residual": 40, "y": Q, "ld_y": 64},
                 {"residual": Q, "ld_residual": 40, "h": Q, "ld_h": 41}):
        n = fp4.fp4_rmsnorm_fwd(rows=4, cols=40, dtype=0, gamma_t=0, x=P, ld_x=40, gamma=P, eps=1e-5, **over)
        assert L.fp4_rmsnorm(ctypes.byref(n), None) == unsupported, over
    for over in ({"dx": P, "ld_dx": 48}, {"dres": Q, "ld_dres": 48, "dx": Q, "ld_dx": 40}):
        n = fp4.fp4_rmsnorm_bwd(rows=4, cols=40, dtype=0, gamma_t=0, dy=P, ld_dy=40, h=0x3000, ld_h=40, gamma=P, rstd=P, **over)
        assert L.fp4_rmsnorm_backward(ctypes.byref(n), None) == unsupported, over
    n = fp4.fp4_act_bwd(rows=4, cols=40, dtype=0, act=2, dy=P, ld_dy=40, z=Q, ld_z=40, dz=P, ld_dz=41)
    assert L.fp4_act_backward(ctypes.byref(n), None) == unsupported
    qs = [fp4.fp4_tensor(P, P, None, P, rows, 256, 1, 0, 0, 0) for rows in (100, 48)]
    a, b = (ctypes.byref(fp4.fp4_operand(kind=0, q=ctypes.pointer(q))) for q in qs)
    for ld, residual_t, out_t in ((56, 0, 0), (48, 1, 0), (48, 0, 1)):
        e = fp4.fp4_epilogue(residual=P, ld_residual=ld, residual_t=residual_t)
        assert L.fp4_gemm_fused(a, b, ctypes.byref(e), out_t, P, 48, None, 0, None) == unsupported
