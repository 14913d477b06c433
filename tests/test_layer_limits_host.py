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
