"""A quantization's tensor amax and tensor scale are two scalars (no GPU needed:
every call below is refused before anything is launched)."""
import ctypes
import os

import pytest

UNSUPPORTED = 4


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


def out(fp4, amax, tscale, **kw):
    return fp4.fp4_tensor(0x10000, 0x20000, amax, tscale, 0, 0, 0, kw.get("had_on", 0), 0, 0)


@pytest.mark.parametrize("ready", [0, 1])
def test_amax_that_is_the_tensor_scale(fp4, ready):
    L, A, T, A2, T2 = fp4.lib(), 0x30000, 0x40000, 0x50000, 0x60000
    args = (0x1000, 1, 64, 128, 128)
    one = ctypes.byref(out(fp4, A, A))
    assert L.fp4_quantize(*args, 0, 0, 0, 0, ready, one, None) == UNSUPPORTED
    assert L.fp4_quantize(*args, 1, 1, 0, 0, ready, one, None) == UNSUPPORTED
    assert L.fp4_quantize_noise(*args, 0, 0, 0, 0, ready, one, 0x70000, None) == UNSUPPORTED
    assert L.fp4_quantize_shard(*args, 0, 64, 0, 0, 0, 0, ready, one, None, None) == UNSUPPORTED
    # of either output, its own or the other's; with a rotation each has its own amax
    for (a1, t1), (a2, t2) in (((A, A), (A, T2)), ((A, T), (A, A)), ((A, T), (A2, A2)), ((A, T), (T, T2)), ((A, T), (A2, A))):
        for had in (0, 1):
            if had and a1 == a2:
                continue
            c, r = (ctypes.byref(out(fp4, *p, had_on=had)) for p in ((a1, t1), (a2, t2)))
            assert L.fp4_quantize_dual(*args, 0, 0, 0, 1, 0, 0, ready, c, r, None) == UNSUPPORTED
            assert L.fp4_quantize_dual_noise(*args, 0, 0, 0, 1, 0, 0, ready, c, r, 0x70000, None, None) == UNSUPPORTED
            assert L.fp4_quantize_dual_shard(*args, 0, 64, 0, 0, 0, 1, 0, 0, ready, c, r, None, None, None) == UNSUPPORTED
        c, r = (ctypes.byref(out(fp4, *p)) for p in ((a1, t1), (a2, t2)))
        assert L.fp4_quantize_2d(*args, 0, 0, 0, ready, c, r, None) == UNSUPPORTED
