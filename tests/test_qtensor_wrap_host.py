"""Quantized tensors on buffers the caller has, without a GPU: what the
constructor leaves for the calls to check."""
import pytest


@pytest.fixture(scope="module")
def fp4():
    import fp4_fully_quantized_amd as m
    return m


def test_wrap_keeps_what_it_is_given(fp4):
    import torch
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    a, t = torch.zeros(1), torch.ones(1)
    q = fp4.QTensor.wrap(codes, scales, fp4.FP4_NVFP4, tscale=t)
    assert q.amax is None and q.tscale is t and (q.rows, q.cols) == (4, 64)
    assert q.desc().amax is None and q.desc().tscale == t.data_ptr()
    q = fp4.QTensor.wrap(codes, scales, fp4.FP4_NVFP4, amax=a, tscale=t)
    assert q.amax is a and q.tscale is t
    q = fp4.QTensor.wrap(codes, scales[:, :2].contiguous(), fp4.FP4_MXFP4)
    assert q.amax is None and q.tscale is None


def test_amax_from_without_an_amax(fp4):
    import torch
    codes, scales = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    q = fp4.QTensor.wrap(codes, scales, fp4.FP4_NVFP4, tscale=torch.ones(1))
    x = torch.zeros((16, 64))
    for call in (lambda: fp4.quantize(x, amax_from=q), lambda: fp4.quantize_dual(x, amax_from=q),
                 lambda: fp4.quantize_dual(x, had_signs_cols=1, amax_from=(q, q)), lambda: fp4.quantize_2d(x, amax_from=q)):
        with pytest.raises(ValueError, match="amax_from has no amax"):
            call()
