"""The operators around the FP4 product at the widest outputs a product has."""
import pytest

from gpu_util import say
from layer_ref import U

pytestmark = pytest.mark.gpu

WIDE = (1 << 24) + 40


@pytest.fixture(scope="module")
def fp4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_fully_quantized_amd as m
    m.lib()
    return m


def same8(a, b, cols):
    import torch
    n = a.codes.shape[1]
    return torch.equal(a.codes[:, :n], b.codes[:, -n:]) and torch.equal(a.scales, b.scales[:, -a.scales.shape[1]:])


@pytest.mark.parametrize("fmt", [0, 1])
def test_product_wider_than_2_to_24(fp4, fmt):
    """Bias, residual and checkpoint go as wide as the product itself: its last columns are those of the last rows of
    B alone, and the backward pass reads the checkpoint."""
    import torch
    say("gemm fused, wide", fmt)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    A = fp4.quantize(torch.randn((1, 128), generator=gen, device="cuda"), fmt=fmt)
    B = fp4.quantize(torch.randn((WIDE, 128), generator=gen, device="cuda", dtype=torch.bfloat16), fmt=fmt)
    bias, res = torch.randn(WIDE, generator=gen, device="cuda"), torch.randn((1, WIDE), generator=gen, device="cuda")
    y, z8 = fp4.gemm_fused(A, B, bias=bias, act=fp4.FP4_ACT_RELU, residual=res, checkpoint=True)
    last = 1032   # whole blocks of the checkpoint from column WIDE - 1032 on
    b = fp4.QTensor.wrap(B.codes[-last:], B.scales[-last:], fmt, tscale=B.tscale)
    dot = fp4.dequantize(A).double() @ fp4.dequantize(b).double().t().contiguous()
    mag = fp4.dequantize(A).double().abs() @ fp4.dequantize(b).double().abs().t().contiguous()
    z = dot + bias[-last:].double()
    # the product's own bound, the decoded operands' rounding (NVFP4), two additions
    tol = 1e-5 * mag + 3 * U * mag + 2 * U * (z.abs() + res[:, -last:].double().abs()) + 1e-37
    assert ((y[:, -last:].double() - (z.clamp(min=0) + res[:, -last:].double())).abs() <= tol).all()
    yl, zl = fp4.gemm_fused(A, b, bias=bias[-last:], act=fp4.FP4_ACT_RELU, residual=res[:, -last:], checkpoint=True)
    assert torch.equal(yl, y[:, -last:]) and same8(zl, z8, last)
    dy = torch.randn((1, WIDE), generator=gen, device="cuda")
    g = fp4.act_backward(dy, z8, fp4.FP4_ACT_SILU, amax=True)
    gl = fp4.act_backward(dy[:, -last:], zl, fp4.FP4_ACT_SILU)
    assert torch.equal(g.dz[:, -last:], gl.dz) and torch.equal(g.dbias[-last:], gl.dbias)
    assert float(g.amax) == float(g.dz.abs().max())


def test_rows_wider_than_2_to_24(fp4):
    import torch
    say("8 bits and norm, wide")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    x, last = torch.randn((2, WIDE), generator=gen, device="cuda"), 1032
    q = fp4.mx8_quantize(x)
    assert same8(fp4.mx8_quantize(x[:, -last:]), q, last)
    assert torch.equal(fp4.mx8_dequantize(q)[:, -last:], fp4.mx8_dequantize(fp4.mx8_quantize(x[:, -last:])))
    g = torch.randn(WIDE, generator=gen, device="cuda")
    o = fp4.rmsnorm(x, g, amax=True)
    rstd = 1 / torch.sqrt(x.double().square().mean(1) + 1e-5)
    # a lane adds 8 values of each of WIDE / 8192 chunks, then 6 + 16 across lanes; half of it reaches rstd
    tol = ((WIDE / 1024 + 22 + 3) / 2 + 8) * U
    assert ((o.rstd.double() - rstd).abs() <= tol * rstd).all()
    want = x.double() * rstd[:, None] * g.double()
    assert ((o.y.double() - want).abs() <= (tol + U) * want.abs() + 1e-37).all()
    assert float(o.amax) == float(o.y.abs().max())
    dy = torch.randn((2, WIDE), generator=gen, device="cuda") * 1e-3
    dx, dgamma = fp4.rmsnorm_backward(dy, x, g, o.rstd)
    r = o.rstd.double()[:, None]
    xhat, gd = x.double() * r, dy.double() * g.double()
    m, mm = (gd * xhat).mean(1, keepdim=True), (gd * xhat).abs().mean(1, keepdim=True)
    tol = (WIDE / 1024 + 22 + 10) * U * r * (gd.abs() + xhat.abs() * mm)
    assert ((dx.double() - r * (gd - xhat * m)).abs() <= tol + 1e-37).all()
    assert ((dgamma.double() - (dy.double() * xhat).sum(0)).abs() <= 8 * U * (dy.double() * xhat).abs().sum(0) + 1e-37).all()
