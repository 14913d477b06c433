"""Quantized tensors on buffers the caller has: what takes them, and what has to
refuse them for want of the tensor amax or scale."""
import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_fully_quantized_amd as m
    m.lib()
    return m


def rand(seed, *shape):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


@pytest.mark.parametrize("fmt", [0, 1])
def test_wrapped_operands(fp4, fmt):
    """A product and a dequantization need no amax: a wrapped tensor, or whole rows of one, are operands."""
    import torch
    say("wrapped operands", fmt)
    A, B = fp4.quantize(rand(1, 96, 512), fmt=fmt), fp4.quantize(rand(2, 200, 512), fmt=fmt)
    a = fp4.QTensor.wrap(A.codes[16:48], A.scales[16:48], fmt, tscale=A.tscale)
    b = fp4.QTensor.wrap(B.codes, B.scales, fmt, tscale=B.tscale)
    assert a.amax is None and b.amax is None
    assert torch.equal(fp4.gemm(a, b), fp4.gemm(A, B)[16:48])
    assert torch.equal(fp4.gemm_fused(a, b, act=fp4.FP4_ACT_SILU)[0], fp4.gemm_fused(A, B, act=fp4.FP4_ACT_SILU)[0][16:48])
    assert fp4.fp4_gemm_fused_workspace_bytes(a, b) >= 0
    assert torch.equal(fp4.dequantize(a), fp4.dequantize(A)[16:48])


def test_wrap_without_amax_is_no_amax(fp4):
    """amax_from takes a tensor that has one: a tensor scale is no stand-in for it."""
    import torch
    say("wrap without amax")
    x = rand(3, 64, 512)
    q = fp4.quantize(x)
    w = fp4.QTensor.wrap(q.codes, q.scales, fp4.FP4_NVFP4, tscale=q.tscale)
    none = fp4.rmsnorm(x, torch.ones(512, device="cuda"))
    for bad in (w, none):
        with pytest.raises(ValueError, match="amax"):
            fp4.quantize(x, amax_from=bad)
        with pytest.raises(ValueError, match="amax"):
            fp4.quantize_dual(x, amax_from=bad)
        with pytest.raises(ValueError, match="amax"):
            fp4.quantize_2d(x, amax_from=bad)
    given = fp4.QTensor.wrap(q.codes, q.scales, fp4.FP4_NVFP4, amax=q.amax, tscale=q.tscale)
    again = fp4.quantize(x, amax_from=given)
    assert torch.equal(again.codes, q.codes) and torch.equal(again.tscale, q.tscale)


def test_wrap_as_an_output(fp4):
    """An output has an amax and a tensor scale of its own: neither a tensor without an amax nor one whose amax is its
    tensor scale is quantized into (one kernel reads the one while it writes the other)."""
    import torch
    say("wrap as an output")
    x = rand(4, 64, 512)
    want = fp4.quantize(x)
    s, t = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")

    def out(**kw):
        return fp4.QTensor.wrap(torch.empty_like(want.codes), torch.empty_like(want.scales), fp4.FP4_NVFP4, **kw)

    def into(q):
        fp4.fp4_quantize(x, fp4.FP4_AXIS_COLS, fp4.FP4_RTN, 0, 0, False, q)
    for bad in (out(tscale=s), out(amax=s, tscale=s)):
        with pytest.raises(ValueError, match="amax"):
            into(bad)
    good = out(amax=s, tscale=t)
    into(good)
    assert torch.equal(good.codes, want.codes) and torch.equal(t, want.tscale) and torch.equal(s, want.amax)


def test_wrap_without_tensor_scale(fp4):
    """An NVFP4 operand without its tensor scale is refused as every other argument is."""
    say("wrap without a tensor scale")
    q = fp4.quantize(rand(5, 64, 512))
    w = fp4.QTensor.wrap(q.codes, q.scales, fp4.FP4_NVFP4)
    for call in (lambda: fp4.gemm(w, q), lambda: fp4.gemm_fused(w, q), lambda: fp4.gemm_fused(q, w), lambda: fp4.dequantize(w)):
        with pytest.raises(ValueError, match="tscale"):
            call()
