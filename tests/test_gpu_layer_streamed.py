"""The row-wise operators on matrices past the caches' size, whose accesses are
marked as not to be kept: every row's result is that of the same rows as a smaller
matrix, and the first and last rows, and all sums over rows, agree with 64 bits."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import say
from layer_ref import U, UB

pytestmark = pytest.mark.gpu

# 168 MB of fp32 and 169 of bf16, rows on 16 bytes, a last chunk and block that are not whole, rows not a multiple of
# anything; and rows of one wave.
SIZES = {"f32": [(10247, 4100), (81001, 520)], "bf16": [(20500, 4120), (162001, 520)]}


@pytest.fixture(scope="module")
def fp4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_fully_quantized_amd as m
    m.lib()
    return m


def rand(seed, kind, *shape, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to({"f32": torch.float32, "bf16": torch.bfloat16}[kind])


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def ends(t):
    import torch
    return torch.cat((t[:40], t[-40:]))


def parts(rows):
    """Ranges of rows whose matrices stay in the caches."""
    step = rows // 3 + 1
    return [slice(at, min(at + step, rows)) for at in range(0, rows, step)]


CASES = [(kind, *shape) for kind in SIZES for shape in SIZES[kind]]


@pytest.mark.parametrize("kind,rows,cols", CASES)
def test_8_bits(fp4, kind, rows, cols):
    import torch
    say("8 bits, streamed", kind, rows, cols)
    x = rand(1, kind, rows, cols, scale=3.0)
    q = fp4.mx8_quantize(x)
    for p in parts(rows):
        s = fp4.mx8_quantize(x[p])
        assert torch.equal(s.codes, q.codes[p]) and torch.equal(s.scales, q.scales[p])
    codes, scales = ref.mx8_encode(host(ends(x)))
    assert np.array_equal(ends(q.scales).cpu().numpy(), scales) and np.array_equal(ends(q.codes).cpu().numpy(), codes)
    back = fp4.mx8_dequantize(q, x.dtype)
    assert np.array_equal(host(ends(back)), ref.mx8_decode(codes, scales, cols))
    for p in parts(rows):
        assert torch.equal(back[p], fp4.mx8_dequantize(fp4.MX8Tensor.wrap(q.codes[p], q.scales[p], cols), x.dtype))


@pytest.mark.parametrize("kind,rows,cols", CASES)
def test_norm(fp4, kind, rows, cols):
    """h, y, h8 and y8; then the backward pass from the matrix h with dres, and from h8."""
    import torch
    say("norm, streamed", kind, rows, cols)
    half = UB if kind == "bf16" else U
    x, r = rand(1, kind, rows, cols, scale=2.0), rand(2, kind, rows, cols)
    g = 1 + 0.1 * rand(3, "f32", cols)
    o = fp4.rmsnorm(x, g, residual=r, y8=True, h8=True, amax=True)
    for p in parts(rows):
        s = fp4.rmsnorm(x[p], g, residual=r[p], y8=True, h8=True)
        for a, b in ((o.h, s.h), (o.y, s.y), (o.rstd, s.rstd), (o.y8.codes, s.y8.codes), (o.y8.scales, s.y8.scales),
                     (o.h8.codes, s.h8.codes), (o.h8.scales, s.h8.scales)):
            assert torch.equal(a[p], b)
    assert float(o.amax) == float(o.y.abs().max())
    h = (host(ends(x)) + host(ends(r))).astype(np.float32).astype(np.float64)
    rstd, y = ref.norm(h, host(g), 1e-5)
    sums = (48 + 22 + 3) / 2 + 8   # the row's sum, at most 48 additions in a lane; half of it reaches rstd
    assert (np.abs(host(ends(o.h)) - h) <= half * np.abs(h)).all()
    assert (np.abs(host(ends(o.rstd[:, None]))[:, 0] - rstd) <= sums * U * rstd).all()
    assert (np.abs(host(ends(o.y)) - y) <= (sums * U + half * (1 + 1e-5)) * np.abs(y) + 1e-37).all()
    dy, dres = rand(4, kind, rows, cols, scale=1e-3), rand(5, kind, rows, cols, scale=1e-3)
    for kept in (o.h, o.h8):
        dx, dgamma = fp4.rmsnorm_backward(dy, kept, g, o.rstd, dres=dres)
        for p in parts(rows):
            k = kept[p] if kept is o.h else fp4.MX8Tensor.wrap(kept.codes[p], kept.scales[p], cols)
            assert torch.equal(dx[p], fp4.rmsnorm_backward(dy[p], k, g, o.rstd[p], dres=dres[p])[0])
        hv = kept if kept is o.h else fp4.mx8_dequantize(kept)
        wx, _, mag, _ = ref.norm_grad(host(ends(dy)), host(ends(hv)), host(g), host(ends(o.rstd[:, None]))[:, 0])
        wx = wx + host(ends(dres))
        assert (np.abs(host(ends(dx)) - wx) <= 80 * U * mag + 2 * U * np.abs(wx) + half * np.abs(wx) * (1 + 1e-5) + 1e-37).all()
        t = dy.double() * (hv.double() * o.rstd.double()[:, None])
        # a lane adds its workgroup's rows (of at least 256), then at most 64 + 16 partial rows
        assert ((dgamma.double() - t.sum(0)).abs() <= (rows / 256 + 90) * U * t.abs().sum(0) + 1e-37).all()
        del t, hv


@pytest.mark.parametrize("kind,rows,cols", CASES)
def test_act_backward(fp4, kind, rows, cols):
    import torch
    say("act backward, streamed", kind, rows, cols)
    half = UB if kind == "bf16" else U
    z, dy = rand(1, kind, rows, cols, scale=2.0), rand(2, kind, rows, cols, scale=1e-3)
    for act in (fp4.FP4_ACT_GELU, fp4.FP4_ACT_SILU):
        for kept in (z, fp4.mx8_quantize(z)):
            o = fp4.act_backward(dy, kept, act, amax=True)
            for p in parts(rows):
                k = kept[p] if kept is z else fp4.MX8Tensor.wrap(kept.codes[p], kept.scales[p], cols)
                assert torch.equal(o.dz[p], fp4.act_backward(dy[p], k, act).dz)
            zv = z if kept is z else fp4.mx8_dequantize(kept)
            want = host(ends(dy)) * ref.act_slope(host(ends(zv)), act)
            tol = 16 * U * np.abs(host(ends(dy)))
            assert (np.abs(host(ends(o.dz)) - want) <= tol + half * (np.abs(want) + tol) + 1e-37).all()
            assert float(o.amax) == float(o.dz.abs().max())
            zd = zv.double()
            t = zd if act == fp4.FP4_ACT_SILU else ref.GELU_2C * zd * (1 + ref.GELU_A * zd * zd)
            rate = 1.0 if act == fp4.FP4_ACT_SILU else ref.GELU_2C * (1 + 3 * ref.GELU_A * zd * zd)
            s = torch.sigmoid(t)
            d = dy.double() * (s + zd * s * (1 - s) * rate)
            tol = 16 * U * dy.double().abs()
            chain = rows / 8 + 80
            assert ((o.dbias.double() - d.sum(0)).abs() <= (tol + chain * U * (d.abs() + tol)).sum(0) + 1e-37).all()
            del zd, t, s, d, rate, tol
