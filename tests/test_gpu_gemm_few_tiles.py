"""The FP4 product of few tiles on its two largest tile shapes (64 x 32 and 64 x 64
outputs a workgroup, which the rule on sizes picks from about a hundred rows on)
against the product in 64 bits: ragged last tiles of one row and four columns, one
step of K and several a wave, whole tiles, every kind of epilogue."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import say
from layer_ref import U, UB

pytestmark = pytest.mark.gpu

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


@pytest.fixture(scope="module")
def fp4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_fully_quantized_amd as m
    m.lib()
    return m


def decode(q):
    """The values of a quantized matrix in float64, from the format: codes times block scales times tensor scale."""
    c, s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    v = E2M1[np.stack((c & 15, c >> 4), -1)].reshape(q.rows, s.shape[1], -1)
    if q.fmt == 0:
        scale = ref.E4M3[s] * float(q.tscale)
    else:
        scale = 2.0 ** (s.astype(np.float64) - 127)
    return (v * scale[..., None]).reshape(q.rows, q.cols)


def matrix(seed, *shape, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda") * scale


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


# (M, N, K): 64 x 32 outputs a workgroup, then 64 x 64. Both formats pick the same on these.
SHAPES = [(129, 2500, 128), (129, 2570, 384), (330, 1100, 1152), (130, 2500, 4096), (128, 4096, 2176),
          (257, 2500, 128), (300, 2500, 384), (700, 1001, 1152), (257, 2570, 4096), (512, 4096, 640)]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("mnk", SHAPES)
def test_gemm_fused_large_few_tile_shapes(fp4, mnk, fmt):
    import torch
    M, N, K = mnk
    A, B = fp4.quantize(matrix(1, M, K), fmt=fmt), fp4.quantize(matrix(2, N, K, scale=0.15), fmt=fmt)
    a, b = decode(A), decode(B)
    dot, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    tol = 1e-5 * mag                      # the product's own bound
    kinds = {"f32": torch.float32, "bf16": torch.bfloat16}
    for act, bias, residual, z8, out in ((0, None, None, False, "f32"), (1, "f32", "bf16", False, "bf16"),
                                         (2, "bf16", "f32", True, "f32"), (3, "f32", "bf16", True, "bf16"),
                                         (3, "bf16", None, False, "f32")):
        say("few tiles", mnk, fmt, act, bias, residual, z8, out)
        bt = matrix(3, N).to(kinds[bias]) if bias else None
        rt = matrix(4, M, N + 3, scale=2.0).to(kinds[residual])[:, 1:N + 1] if residual else None
        y, q = fp4.gemm_fused(A, B, bias=bt, act=act, residual=rt, checkpoint=z8, dtype=kinds[out])
        z = dot + (host(bt) if bias else 0.0)
        tz = tol + 2 * U * (np.abs(z) + tol)
        want = ref.act(z, act) + (host(rt) if residual else 0.0)
        # slopes stay under 1.13; an activation's own error is 16 U |z|
        tw = 1.13 * tz + 16 * U * np.abs(z) + U * (np.abs(want) + tz) + 1e-37
        got = host(y)
        worst = np.abs(got - want) / (tw + (UB if out == "bf16" else U) * (np.abs(want) + tw))
        assert np.isfinite(got).all() and worst.max() <= 1, f"off by {worst.max()} of the tolerance"
        if z8:
            ref.check_mx8_of(z, tz + 1e-37, q.codes.cpu().numpy(), q.scales.cpu().numpy(), f"z8 {mnk}")
        again, _ = fp4.gemm_fused(A, B, bias=bt, act=act, residual=rt, checkpoint=z8, dtype=kinds[out])
        assert torch.equal(again, y)
    # an output inside a wider matrix, over the residual: nothing else is written
    wide = torch.full((M + 1, N + 5), 7.0, device="cuda")
    keep = matrix(5, M, N)
    wide[:M, 2:2 + N] = keep
    fp4.fp4_gemm_fused(A, B, wide[:M, 2:2 + N], residual=wide[:M, 2:2 + N])
    want = dot + host(keep)
    assert (np.abs(host(wide[:M, 2:2 + N]) - want) <= tol + 2 * U * (np.abs(dot) + np.abs(want) + tol)).all()
    assert (wide[:, :2] == 7).all() and (wide[:, 2 + N:] == 7).all() and (wide[M] == 7).all()
