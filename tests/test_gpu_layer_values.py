"""NaN, infinities and padding in the operators around the FP4 product: what
one bad value may reach, and what it may not."""
import numpy as np
import pytest

import layer_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fp4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import fp4_fully_quantized_amd as m
    m.lib()
    return m


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def equal_codes(got, want):
    """The same codes, a NaN of either sign being one."""
    assert np.array_equal(np.where(want == 127, got & 127, got), want)


def check_mx8(q, x, what):
    """q is the 8-bit form of x (float64, finite or NaN) by the definition."""
    codes, scales = ref.mx8_encode(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales), what
    equal_codes(q.codes.cpu().numpy(), codes)


# ---------------------------------------------------------------- 8 bits
# Runs of NaN in a row of 96 (first column, length): inside a lane's eight columns, just those, across them, a
# whole block, a block and more, the end of the row.
RUNS = [(5, 1), (8, 7), (8, 8), (4, 8), (16, 16), (32, 32), (24, 48), (88, 8), (64, 32), (0, 96)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [96, 91])
def test_mx8_runs_of_nan_leave_their_block(fp4, kind, cols):
    """A NaN is E4M3's NaN and does not count for its block's maximum, however many of them there are, quiet or
    signalling."""
    import torch
    say("mx8 runs of NaN", kind, cols)
    x = np.random.default_rng(8).standard_normal((2 * len(RUNS), 96)).astype(np.float32) * 3
    t = torch.from_numpy(x).to({"bf16": torch.bfloat16, "f32": torch.float32}[kind])
    bits = t.view(torch.int16 if kind == "bf16" else torch.int32)
    for i, (at, n) in enumerate(RUNS):
        for row, quiet in ((2 * i, True), (2 * i + 1, False)):
            bits[row, at:at + n] = (0x7FC0 if quiet else 0x7F81) << (0 if kind == "bf16" else 16)
    t = t.to("cuda")[:, :cols]
    want = host(t)
    assert np.isnan(want).any()
    q = fp4.mx8_quantize(t)
    check_mx8(q, want, "mx8")
    back = host(fp4.mx8_dequantize(q))
    assert np.array_equal(np.isnan(back), np.isnan(want))


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("mnk", [(5, 96, 256), (300, 1096, 512), (4096, 4160, 256)])
def test_gemm_fused_checkpoint_of_nan(fp4, mnk, fmt):
    """Bias columns of NaN (a lane's eight, and a whole block): z is NaN there, the rest of each block is z's own
    8-bit form; few-tile kernel, tile edges and whole tiles."""
    import torch
    say("gemm fused z8 of NaN", mnk, fmt)
    M, N, K = mnk
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    A = fp4.quantize(torch.randn((M, K), generator=gen, device="cuda"), fmt=fmt)
    B = fp4.quantize(torch.randn((N, K), generator=gen, device="cuda") * 0.05, fmt=fmt)
    b = torch.randn(N, generator=gen, device="cuda")
    clean, q0 = fp4.gemm_fused(A, B, bias=b, checkpoint=True)
    bad = torch.zeros(N, dtype=torch.bool, device="cuda")
    bad[8:16] = bad[32:64] = bad[N - 32:N - 24] = True
    b[bad] = float("nan")
    y, q = fp4.gemm_fused(A, B, bias=b, checkpoint=True)
    assert torch.equal(torch.isnan(y), bad.expand(M, N)) and torch.equal(y[:, ~bad], clean[:, ~bad])
    rows = slice(0, M, max(1, M // 40))   # the definition on the host, on some of the rows
    codes, scales = ref.mx8_encode(host(y[rows]))
    assert np.array_equal(q.scales[rows].cpu().numpy(), scales)
    equal_codes(q.codes[rows].cpu().numpy(), codes)
    whole = fp4.mx8_quantize(y)
    assert torch.equal(q.codes, whole.codes) and torch.equal(q.scales, whole.scales)


@pytest.mark.parametrize("cols", [300, 5000, 20000])
def test_norm_checkpoint_of_nan(fp4, cols):
    """A residual row with a run of NaN: h8 is h's 8-bit form."""
    import torch
    say("norm h8 of NaN", cols)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    x = torch.randn((6, cols), generator=gen, device="cuda")
    r = torch.randn((6, cols), generator=gen, device="cuda")
    r[2, 40:48] = float("nan")
    r[4, 64:96] = float("nan")
    o = fp4.rmsnorm(x, torch.ones(cols, device="cuda"), residual=r, h8=True)
    check_mx8(o.h8, host(x + r), "h8")
    assert np.array_equal(np.isnan(host(fp4.mx8_dequantize(o.h8))), np.isnan(host(x + r)))


# ---------------------------------------------------------------- padding
@pytest.mark.parametrize("cols", [1, 40, 300, 5003, 20001])
def test_norm_pads_stay_zero(fp4, cols):
    """The codes past a row's last column are zeros also where the row's rstd is not finite: a NaN or an infinity in
    the row, a row of zeros with eps = 0."""
    import torch
    say("norm pads", cols)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randn((5, cols), generator=gen, device="cuda")
    x[1, 0] = float("nan")
    x[2] = 0
    x[3, cols - 1] = float("inf")
    g = torch.ones(cols, device="cuda")
    for residual in (None, torch.zeros_like(x)):
        o = fp4.rmsnorm(x, g, eps=0.0, residual=residual, y8=True, h8=True)
        assert torch.isnan(o.y[1:3]).all() and torch.isfinite(o.y[[0, 4]]).all()
        for q, v in ((o.y8, o.y), (o.h8, x)):
            assert not q.codes[:, cols:].any()
            for r in (0, 1, 2, 4):   # the infinity's block stands for NaN whatever its codes
                codes, scales = ref.mx8_encode(host(v[r:r + 1]))
                assert np.array_equal(q.scales[r:r + 1].cpu().numpy(), scales)
                equal_codes(q.codes[r:r + 1].cpu().numpy(), codes)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("cols", [1, 40, 91, 2501])
def test_pads_of_a_block_with_an_infinity(fp4, kind, cols):
    """Zeros there too: in a matrix's 8-bit form, and in a product's checkpoint."""
    import torch
    say("pads, infinity", kind, cols)
    x = torch.ones((9, cols), device="cuda").to({"bf16": torch.bfloat16, "f32": torch.float32}[kind])
    x[::2, cols - 1] = float("inf")
    q = fp4.mx8_quantize(x)
    assert not q.codes[:, cols:].any() and (q.scales[::2, -1] == 255).all()
    assert torch.isnan(fp4.mx8_dequantize(q)[::2, cols - 1]).all()
    for rows in (9, 2500):   # the kernel of few tiles, and the tiled one's edges
        A, B = fp4.quantize(torch.ones((rows, 256), device="cuda")), fp4.quantize(torch.ones((cols, 256), device="cuda"))
        b = torch.zeros(cols, device="cuda")
        b[cols - 1] = float("inf")
        _, z = fp4.gemm_fused(A, B, bias=b, checkpoint=True)
        assert not z.codes[:, cols:].any() and (z.scales[:, -1] == 255).all()


# ---------------------------------------------------------------- amax
def largest(v):
    """max |v| over the values that are no NaN (0 if none)."""
    a = np.abs(host(v))
    return float(np.where(np.isnan(a), 0.0, a).max())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 40), (6, 500), (37, 4096), (1500, 1003), (5, 20000)])
def test_norm_amax_with_nan(fp4, rows, cols, kind):
    """amax is max |y| over the stored values that are no NaN, whether y or its 8-bit form is stored: what quantize's
    own pass over them finds."""
    import torch
    say("norm amax with NaN", rows, cols, kind)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x = torch.randn((rows, cols), generator=gen, device="cuda").to({"bf16": torch.bfloat16, "f32": torch.float32}[kind])
    g = torch.randn(cols, generator=gen, device="cuda")
    for where in ("gamma", "row", "all", "infinity"):
        xx, gg = x.clone(), g.clone()
        if where == "gamma":
            gg[3] = float("nan")
        elif where == "row":
            xx[rows // 2, 7] = float("nan")
        elif where == "all":
            gg[:] = float("nan")
        else:
            gg[5] = float("inf")
        for y, y8 in ((True, False), (False, True), (True, True)):
            o = fp4.rmsnorm(xx, gg, y=y, y8=y8, amax=True)
            stored = o.y if y else fp4.mx8_dequantize(o.y8)
            assert float(o.amax) == largest(stored), (where, y, y8)
        if cols % 16 == 0 and where in ("gamma", "row", "all"):
            n = fp4.rmsnorm(xx, gg, amax=True)
            a, b = fp4.quantize(n.y, amax_from=n), fp4.quantize(n.y)
            assert torch.equal(a.amax, b.amax) and torch.equal(a.tscale, b.tscale), where
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales), where


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 40), (70, 1001), (513, 2504)])
def test_act_backward_amax_with_nan(fp4, rows, cols, kind):
    import torch
    say("act backward amax with NaN", rows, cols, kind)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[kind]
    z = torch.randn((rows, cols), generator=gen, device="cuda").to(t)
    dy = torch.randn((rows, cols), generator=gen, device="cuda").to(t)
    for act in (0, 1, 2, 3):
        for bad in (float("nan"), float("inf")):
            d = dy.clone()
            d[rows // 2, 8:17] = bad
            z[rows // 2, 8:17] = 1.0
            o = fp4.act_backward(d, z, act, amax=True)
            assert float(o.amax) == largest(o.dz), (act, bad)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 2048), (700, 4096)])
def test_tensor_amax_with_nan(fp4, rows, cols, kind):
    """The largest magnitude of the values that are no NaN, of a contiguous matrix as of a strided one: a NaN hides
    none of the values beside it."""
    import torch
    say("tensor amax with NaN", rows, cols, kind)
    t = {"bf16": torch.bfloat16, "f32": torch.float32}[kind]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    wide = torch.randn((rows, cols + 8), generator=gen, device="cuda").to(t)
    bits = wide.view(torch.int16 if kind == "bf16" else torch.int32)
    shift = 0 if kind == "bf16" else 16
    r = rows // 2
    wide[r, 3] = -1000.0
    bits[r, 4:6] = 0x7FC0 << shift
    bits[r, 6] = 0x7F81 << shift    # signalling
    bits[r, 7] = (0xFFFF - 0x10000) << shift
    out = torch.empty(1, device="cuda")
    for src in (wide[:, :cols], wide[:, :cols].contiguous()):
        fp4.fp4_tensor_amax(src, out)
        assert float(out) == 1000.0
    for big in (float("inf"), float("-inf")):
        wide[r, 3] = big
        for src in (wide[:, :cols], wide[:, :cols].contiguous()):
            fp4.fp4_tensor_amax(src, out)
            assert float(out) == float("inf")
    wide[:] = float("nan")
    fp4.fp4_tensor_amax(wide[:, :cols].contiguous(), out)
    assert float(out) == 0.0
