"""Layer norm of rows far from zero: the statistics, and the gradients from the statistics that the call is given.

The backward call takes mean and rstd, so that its xhat = (x - mean) rstd is two roundings from the formula's, whatever
the offset: with U = 2^-24, half a step of fp32, at most 2 U of itself, where x rstd - mean rstd would be off by U times
|mean| rstd.
"""
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}
H, U = util.H, util.U
# additions one after the other in a row's sum: at most 16 in a thread and half of a pair, the two halves, 5 steps in a
# warp, 5 across the warps; then the product with the rounded 1 / c
DEPTH = 16 + 1 + 5 + 5 + 2


def forward_and_backward(x, w, bi, dy, eps=1e-6, per_batch=False):
    b, h, n, c = x.shape
    p = llsa.NormProblem(b, h, n, c, eps=eps, dtype=NUMBER[x.dtype], param_dtype=NUMBER[w.dtype], per_batch=per_batch)
    op = llsa.LayerNorm(p)
    for t in (op.y, op.mean, op.rstd, op.dx, op.dweight, op.dbias):
        t.fill_(math.nan)
    op.work.fill_(255)
    op.forward(x, w, bi)
    op.backward_pass(x, w, dy)
    torch.cuda.synchronize()
    return op


def compare(name, got, want, bound):
    util.check(name, got, want.cpu(), bound.cpu())


def check_statistics(op, x, eps):
    x = x.double()
    mean = x.mean(-1)
    xc = x - mean[..., None]
    rstd = 1 / torch.sqrt((xc * xc).mean(-1) + eps)
    e_mean = DEPTH * U * x.abs().mean(-1)
    # the variance: the rounded mean enters squared, the deviations by their own rounding; then 1 / sqrt to 2 ulp (4 U)
    e_rel = 0.5 * ((DEPTH + 6) * U + (e_mean * rstd) ** 2) + 6 * U
    compare("mean", op.mean, mean, e_mean)
    compare("rstd", op.rstd, rstd, rstd * e_rel)


def check_gradients(op, x, w, dy):
    """Against the formulas in 64 bits for the mean and rstd that the forward call left."""
    half, phalf = H[x.dtype], H[w.dtype]
    x, dy = x.double(), dy.double()
    w = w.double()
    mean, rstd = op.mean.double()[..., None], op.rstd.double()[..., None]
    xhat = (x - mean) * rstd
    e_xhat = 2 * U * xhat.abs()
    g = dy * w
    c1, c2 = g.mean(-1, keepdim=True), (g * xhat).mean(-1, keepdim=True)
    dx = rstd * (g - c1 - xhat * c2)
    e_c1 = (DEPTH + 2) * U * g.abs().mean(-1, keepdim=True)
    e_c2 = (DEPTH + 4) * U * (g * xhat).abs().mean(-1, keepdim=True) + (g.abs() * e_xhat).mean(-1, keepdim=True)
    e_dx = rstd * (4 * U * (g.abs() + c1.abs() + (xhat * c2).abs()) + e_c1 + xhat.abs() * e_c2 + e_xhat * c2.abs()) \
        + 4 * U * dx.abs()
    compare("dx", op.dx, dx, half * dx.abs() + (1 + half) * e_dx)
    rows = x[..., 0].numel()
    depth = rows + 40                          # a thread's rows, the threads and warps of a block, the blocks
    dw, db = (dy * xhat).sum((0, 1, 2)), dy.sum((0, 1, 2))
    e_dw = (dy.abs() * e_xhat).sum((0, 1, 2)) + depth * U * (dy * xhat).abs().sum((0, 1, 2))
    compare("dweight", op.dweight, dw, phalf * dw.abs() + (1 + phalf) * e_dw)
    compare("dbias", op.dbias, db, phalf * db.abs() + (1 + phalf) * depth * U * dy.abs().sum((0, 1, 2)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shift,eps", [(0.5, 1e-6), (1000.0, 1e-6), (-30000.0, 1e-5)])
# widths of every load (16 bytes, 8 or 4, single values), part of a warp, a warp and a block
@pytest.mark.parametrize("c", [2, 45, 64, 128, 250, 384, 602, 768, 1001, 1024, 1152, 2048, 4100, 5001, 8192, 16384])
def test_offset_rows(dtype, shift, eps, c):
    gen = torch.Generator().manual_seed(c)
    x = util.tokens(gen, 1, 1, 5, c, dtype, shift=shift)
    dy = util.tokens(gen, 1, 1, 5, c, dtype)
    w, bi = (1 + 0.3 * torch.randn(c, generator=gen)).cuda(), (0.3 * torch.randn(c, generator=gen)).cuda()
    op = forward_and_backward(x, w, bi, dy, eps)
    check_statistics(op, x, eps)
    check_gradients(op, x, w, dy)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [3.3, 100.1, 10000.7, 1e36])
@pytest.mark.parametrize("c", [64, 128, 8])
def test_constant_rows_of_any_value(dtype, value, c):
    """A row's sum is exact here (at most two values a thread and half of a pair, a power of two of them), and so is its
    mean: xhat is zero, and with it dweight and the last term of dx.  1e36: |mean| rstd is beyond fp32."""
    gen = torch.Generator().manual_seed(1)
    x = torch.full((1, 1, 7, c), value, device="cuda").to(dtype)
    dy = util.tokens(gen, 1, 1, 7, c, dtype)
    w, bi = torch.ones(c, device="cuda"), torch.arange(float(c), device="cuda")
    op = forward_and_backward(x, w, bi, dy)
    assert torch.equal(op.mean, x[..., 0].float())
    assert torch.equal(op.y, bi.to(dtype).expand_as(op.y))
    assert bool((op.dweight == 0).all())
    check_gradients(op, x, w, dy)


# every shape of a block-wide row's threads and loads, forward (128, 256: 1184 blocks, 512: 592, 1024: 296) and backward
# (fewer), with rows for at least three steps of each block and some blocks a fourth
WIDE = [(BF16, 768, 3557), (BF16, 1152, 3557), (BF16, 4096, 3557), (BF16, 5000, 1781), (BF16, 8192, 1781), (BF16, 16384, 1781),
        (BF16, 1012, 3557), (BF16, 2044, 3557), (BF16, 4092, 3557), (BF16, 8188, 1781), (BF16, 16380, 1781),
        (BF16, 330, 3557), (BF16, 602, 3557), (BF16, 1514, 3557), (BF16, 3010, 1781), (BF16, 6002, 1781), (BF16, 10002, 893),
        (BF16, 301, 3557), (BF16, 777, 3557), (BF16, 1501, 1781), (BF16, 3001, 1781), (BF16, 5001, 1781), (BF16, 9001, 893),
        (F32, 1000, 3557), (F32, 2048, 3557), (F32, 4096, 1781), (F32, 8192, 1781), (F32, 16384, 893),
        (F32, 330, 3557), (F32, 602, 3557), (F32, 1514, 3557), (F32, 3010, 1781), (F32, 6002, 1781), (F32, 10002, 893),
        (F32, 301, 3557), (F32, 777, 3557), (F32, 1501, 1781), (F32, 3001, 1781), (F32, 5001, 1781), (F32, 9001, 893)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,c,n", WIDE)
def test_many_rows_a_block(dtype, c, n):
    """The next rows fetched while these are worked on, the sums' buffers taken in turn, two rows a barrier."""
    gen = torch.Generator(device="cuda").manual_seed(c)
    x, dy = (torch.randn(1, 1, n, c, generator=gen, device="cuda").add_(s).to(dtype) for s in (0.5, 0.0))
    w, bi = (1 + 0.3 * torch.randn(c, generator=gen, device="cuda")), 0.3 * torch.randn(c, generator=gen, device="cuda")
    op = forward_and_backward(x, w, bi, dy)
    check_statistics(op, x, 1e-6)
    check_gradients(op, x, w, dy)
    # y from the statistics: the deviation, two products and a sum, each rounded, and the result's type
    xhat = (x.double() - op.mean.double()[..., None]) * op.rstd.double()[..., None]
    y = xhat * w.double() + bi.double()
    compare("y", op.y, y, H[dtype] * y.abs() + (1 + H[dtype]) * U * (4 * (xhat * w.double()).abs() + y.abs()))
