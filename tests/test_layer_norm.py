"""Layer norm: the formulas in 64 bits, widths, layouts, weights and refusals."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}


def run_case(dtype, pt, b, h, n, c, layout="bhnd", per_batch=False, weight=True, bias=True, eps=1e-6, shift=0.5,
             scale=1.0, seed=0, token_major=None):
    gen = torch.Generator().manual_seed(seed)
    x = util.tokens(gen, b, h, n, c, dtype, layout, shift=shift, scale=scale)
    dy = util.tokens(gen, b, h, n, c, dtype, layout)
    shape = (b, c) if per_batch else (c,)
    w = (1 + 0.3 * torch.randn(shape, generator=gen)).to(pt).cuda() if weight else None
    bi = (0.3 * torch.randn(shape, generator=gen)).to(pt).cuda() if bias else None
    p = llsa.NormProblem(b, h, n, c, eps=eps, dtype=NUMBER[dtype], param_dtype=NUMBER[pt], per_batch=per_batch)
    op = llsa.LayerNorm(p, token_major=layout != "bhnd" if token_major is None else token_major)
    for t in (op.y, op.mean, op.rstd, op.dx, op.dweight, op.dbias):
        t.fill_(math.nan)
    op.work.fill_(255)
    op.forward(x, w, bi)
    op.backward_pass(x, w, dy)
    torch.cuda.synchronize()
    ref = util.norm_reference(x, w, bi, eps, dtype, pt, per_batch, dy)
    for name, (want, bound) in ref.items():
        util.check(name, getattr(op, name), want, bound)
    return op


TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]
# every width at which the kernels change their shape, its neighbours, and odd ones
WIDTHS = [1, 2, 7, 8, 9, 17, 32, 33, 45, 64, 72, 100, 127, 128, 129, 256, 257, 264, 384, 388, 512, 520, 768, 1000, 1001, 1024,
          1032, 1152, 2048, 2056, 4096, 4104, 5001, 8192, 8200, 16383, 16384, 301, 777, 1501, 3001, 9001, 12, 20, 50, 92, 154, 244, 330, 602, 1012, 1514, 3010, 6004, 10002]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
@pytest.mark.parametrize("c", WIDTHS)
def test_widths(dtype, pt, c):
    run_case(dtype, pt, 1, 1, 37 if c > 1 else 5, c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
@pytest.mark.parametrize("n", [1, 2, 31, 257, 5000])
@pytest.mark.parametrize("c", [64, 384, 101])
def test_rows(dtype, pt, n, c):
    run_case(dtype, pt, 2, 1, n, c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "fused"])
@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("c", [64, 40, 33, 1200])
def test_layouts_and_modulation(dtype, pt, layout, per_batch, c):
    run_case(dtype, pt, 3, 5, 43, c, layout=layout, per_batch=per_batch)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("c", [64, 2048])
def test_without_weights(dtype, pt, weight, bias, c):
    run_case(dtype, pt, 2, 1, 50, c, weight=weight, bias=bias)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
@pytest.mark.parametrize("shift,scale,eps", [(1000.0, 1.0, 1e-6), (0.0, 1e-6, 1e-5), (0.0, 1e15, 1e-6), (3.0, 1.0, 0.0)])
def test_offsets_and_scales(dtype, pt, shift, scale, eps):
    run_case(dtype, pt, 1, 2, 60, 384, shift=shift, scale=scale, eps=eps)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
def test_input_and_output_layouts_may_differ(dtype, pt):
    run_case(dtype, pt, 2, 6, 70, 64, layout="fused", token_major=False)
    run_case(dtype, pt, 2, 6, 70, 64, layout="bhnd", token_major=True)


@pytest.mark.gpu
@pytest.mark.parametrize("pt", [BF16, F32])
@pytest.mark.parametrize("c,first", [(64, 0), (64, 8), (40, 3), (2048, 1)])
def test_modulation_from_a_projection(pt, c, first):
    """weight and bias as slices of one [batch, several c] output, on 16-byte boundaries and off them."""
    gen = torch.Generator().manual_seed(11)
    b, n = 3, 41
    x, dy = (util.tokens(gen, b, 1, n, c, BF16) for _ in range(2))
    wide = torch.randn(b, first + 6 * c, generator=gen).to(pt).cuda()
    w, bi = wide[:, first + c:first + 2 * c], wide[:, first + 4 * c:first + 5 * c]
    p = llsa.NormProblem(b, 1, n, c, param_dtype=NUMBER[pt], per_batch=True)
    op = llsa.LayerNorm(p)
    op.forward(x, w, bi)
    op.backward_pass(x, w, dy)
    for name, (want, bound) in util.norm_reference(x, w, bi, p.eps, BF16, pt, True, dy).items():
        util.check(name, getattr(op, name), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("c", [64, 33])
def test_offsets_beyond_32_bits(c):
    gen = torch.Generator().manual_seed(12)
    b, n = 2, 50
    far = (1 << 31) + 4096
    big = torch.empty(far + 4 * n * c, dtype=BF16, device="cuda")
    x, y, dy, dx = (big.as_strided((b, 1, n, c), (far, n * c, c, 1), i * n * c) for i in range(4))
    for t in (x, dy):
        t.copy_(torch.randn(t.shape, generator=gen).to(BF16))
    w = torch.randn(c, generator=gen).cuda()
    p = llsa.NormProblem(b, 1, n, c, param_dtype=llsa.FP32)
    mean, rstd = (torch.empty(b, 1, n, device="cuda") for _ in range(2))
    llsa.layer_norm_fwd(p, x, w, None, y, mean, rstd)
    llsa.layer_norm_bwd(p, x, dy, w, mean, rstd, dx=dx)
    ref = util.norm_reference(x, w, None, p.eps, BF16, F32, False, dy)
    util.check("y", y, *ref["y"])
    util.check("dx", dx, *ref["dx"])


@pytest.mark.gpu
def test_constant_rows():
    """No variance: xhat is zero, y the bias; eps keeps the gradients finite."""
    p = llsa.NormProblem(1, 1, 4, 64, dtype=llsa.FP32)
    op = llsa.LayerNorm(p)
    x = torch.full((1, 1, 4, 64), 5.0, device="cuda")
    w, b = torch.ones(64, device="cuda"), torch.arange(64., device="cuda")
    op.forward(x, w, b)
    assert torch.equal(op.y, b.expand_as(op.y))
    dy = torch.randn(1, 1, 4, 64, device="cuda")
    op.backward_pass(x, w, dy)
    assert bool(torch.isfinite(op.dx).all()) and bool((op.dweight == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("c", [64, 1001, 4096])
def test_in_place(c):
    gen = torch.Generator().manual_seed(1)
    p = llsa.NormProblem(2, 1, 33, c)
    x, dy = (util.tokens(gen, 2, 1, 33, c, BF16) for _ in range(2))
    w, b = (torch.randn(c, generator=gen).to(BF16).cuda() for _ in range(2))
    op = llsa.LayerNorm(p)
    op.forward(x, w, b)
    dx = op.backward_pass(x, w, dy)[0]
    x2, g2 = x.clone(), dy.clone()
    llsa.layer_norm_fwd(p, x2, w, b, x2)
    assert torch.equal(x2, op.y)
    llsa.layer_norm_bwd(p, x, g2, w, op.mean, op.rstd, dx=g2)
    assert torch.equal(g2, dx)


@pytest.mark.gpu
def test_parts_of_the_backward():
    """dx alone, a weight's gradient alone: the same values as together."""
    gen = torch.Generator().manual_seed(2)
    p = llsa.NormProblem(2, 3, 50, 64, per_batch=True)
    x, dy = (util.tokens(gen, 2, 3, 50, 64, BF16) for _ in range(2))
    w = torch.randn(2, 64, generator=gen).to(BF16).cuda()
    op = llsa.LayerNorm(p)
    op.forward(x, w)
    want = [t.clone() for t in op.backward_pass(x, w, dy)]
    out = [torch.zeros_like(t) for t in want]
    llsa.layer_norm_bwd(p, x, dy, w, op.mean, op.rstd, dx=out[0])
    llsa.layer_norm_bwd(p, x, dy, w, op.mean, op.rstd, dweight=out[1], workspace=op.work)
    llsa.layer_norm_bwd(p, x, dy, w, op.mean, op.rstd, dbias=out[2], workspace=op.work)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,pt", TYPES)
def test_gradients_against_differences(dtype, pt):
    gen = torch.Generator().manual_seed(3)
    b, h, n, c = 1, 2, 9, 72
    x, dy = (util.tokens(gen, b, h, n, c, dtype) for _ in range(2))
    w, bi = ((1 + 0.3 * torch.randn(c, generator=gen)).to(pt).cuda() for _ in range(2))
    p = llsa.NormProblem(b, h, n, c, dtype=NUMBER[dtype], param_dtype=NUMBER[pt])
    op = llsa.LayerNorm(p)
    op.forward(x, w, bi)
    got = [t.cpu().double() for t in op.backward_pass(x, w, dy)]
    at = [t.cpu().double() for t in (x, w, bi)]
    g = dy.cpu().double()

    def value(x, w, bi):
        xc = x - x.mean(-1, keepdim=True)
        return float(((xc / torch.sqrt((xc * xc).mean(-1, keepdim=True) + p.eps) * w + bi) * g).sum())

    bounds = util.norm_reference(x, w, bi, p.eps, dtype, pt, False, dy)
    for i, name in enumerate(("dx", "dweight", "dbias")):
        u = torch.randn(got[i].shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + e * u, at[i] - e * u
        slope = (value(*up) - value(*down)) / (2 * e)
        allowed = float((bounds[name][1] * u.abs()).sum()) + 1e-6 * (1 + abs(slope))
        assert abs(float((got[i] * u).sum()) - slope) <= allowed, name


@pytest.mark.gpu
@pytest.mark.parametrize("c,layout", [(64, "bnhd"), (101, "bnhd"), (2056, "bhnd")])
def test_guards_bits_streams_and_graphs(c, layout):
    """Nothing outside the outputs changes; the same bits from dirty buffers, on another stream and replayed."""
    gen = torch.Generator().manual_seed(4)
    b, h, n = 2, 3, 61
    x, dy = (util.tokens(gen, b, h, n, c, BF16, layout) for _ in range(2))
    w, bi = (torch.randn(c, generator=gen).cuda() for _ in range(2))
    p = llsa.NormProblem(b, h, n, c, param_dtype=llsa.FP32)
    op = llsa.LayerNorm(p, token_major=layout == "bnhd")
    op.forward(x, w, bi)
    op.backward_pass(x, w, dy)
    names = ("y", "mean", "rstd", "dx", "dweight", "dbias")
    want = {k: getattr(op, k).clone() for k in names}
    guard = 4096
    whole = {}
    for k in names + ("work",):
        t = getattr(op, k)
        nbytes = t.numel() * t.element_size()
        flat = torch.full((nbytes + 2 * guard,), 255, dtype=torch.uint8, device="cuda")
        whole[k] = (flat, nbytes)
        inner = flat[guard:guard + nbytes].view(t.dtype)
        setattr(op, k, inner.as_strided(t.shape, t.stride()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.forward(x, w, bi, stream=side)
    op.backward_pass(x, w, dy, stream=side)
    side.synchronize()
    for k in names:
        assert torch.equal(getattr(op, k), want[k]), k
    for flat, nbytes in whole.values():
        assert bool((flat[:guard] == 255).all()) and bool((flat[guard + nbytes:] == 255).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(x, w, bi)
        op.backward_pass(x, w, dy)
    for k in names:
        getattr(op, k).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for k in names:
        assert torch.equal(getattr(op, k), want[k]), k
    x.mul_(3)
    graph.replay()
    torch.cuda.synchronize()
    for k, (v, bound) in util.norm_reference(x, w, bi, p.eps, BF16, F32, False, dy).items():
        util.check(k, getattr(op, k), v, bound)


# ------------------------------------------------------------------ refusals (no GPU)

def problem(**kw):
    base = dict(batch=2, heads=3, n=10, c=64)
    base.update(kw)
    return llsa.NormProblem(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(c=1), 0), (dict(c=16384), 0), (dict(param_dtype=llsa.FP32), 0), (dict(dtype=llsa.FP32), 0),
    (dict(per_batch=True), 0), (dict(eps=0.0), 0),
    (dict(c=16385), 7), (dict(c=0), 1), (dict(batch=0), 1), (dict(heads=0), 1), (dict(n=0), 1),
    (dict(dtype=llsa.FP32, param_dtype=llsa.BF16), 1), (dict(dtype=3), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(eps=math.inf), 1), (dict(batch=1 << 16, heads=1 << 15), 2), (dict(batch=70000, per_batch=True), 2),
])
def test_validation(kw, status):
    assert llsa.norm_validate(problem(**kw)) == status


@pytest.mark.parametrize("name,strides,status", [
    ("x", (0, 640, 64), 0), ("x", (1921, 641, 65), 0), ("y", (0, 640, 64), 1), ("dx", (1920, 640, 63), 1),
    ("y", (1920, 64, 192), 0), ("dy", (1920, -640, 64), 1), ("x", (1 << 40, 640, 64), 2),
])
def test_stride_rules(name, strides, status):
    c = problem().cp()
    s = getattr(c, name)
    s.batch, s.head, s.token = strides
    assert llsa.lib().llsa_norm_validate(ctypes.byref(c)) == status


def test_entry_points_reject_bad_buffers_before_launch():
    L, good = llsa.lib(), 1 << 20            # never dereferenced
    c = problem().cp()
    r = ctypes.byref(c)

    def fwd(i, x):
        a = [good] * 6
        a[i] = x
        return L.llsa_layer_norm_fwd(r, *a, None)

    assert fwd(0, None) == 1 and fwd(3, None) == 1
    for i in range(6):
        assert fwd(i, good + 1) == 3, i

    def bwd(i, x):
        a = [good] * 9
        a[i] = x
        return L.llsa_layer_norm_bwd(r, *a, None)

    for i in (0, 1, 3, 4, 8):
        assert bwd(i, None) == 1, i
    for i in range(9):
        assert bwd(i, good + 1) == 3, i
    assert bwd(8, good + 8) == 3
    a = [good] * 9
    a[5] = a[6] = a[7] = None
    assert L.llsa_layer_norm_bwd(r, *a, None) == 1
    assert L.llsa_norm_query_sizes(r, None) == 1


def test_the_binding_checks_its_tensors():
    p = problem()
    x, w = torch.zeros(p.shape, dtype=BF16), torch.zeros(64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.layer_norm_fwd(p, x, w, w, x)
    with pytest.raises(ValueError, match="weight"):
        llsa.layer_norm_fwd(p, x, w.float(), w, x)
    with pytest.raises(ValueError, match="bias"):
        llsa.layer_norm_fwd(p, x, w, w[:5], x)
    with pytest.raises(ValueError, match="expanded"):
        llsa.layer_norm_fwd(problem(per_batch=True), x, w.expand(2, 64), None, x)
    with pytest.raises(ValueError, match="shape"):
        llsa.layer_norm_fwd(p, x[..., :8], w, w, x)
    with pytest.raises(ValueError, match="expanded"):
        llsa.layer_norm_fwd(p, x[:1, :1, :1].expand(p.shape), w, w, x)
    with pytest.raises(llsa.LLSAError):
        llsa.LayerNorm(problem(c=20000), device="cpu")
