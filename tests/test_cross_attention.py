"""Cross attention to an encoder's states: the formulas in 64 bits, masks, layouts, splits and refusals."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}


def run_case(dtype, b, h, hk, nq, nk, d, layout="bhnd", lens=None, mask=None, scale=None, train=True, seed=0,
             fill=None, sharp=1.0, dO_layout=None, key_layout=None):
    """One forward and backward, checked element by element; returns the operator."""
    gen = torch.Generator().manual_seed(seed)
    q = util.tokens(gen, b, h, nq, d, dtype, layout, scale=sharp)
    k = util.tokens(gen, b, hk, nk, d, dtype, key_layout or layout, shift=0.25)
    v = util.tokens(gen, b, hk, nk, d, dtype, key_layout or layout)
    g = util.tokens(gen, b, h, nq, d, dtype, dO_layout or layout)
    kv_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    key_mask = None if mask is None else torch.tensor(mask).to(torch.uint8).cuda()
    ok = util.valid_keys(b, nk, kv_len, key_mask)
    if fill is not None:
        for t in (k, v):
            t.masked_fill_(~ok[:, None, :, None].cuda(), fill)
    p = llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk, scale=scale, dtype=NUMBER[dtype])
    op = llsa.CrossAttention(p, backward=train, token_major=layout != "bhnd")
    for name in ("o", "lse", "dq", "dk", "dv", "work"):
        t = getattr(op, name, None)
        if t is not None:
            t.view(torch.uint8).fill_(255) if name == "work" else t.fill_(math.nan)
    op.forward(q, k, v, kv_len=kv_len, key_mask=key_mask)
    if train:
        op.backward_pass(q, k, v, g, kv_len=kv_len, key_mask=key_mask)
    torch.cuda.synchronize()
    assert llsa.device_error() == 0
    ref = util.cross_reference(q, k, v, ok, p.scale, g if train else None)
    for name, (want, bound) in ref.items():
        util.check(name, getattr(op, name), want, bound)
    return op


# sizes around the tiles (16, 32, 64, 128), one of each, long axes
SIZES = [(1, 1), (1, 2), (2, 1), (3, 17), (64, 64), (65, 63), (128, 128), (129, 127), (127, 257), (256, 77),
         (300, 129), (1, 700), (700, 1), (31, 1031), (1030, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("nq,nk", SIZES)
def test_lengths(dtype, nq, nk):
    run_case(dtype, 2, 2, 2, nq, nk, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 80, 96, 104, 120, 128])
def test_head_dimensions(dtype, d):
    run_case(dtype, 1, 3, 3, 150, 140, d, layout="bnhd")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("h,hk,nq", [(4, 2, 130), (8, 1, 5), (6, 3, 1), (16, 2, 1), (12, 1, 40), (5, 5, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_heads(dtype, h, hk, nq, d):
    run_case(dtype, 2, h, hk, nq, 200, d, layout="bnhd")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,key_layout,dO_layout", [("bnhd", "fused", "bhnd"), ("bhnd", "bnhd", "fused"),
                                                         ("fused", "fused", "fused")])
@pytest.mark.parametrize("d", [64, 72])
def test_strides(dtype, layout, key_layout, dO_layout, d):
    run_case(dtype, 2, 3, 3, 70, 90, d, layout=layout, key_layout=key_layout, dO_layout=dO_layout)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", [None, math.nan, math.inf, -3e38])
@pytest.mark.parametrize("nq", [1, 200])
def test_lengths_of_the_keys(dtype, fill, nq):
    """From none to all, and beyond the ends (clamped); what stands behind a length never matters."""
    run_case(dtype, 7, 2, 2, nq, 300, 64, lens=[0, 1, 127, 129, 300, 400, -5], fill=fill)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("fill", [None, math.nan, math.inf])
@pytest.mark.parametrize("nq,d", [(1, 64), (140, 64), (140, 128)])
def test_masks(dtype, fill, nq, d):
    """Holes, a whole tile without keys, one key only, none at all; with and without lengths."""
    gen = torch.Generator().manual_seed(5)
    nk = 270
    mask = torch.rand(6, nk, generator=gen) < 0.5
    mask[1, 128:256] = False
    mask[2] = False
    mask[3] = False
    mask[3, 269] = True
    mask[4, :140] = False
    run_case(dtype, 6, 2, 1, nq, nk, d, mask=mask.tolist(), fill=fill)
    run_case(dtype, 6, 2, 1, nq, nk, d, mask=mask.tolist(), lens=[270, 200, 270, 269, 130, 7], fill=fill)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("b,h,hk,nq,nk", [(2, 80, 80, 300, 130), (3, 64, 16, 129, 70), (2, 160, 4, 100, 300),
                                          (4, 50, 50, 257, 400)])
def test_many_heads(b, h, hk, nq, nk, d):
    """Enough tiles to fill the device several times over, with lengths that leave some of them nothing."""
    run_case(BF16, b, h, hk, nq, nk, d, layout="bnhd", lens=[nk, nk // 2, 0, 1][:b])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sharp,scale", [(20.0, None), (1.0, 3.0), (1.0, 1e-4)])
def test_sharp_and_flat_softmax(dtype, sharp, scale):
    """Logits far apart: the running maximum moves often; and almost equal."""
    run_case(dtype, 1, 2, 2, 130, 600, 64, sharp=sharp, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_growing_logits(dtype):
    """Each key beats the ones before it: the running maximum rises in every tile."""
    b, h, nq, nk, d = 1, 1, 130, 520, 64
    q = torch.ones(b, h, nq, d, dtype=dtype, device="cuda")
    k = (torch.arange(nk, device="cuda").float() / 16).view(1, 1, nk, 1).expand(b, h, nk, d).to(dtype).contiguous()
    gen = torch.Generator().manual_seed(2)
    v = util.tokens(gen, b, h, nk, d, dtype)
    for kk in (k, k.flip(2).contiguous()):
        p = llsa.CrossProblem(b, h, nq, nk, d, dtype=NUMBER[dtype])
        op = llsa.CrossAttention(p, backward=False)
        op.forward(q, kk, v)
        ref = util.cross_reference(q, kk, v, torch.ones(b, nk, dtype=torch.bool), p.scale)
        for name, (want, bound) in ref.items():
            util.check(name, getattr(op, name), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_broadcast_inputs(dtype):
    """One image's queries against every prompt, one prompt for every image: strides of zero in the inputs."""
    gen = torch.Generator().manual_seed(3)
    b, h, nq, nk, d = 3, 2, 90, 50, 64
    q1, k1, v1 = (util.tokens(gen, 1, h, n, d, dtype) for n in (nq, nk, nk))
    g1 = util.tokens(gen, 1, 1, nq, d, dtype)
    q, k, v = (t.expand(b, -1, -1, -1) for t in (q1, k1, v1))
    g = g1.expand(b, h, -1, -1)
    p = llsa.CrossProblem(b, h, nq, nk, d, dtype=NUMBER[dtype])
    op = llsa.CrossAttention(p)
    op.forward(q, k, v)
    op.backward_pass(q, k, v, g)
    ref = util.cross_reference(q, k, v, torch.ones(b, nk, dtype=torch.bool), p.scale, g)
    for name, (want, bound) in ref.items():
        util.check(name, getattr(op, name), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("nq", [5, 90])
def test_one_state_repeated_over_the_tokens(nq):
    """A token stride of zero, which the tensor-core kernels do not take: the other path, the same results."""
    gen = torch.Generator().manual_seed(10)
    b, h, nk, d = 2, 8, 150, 64
    q, g = (util.tokens(gen, b, h, nq, d, BF16) for _ in range(2))
    k = util.tokens(gen, b, h, nk, d, BF16)
    v = util.tokens(gen, b, h, 1, d, BF16).expand(b, h, nk, d)
    p = llsa.CrossProblem(b, h, nq, nk, d)
    op = llsa.CrossAttention(p)
    op.forward(q, k, v)
    op.backward_pass(q, k, v, g)
    for name, (want, bound) in util.cross_reference(q, k, v, torch.ones(b, nk, dtype=torch.bool), p.scale, g).items():
        util.check(name, getattr(op, name), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk", [(200, 70), (200, 300), (1, 300)])
def test_offsets_beyond_32_bits(nq, nk):
    """The second batch row of every tensor lies more than 2^31 elements behind the first."""
    gen = torch.Generator().manual_seed(11)
    b, h, d = 2, 2, 64
    far = (1 << 31) + 4096
    p = llsa.CrossProblem(b, h, nq, nk, d)
    big = torch.empty(far + 8 * h * (nq + nk) * d, dtype=BF16, device="cuda")
    at = 0

    def place(shape):
        nonlocal at
        t = big.as_strided(shape, (far, shape[2] * d, d, 1), at)
        at += h * shape[2] * d
        return t

    q, g, o, dq = (place(p.q_shape) for _ in range(4))
    k, v, dk, dv = (place(p.k_shape) for _ in range(4))
    for t in (q, g, k, v):
        t.copy_(torch.randn(t.shape, generator=gen).to(BF16))
    lse = torch.empty(p.q_shape[:3], device="cuda")
    sizes = llsa.cross_query_sizes(p)
    work = torch.empty(max(sizes["fwd_workspace_bytes"], sizes["bwd_workspace_bytes"]), dtype=torch.uint8, device="cuda")
    llsa.cross_attn_fwd(p, q, k, v, o, lse, workspace=work)
    llsa.cross_attn_bwd(p, q, k, v, o, g, lse, dq, dk, dv, workspace=work)
    got = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    for name, (want, bound) in util.cross_reference(q, k, v, torch.ones(b, nk, dtype=torch.bool), p.scale, g).items():
        util.check(name, got[name], want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_gradients_against_differences(dtype):
    """<dq, u> + <dk, s> + <dv, t> is the derivative of <O, dO> along (u, s, t), by central differences in 64 bits."""
    gen = torch.Generator().manual_seed(4)
    b, h, hk, nq, nk, d = 1, 2, 1, 40, 60, 64
    q, g = (util.tokens(gen, b, h, nq, d, dtype) for _ in range(2))
    k, v = (util.tokens(gen, b, hk, nk, d, dtype) for _ in range(2))
    p = llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk, dtype=NUMBER[dtype])
    op = llsa.CrossAttention(p)
    op.forward(q, k, v)
    dq, dk, dv = (t.cpu().double() for t in op.backward_pass(q, k, v, g))
    x = [t.cpu().double() for t in (q, k, v)]
    go = g.cpu().double()

    def value(q, k, v):
        k, v = k.repeat_interleave(h // hk, 1), v.repeat_interleave(h // hk, 1)
        return float(((torch.softmax((q @ k.mT) * p.scale, -1) @ v) * go).sum())

    bounds = util.cross_reference(q, k, v, torch.ones(b, nk, dtype=torch.bool), p.scale, g)
    for i, (got, name) in enumerate(((dq, "dq"), (dk, "dk"), (dv, "dv"))):
        u = torch.randn(got.shape, generator=gen, dtype=torch.float64)
        e = 1e-5
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + e * u, x[i] - e * u
        slope = (value(*up) - value(*down)) / (2 * e)
        # the elements' bounds along u; the difference quotient itself is good to about 1e-7 of it
        allowed = float((bounds[name][1] * u.abs()).sum()) + 1e-6 * (1 + abs(slope))
        assert abs(float((got * u).sum()) - slope) <= allowed, name


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("b,h,hk,nq,nk,d", [(2, 4, 2, 333, 517, 64), (2, 16, 16, 1100, 300, 72), (1, 4, 4, 5000, 77, 64),
                                            (2, 8, 2, 1, 2000, 128), (1, 2, 1, 900, 1, 128)])
def test_same_bits_every_time_and_beyond_the_outputs_nothing_changes(dtype, b, h, hk, nq, nk, d):
    gen = torch.Generator().manual_seed(6)
    q, g = (util.tokens(gen, b, h, nq, d, dtype) for _ in range(2))
    k, v = (util.tokens(gen, b, hk, nk, d, dtype) for _ in range(2))
    p = llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk, dtype=NUMBER[dtype])
    sizes = llsa.cross_query_sizes(p)
    got = []
    for fill in (0, 255):
        guard = 4096

        def guarded(nbytes):
            t = torch.full((nbytes + 2 * guard,), fill, dtype=torch.uint8, device="cuda")
            return t, t[guard:guard + nbytes]

        outs = {}
        es = q.element_size()
        for name, shape, dt in (("o", p.q_shape, dtype), ("lse", p.q_shape[:3], F32), ("dq", p.q_shape, dtype),
                                ("dk", p.k_shape, dtype), ("dv", p.k_shape, dtype)):
            n = math.prod(shape) * (4 if dt == F32 else es)
            whole, inner = guarded(n)
            outs[name] = (whole, inner.view(dt).view(shape), n)
        fw, fi = guarded(sizes["fwd_workspace_bytes"])
        bw, bi = guarded(sizes["bwd_workspace_bytes"])
        t = {name: x[1] for name, x in outs.items()}
        llsa.cross_attn_fwd(p, q, k, v, t["o"], t["lse"], workspace=fi if fi.numel() else None)
        llsa.cross_attn_bwd(p, q, k, v, t["o"], g, t["lse"], t["dq"], t["dk"], t["dv"], workspace=bi)
        torch.cuda.synchronize()
        for whole, n in [(x[0], x[2]) for x in outs.values()] + [(fw, sizes["fwd_workspace_bytes"]),
                                                                  (bw, sizes["bwd_workspace_bytes"])]:
            assert bool((whole[:guard] == fill).all()) and bool((whole[guard + n:] == fill).all())
        got.append({name: x.clone() for name, x in t.items()})
    for name in got[0]:
        assert torch.equal(got[0][name], got[1][name]), name


@pytest.mark.gpu
def test_rows_between_strided_outputs_stay():
    """Outputs that are slices of a wider buffer: what lies between their rows keeps its values."""
    gen = torch.Generator().manual_seed(7)
    b, h, n, nk, d = 2, 3, 75, 40, 72
    q, g = (util.tokens(gen, b, h, n, d, BF16, "bnhd") for _ in range(2))
    k, v = (util.tokens(gen, b, h, nk, d, BF16, "bnhd") for _ in range(2))
    p = llsa.CrossProblem(b, h, n, nk, d)
    big = {name: torch.full((b, m, 3, h, d), 7.0, dtype=BF16, device="cuda")
           for name, m in (("o", n), ("dq", n), ("dk", nk), ("dv", nk))}
    t = {name: x[:, :, 1].transpose(1, 2) for name, x in big.items()}
    lse = torch.empty(b, h, n, device="cuda")
    sizes = llsa.cross_query_sizes(p)
    work = torch.empty(max(sizes["fwd_workspace_bytes"], sizes["bwd_workspace_bytes"]), dtype=torch.uint8,
                       device="cuda")
    llsa.cross_attn_fwd(p, q, k, v, t["o"], lse, workspace=work)
    llsa.cross_attn_bwd(p, q, k, v, t["o"], g, lse, t["dq"], t["dk"], t["dv"], workspace=work)
    ref = util.cross_reference(q, k, v, torch.ones(b, nk, dtype=torch.bool), p.scale, g)
    for name in t:
        util.check(name, t[name], *ref[name])
        assert bool((big[name][:, :, 0] == 7).all()) and bool((big[name][:, :, 2] == 7).all()), name


@pytest.mark.gpu
@pytest.mark.parametrize("nq,nk", [(300, 200), (1, 3000)])
def test_streams_and_graphs(nq, nk):
    """On another stream, and captured: replays follow the inputs' new values and the lengths in device memory."""
    gen = torch.Generator().manual_seed(8)
    b, h, d = 2, 2, 64
    q, g = (util.tokens(gen, b, h, nq, d, BF16) for _ in range(2))
    k, v = (util.tokens(gen, b, h, nk, d, BF16) for _ in range(2))
    kv_len = torch.tensor([nk, nk // 2], dtype=torch.int32, device="cuda")
    p = llsa.CrossProblem(b, h, nq, nk, d)
    op = llsa.CrossAttention(p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.forward(q, k, v, kv_len=kv_len, stream=side)
    op.backward_pass(q, k, v, g, kv_len=kv_len, stream=side)
    side.synchronize()
    want = [t.clone() for t in (op.o, op.lse, op.dq, op.dk, op.dv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.forward(q, k, v, kv_len=kv_len)
        op.backward_pass(q, k, v, g, kv_len=kv_len)
    for t in (op.o, op.lse, op.dq, op.dk, op.dv):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for t, w in zip((op.o, op.lse, op.dq, op.dk, op.dv), want):
        assert torch.equal(t, w)
    kv_len.copy_(torch.tensor([3, 0], dtype=torch.int32))
    q.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    ref = util.cross_reference(q, k, v, util.valid_keys(b, nk, kv_len, None), p.scale, g)
    for name, (w, bound) in ref.items():
        util.check(name, getattr(op, name), w, bound)


@pytest.mark.gpu
def test_lse_is_optional():
    gen = torch.Generator().manual_seed(9)
    q, k, v = (util.tokens(gen, 1, 2, 50, 64, BF16) for _ in range(3))
    p = llsa.CrossProblem(1, 2, 50, 50, 64)
    a, b = torch.empty_like(q), torch.empty_like(q)
    need = llsa.cross_query_sizes(p)["fwd_workspace_bytes"]
    work = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    llsa.cross_attn_fwd(p, q, k, v, a, torch.empty(1, 2, 50, device="cuda"), workspace=work)
    llsa.cross_attn_fwd(p, q, k, v, b, workspace=work)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ refusals (no GPU)

def problem(**kw):
    base = dict(batch=2, heads=4, nq=100, nk=50, d=64, kv_heads=2)
    base.update(kw)
    return llsa.CrossProblem(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(d=8), 0), (dict(d=128, dtype=llsa.FP32), 0), (dict(kv_heads=4), 0), (dict(nq=1, nk=1), 0),
    (dict(scale=0.0), 0),
    (dict(batch=0), 1), (dict(heads=0), 1), (dict(kv_heads=3), 1), (dict(kv_heads=0), 1), (dict(kv_heads=8), 1),
    (dict(nq=0), 1), (dict(nk=0), 1), (dict(dtype=2), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(d=0, scale=1.0), 1), (dict(d=60), 7), (dict(d=136), 7),
    (dict(nq=1 << 24), 0), (dict(nk=1 << 24), 0), (dict(nq=(1 << 24) + 1), 2), (dict(nk=(1 << 24) + 1), 2),
    (dict(nq=1 << 24, heads=16, kv_heads=1), 2), (dict(nq=1 << 30, heads=1 << 20, kv_heads=1), 2), (dict(batch=1 << 13, heads=1 << 13), 2),
])
def test_validation(kw, status):
    assert llsa.cross_validate(problem(**kw)) == status


def test_workspaces_hold_what_either_path_keeps():
    """Whatever the strides, which decide between the paths: the row sums and every split's partial results."""
    for kw in (dict(batch=4, heads=16, kv_heads=16, nq=4096, nk=300, d=72), dict(batch=1, heads=6, kv_heads=6, nq=65536),
               dict(nq=1, nk=16384, d=128), dict(nq=64, nk=1000), dict(nq=4096, nk=4096)):
        a, b = (llsa.cross_query_sizes(problem(dtype=t, **kw)) for t in (llsa.BF16, llsa.FP32))
        assert a["fwd_workspace_bytes"] >= b["fwd_workspace_bytes"]
        assert a["bwd_workspace_bytes"] >= b["bwd_workspace_bytes"], kw
    s = llsa.cross_query_sizes(problem(batch=4, heads=16, kv_heads=16, nq=4096, nk=300, d=72))
    rows, keys = 4 * 16 * 4096, 4 * 16 * 300
    # 192 key tiles on 148 SMs: the queries are split, two partial gradients at least
    assert s["bwd_workspace_bytes"] >= rows * 4 + 2 * 2 * keys * 72 * 4


@pytest.mark.parametrize("name,strides,status", [
    ("q", (100 * 64 * 4, 6400, 64), 0),
    ("q", (0, 6400, 64), 0),                 # an input repeated over the batch
    ("o", (0, 6400, 64), 1),                 # a result written twice over
    ("dk", (64, 64, 64), 1),
    ("dq", (100 * 256, 64, 256), 0),         # heads inside the token
    ("dq", (100 * 256, 64, 192), 1),         # tokens that overlap
    ("v", (6400, 3200, 68), 3),              # not a multiple of 16 bytes
    ("k", (6400, -3200, 64), 1),
    ("k", (1 << 40, 3200, 64), 2),
])
def test_stride_rules(name, strides, status):
    c = problem().c()
    s = getattr(c, name)
    s.batch, s.head, s.token = strides
    assert llsa.lib().llsa_cross_validate(ctypes.byref(c)) == status


def test_entry_points_reject_bad_buffers_before_launch():
    L, good = llsa.lib(), 1 << 20            # never dereferenced
    c = problem().c()
    r = ctypes.byref(c)
    need = llsa.cross_query_sizes(problem())
    assert need["lse_bytes"] == 2 * 4 * 100 * 4 and need["bwd_workspace_bytes"] > 0

    def fwd(**kw):
        a = dict(q=good, k=good, v=good, n=None, m=None, o=good, lse=good, w=good)
        a.update(kw)
        return L.llsa_cross_attn_fwd(r, a["q"], a["k"], a["v"], a["n"], a["m"], a["o"], a["lse"], a["w"], None)

    for name in ("q", "k", "v", "o"):
        assert fwd(**{name: None}) == 1 and fwd(**{name: good + 8}) == 3, name
    assert fwd(lse=good + 4) == 3 and fwd(n=good + 2) == 3
    assert fwd(w=good + 8) in (3, 5) or need["fwd_workspace_bytes"] == 0

    def bwd(i, x):
        a = [good] * 13
        a[3] = a[4] = None
        a[i] = x
        return L.llsa_cross_attn_bwd(r, *a, None)

    for i in (0, 1, 2, 5, 6, 7, 8, 9, 10, 11):
        assert bwd(i, None) == 1 and bwd(i, good + 8) == 3, i
    assert bwd(3, good + 1) == 3
    assert L.llsa_cross_attn_fwd(None, *[good] * 8, None) == 1
    assert L.llsa_cross_query_sizes(r, None) == 1


def test_the_binding_checks_its_tensors():
    p = problem()
    q, k = torch.zeros(p.q_shape, dtype=BF16), torch.zeros(p.k_shape, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA"):
        llsa.cross_attn_fwd(p, q, k, k, q)
    with pytest.raises(ValueError, match="shape"):
        llsa.cross_attn_fwd(p, k, k, k, q)
    with pytest.raises(ValueError, match="float32"):
        llsa.cross_attn_fwd(p, q.float(), k, k, q)
    with pytest.raises(ValueError, match="contiguous"):
        llsa.cross_attn_fwd(p, q.transpose(-1, -2).contiguous().transpose(-1, -2), k, k, q)
    with pytest.raises(ValueError, match="expanded"):
        llsa.cross_attn_fwd(p, q[:1, :1, :1].expand(p.q_shape), k, k, q)
    with pytest.raises(ValueError, match="kv_len"):
        llsa.cross_attn_fwd(p, q, k, k, q, kv_len=torch.zeros(2))
    with pytest.raises(ValueError, match="key_mask"):
        llsa.cross_attn_fwd(p, q, k, k, q, key_mask=torch.zeros(2, 49, dtype=torch.bool))
    with pytest.raises(llsa.LLSAError):
        llsa.CrossAttention(problem(d=60), device="cpu")
