"""The operators together, as a conditional block runs them: layer norms of q and of the encoder's states, cross
attention, and the gradients back through all of it; and the self-attention with normed q and k."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402
import synthetic  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}


class Block:
    """q = norm(x) per head, k = norm(y) per head, o = attention(q, k, v); backward to x, y, v and the weights."""

    def __init__(self, dtype, b, h, hk, nq, nk, d, token_major=True):
        self.norm_q = llsa.LayerNorm(llsa.NormProblem(b, h, nq, d, dtype=NUMBER[dtype], param_dtype=llsa.FP32),
                                     token_major=token_major)
        self.norm_k = llsa.LayerNorm(llsa.NormProblem(b, hk, nk, d, dtype=NUMBER[dtype], param_dtype=llsa.FP32),
                                     token_major=token_major)
        self.cross = llsa.CrossAttention(llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk, dtype=NUMBER[dtype]),
                                         token_major=token_major)

    def step(self, x, y, v, w, g, kv_len, stream=None):
        q = self.norm_q.forward(x, w[0], w[1], stream)
        k = self.norm_k.forward(y, w[2], w[3], stream)
        self.cross.forward(q, k, v, kv_len=kv_len, stream=stream)
        dq, dk, dv = self.cross.backward_pass(q, k, v, g, kv_len=kv_len, stream=stream)
        self.norm_q.backward_pass(x, w[0], dq, stream)
        self.norm_k.backward_pass(y, w[2], dk, stream)
        return self.results()

    def results(self):
        n, m, c = self.norm_q, self.norm_k, self.cross
        return dict(q=n.y, k=m.y, o=c.o, lse=c.lse, dq=c.dq, dk=c.dk, dv=c.dv, dx=n.dx, dwq=n.dweight, dbq=n.dbias,
                    dy=m.dx, dwk=m.dweight, dbk=m.dbias)


def inputs(dtype, b, h, hk, nq, nk, d, seed):
    gen = torch.Generator().manual_seed(seed)
    x, g = (util.tokens(gen, b, h, nq, d, dtype, "bnhd", shift=0.3) for _ in range(2))
    y, v = (util.tokens(gen, b, hk, nk, d, dtype, "fused", shift=0.3) for _ in range(2))
    w = [(1 + 0.2 * torch.randn(d, generator=gen)).cuda() if i % 2 == 0 else (0.2 * torch.randn(d, generator=gen)).cuda()
         for i in range(4)]
    return x, y, v, w, g


def check_stages(r, x, y, v, w, g, kv_len, scale):
    """Each stage against the formulas in 64 bits, from the values that the stage before handed on."""
    dtype = x.dtype
    ok = util.valid_keys(x.shape[0], y.shape[2], kv_len, None)
    for name, (want, bound) in util.cross_reference(r["q"], r["k"], v, ok, scale, g).items():
        util.check(name, r[name], want, bound)
    for a, dy, (y_, dx, dw, db), i in ((x, "dq", ("q", "dx", "dwq", "dbq"), 0), (y, "dk", ("k", "dy", "dwk", "dbk"), 2)):
        ref = util.norm_reference(a, w[i], w[i + 1], 1e-6, dtype, F32, False, r[dy])
        for key, name in zip(("y", "dx", "dweight", "dbias"), (y_, dx, dw, db)):
            util.check(name, r[name], *ref[key])


SIZES = [(2, 4, 4, 300, 77, 64), (2, 4, 2, 130, 260, 72), (3, 8, 2, 1, 500, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", SIZES)
def test_block(dtype, size):
    b, h, hk, nq, nk, d = size
    x, y, v, w, g = inputs(dtype, *size, seed=1)
    kv_len = torch.tensor([nk, nk // 3, 0][:b], dtype=torch.int32, device="cuda")
    r = Block(dtype, *size).step(x, y, v, w, g, kv_len)
    check_stages(r, x, y, v, w, g, kv_len, 1 / math.sqrt(d))


@pytest.mark.gpu
def test_block_gradient_along_a_direction():
    """The whole chain's derivative, by central differences of the formula in 64 bits, against the fp32 block."""
    size = (1, 2, 1, 20, 30, 64)
    x, y, v, w, g = inputs(F32, *size, seed=2)
    kv_len = torch.tensor([23], dtype=torch.int32, device="cuda")
    r = Block(F32, *size).step(x, y, v, w, g, kv_len)
    at = [t.cpu().double() for t in (x, y, v, *w)]
    grads = [r[n].cpu().double() for n in ("dx", "dy", "dv", "dwq", "dbq", "dwk", "dbk")]
    go = g.cpu().double()

    def value(x, y, v, wq, bq, wk, bk):
        def norm(t, w, b):
            c = t - t.mean(-1, keepdim=True)
            return c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-6) * w + b
        q, k = norm(x, wq, bq), norm(y, wk, bk).repeat_interleave(2, 1)[:, :, :23]
        p = torch.softmax(q @ k.mT / 8, -1)
        return float(((p @ v.repeat_interleave(2, 1)[:, :, :23]) * go).sum())

    gen = torch.Generator().manual_seed(3)
    u = [torch.randn(t.shape, generator=gen, dtype=torch.float64) for t in at]
    e = 1e-5
    slope = (value(*[a + e * b for a, b in zip(at, u)]) - value(*[a - e * b for a, b in zip(at, u)])) / (2 * e)
    got = sum(float((a * b).sum()) for a, b in zip(grads, u))
    # fp32 roundings: each of some 1e4 terms is good to about 1e-5 of its size (sums of up to 64 and 30 products, the
    # softmax's and the norms' quotients), the difference quotient to about 1e-7
    size_of = sum(float((a * b).abs().sum()) for a, b in zip(grads, u))
    assert abs(got - slope) <= 1e-5 * size_of


@pytest.mark.gpu
def test_block_on_two_streams_and_in_graphs():
    """Two blocks at once on streams of their own give what one gives alone; captured, they replay new inputs."""
    size = SIZES[0]
    b, h, hk, nq, nk, d = size
    sets = [inputs(BF16, *size, seed=s) for s in (4, 5)]
    lens = [torch.tensor([nk, 5], dtype=torch.int32, device="cuda") for _ in range(2)]
    blocks = [Block(BF16, *size) for _ in range(2)]
    want = []
    for blk, s, n in zip(blocks, sets, lens):
        want.append({k: t.clone() for k, t in blk.step(*s, n).items()})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for blk, s, n, st in zip(blocks, sets, lens, streams):
            blk.step(*s, n, stream=st)
    torch.cuda.synchronize()
    for blk, w in zip(blocks, want):
        for k, t in blk.results().items():
            assert torch.equal(t, w[k]), k
    graphs = []
    for blk, s, n in zip(blocks, sets, lens):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            blk.step(*s, n)
        graphs.append(graph)
    for s, n in zip(sets, lens):
        s[0].mul_(1.5)
        n.copy_(torch.tensor([3, nk], dtype=torch.int32))
    for graph, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            graph.replay()
    torch.cuda.synchronize()
    assert llsa.device_error() == 0
    for blk, s, n in zip(blocks, sets, lens):
        check_stages(blk.results(), *s, n, 1 / math.sqrt(d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pipeline_with_normed_q_and_k(dtype):
    """The self-attention path with qk_norm: what norm, path and norm's gradient give one after the other."""
    p = llsa.Problem(batch=2, heads=2, height=64, width=64, d=64, B=16, L=3, K=8, dtype=NUMBER[dtype])
    arrays = synthetic.qkv(7, 2, 2, 64, 64, 64, 4.0, bf16=dtype == BF16)
    q, k, v = (torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype) for a in arrays)
    gen = torch.Generator().manual_seed(8)
    g = util.tokens(gen, 2, 2, 4096, 64, dtype)
    q, k = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))      # as a projection leaves them
    pipe = llsa.Pipeline(p, qk_norm=True)
    for name in ("q_weight", "k_weight", "q_bias", "k_bias"):
        getattr(pipe, name).add_(0.2 * torch.randn(64, generator=gen).cuda())
    pipe.step(q, k, v, g)
    plain = llsa.Pipeline(p)
    n = llsa.NormProblem(2, 2, 4096, 64, dtype=NUMBER[dtype], param_dtype=llsa.FP32)
    nq, nk = llsa.LayerNorm(n), llsa.LayerNorm(n)
    a, b = nq.forward(q, pipe.q_weight, pipe.q_bias), nk.forward(k, pipe.k_weight, pipe.k_bias)
    plain.step(a, b, v, g)
    torch.cuda.synchronize()
    assert torch.equal(pipe.o, plain.o) and torch.equal(pipe.lse, plain.lse)
    # the self-attention's backward adds pooled gradients by atomics (either type): two of its runs differ by
    # roundings, so the norm's gradients are checked from what one run handed on
    dq, dwq, dbq = nq.backward_pass(q, pipe.q_weight, plain.dq)
    ref = util.norm_reference(q, pipe.q_weight, pipe.q_bias, 1e-6, dtype, F32, False, plain.dq)
    for name, t in (("dx", dq), ("dweight", dwq), ("dbias", dbq)):
        util.check(name, t, *ref[name])
    for name, got, want in (("dq", pipe.dq, dq), ("dk", pipe.dk, nk.backward_pass(k, pipe.k_weight, plain.dk)[0]),
                            ("dv", pipe.dv, plain.dv)):
        off = (got.double() - want.double()).norm() / want.double().norm()
        assert off < 1e-2 if dtype == BF16 else off < 1e-4, name       # the path's own bounds (relative Frobenius)


def test_pipeline_rejects_before_allocating():
    with pytest.raises(llsa.LLSAError):
        llsa.Pipeline(llsa.Problem(batch=1, heads=1, height=60, width=64, d=64, B=16, L=3, K=8), device="cpu",
                      qk_norm=True)
