"""Which kernels cross attention runs, by size, type and strides, and the CUDA-core kernels in bf16."""
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}
TENSOR, CUDA = {"fwd": "tensor", "bwd": "tensor"}, {"fwd": "cuda-core", "bwd": "cuda-core"}


@pytest.mark.parametrize("kw", [dict(), dict(nq=1), dict(nk=1), dict(nk=129), dict(d=8), dict(d=128, nk=4096), dict(kv_heads=1),
                                dict(nq=4, kv_heads=1), dict(batch=3000, nq=1), dict(nq=65536)])
def test_the_type_decides(kw):
    base = dict(batch=2, heads=4, nq=200, nk=100)
    base.update(kw)
    assert llsa.cross_attn_paths(llsa.CrossProblem(**base)) == TENSOR
    assert llsa.cross_attn_paths(llsa.CrossProblem(**base, dtype=llsa.FP32)) == CUDA


@pytest.mark.parametrize("nq", [5, 200])
def test_strides_decide(nq):
    """A token stride of zero goes to the CUDA cores, other strides do not; few queries run by plain loads of any stride."""
    p = llsa.CrossProblem(2, 4, nq, 100, 64)

    def made(shape, layout):
        b, h, n, d = shape
        if layout == "repeated":
            return torch.empty(b, h, 1, d, dtype=BF16).expand(shape)
        if layout == "bnhd":
            return torch.empty(b, n, h, d, dtype=BF16).transpose(1, 2)
        if layout == "one image":
            return torch.empty(1, h, n, d, dtype=BF16).expand(shape)
        return torch.empty(shape, dtype=BF16)

    shapes = dict(q=p.q_shape, k=p.k_shape, v=p.k_shape, dO=p.q_shape)
    for layout in ("plain", "bnhd", "one image"):
        assert llsa.cross_attn_paths(p, **{n: made(s, layout) for n, s in shapes.items()}) == TENSOR, layout
    few = nq == 5
    for name, shape in shapes.items():
        got = llsa.cross_attn_paths(p, **{name: made(shape, "repeated")})
        assert got["bwd"] == "cuda-core", name
        assert got["fwd"] == ("tensor" if few or name == "dO" else "cuda-core"), name
    with pytest.raises(ValueError, match="shape"):
        llsa.cross_attn_paths(p, q=made(p.k_shape, "plain"))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 72, 128])
@pytest.mark.parametrize("h,hk", [(3, 3), (4, 2)])
@pytest.mark.parametrize("repeated", ["q", "k", "v", "dO"])
@pytest.mark.parametrize("keys", ["all", "lengths", "mask", "both"])
@pytest.mark.parametrize("nk", [90, 200])
def test_cuda_core_kernels_in_bf16(d, h, hk, repeated, keys, nk):
    """One token repeated in an input: forward and backward on the CUDA cores, with what the other kernels take too."""
    gen = torch.Generator().manual_seed(d + nk)
    b, nq = 2, 90
    t = {}
    for name, heads, n in (("q", h, nq), ("k", hk, nk), ("v", hk, nk), ("dO", h, nq)):
        one = util.tokens(gen, b, heads, 1 if name == repeated else n, d, BF16, "bnhd")
        t[name] = one.expand(b, heads, n, d)
    p = llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk)
    assert llsa.cross_attn_paths(p, **t) == {"fwd": "tensor" if repeated == "dO" else "cuda-core", "bwd": "cuda-core"}
    kv_len = torch.tensor([nk, nk // 2], dtype=torch.int32, device="cuda") if keys in ("lengths", "both") else None
    key_mask = (torch.rand(b, nk, generator=gen) < 0.7).cuda() if keys in ("mask", "both") else None
    op = llsa.CrossAttention(p, token_major=True)
    for x in (op.o, op.lse, op.dq, op.dk, op.dv):
        x.fill_(math.nan)
    op.work.fill_(255)
    op.forward(t["q"], t["k"], t["v"], kv_len=kv_len, key_mask=key_mask)
    op.backward_pass(t["q"], t["k"], t["v"], t["dO"], kv_len=kv_len, key_mask=key_mask)
    torch.cuda.synchronize()
    assert llsa.device_error() == 0
    ok = util.valid_keys(b, nk, kv_len, key_mask)
    for name, (want, bound) in util.cross_reference(t["q"], t["k"], t["v"], ok, p.scale, t["dO"]).items():
        util.check(name, getattr(op, name), want, bound)
