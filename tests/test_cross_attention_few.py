"""Cross attention of few queries: every head dimension, the number of rows at which the kernels change, many batch rows."""
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def run(b, h, hk, nq, nk, d, layout="bhnd", lens=None, mask=None, seed=0):
    gen = torch.Generator().manual_seed(seed)
    q, g = (util.tokens(gen, b, h, nq, d, BF16, layout) for _ in range(2))
    k, v = (util.tokens(gen, b, hk, nk, d, BF16, layout, shift=s) for s in (0.25, 0.0))
    kv_len = None if lens is None else lens.to(torch.int32).cuda()
    key_mask = None if mask is None else mask.cuda()
    op = llsa.CrossAttention(llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk), token_major=layout != "bhnd")
    for t in (op.o, op.lse, op.dq, op.dk, op.dv):
        t.fill_(math.nan)
    op.work.fill_(255)
    op.forward(q, k, v, kv_len=kv_len, key_mask=key_mask)
    op.backward_pass(q, k, v, g, kv_len=kv_len, key_mask=key_mask)
    torch.cuda.synchronize()
    assert llsa.device_error() == 0
    ok = util.valid_keys(b, nk, kv_len, key_mask)
    for name, (want, bound) in util.cross_reference(q, k, v, ok, op.p.scale, g).items():
        util.check(name, getattr(op, name), want, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 88, 104, 120, 128])
@pytest.mark.parametrize("h,hk,nq", [(2, 2, 1), (6, 2, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_head_dimensions(d, h, hk, nq, masked):
    gen = torch.Generator().manual_seed(d)
    run(2, h, hk, nq, 219, d, "fused", lens=torch.tensor([219, 130]),
        mask=torch.rand(2, 219, generator=gen) < 0.6 if masked else None)


@pytest.mark.gpu
@pytest.mark.parametrize("h,hk,nq", [(1, 1, 15), (1, 1, 16), (1, 1, 17), (4, 1, 4), (16, 1, 1), (17, 1, 1), (16, 2, 2), (5, 1, 3),
                                     (3, 1, 5), (6, 1, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_a_key_head(h, hk, nq, d):
    """15, 16, 17 and 18 rows in all: up to 16 go to the kernel for few queries."""
    run(2, h, hk, nq, 333, d, lens=torch.tensor([333, 1]))


@pytest.mark.gpu
@pytest.mark.parametrize("b", [2048, 2049])
@pytest.mark.parametrize("h,hk", [(2, 2), (4, 1)])
def test_many_batch_rows(b, h, hk):
    """As many as the kernel for few queries keeps the lengths of, and one more; lengths from none to all."""
    gen = torch.Generator().manual_seed(b)
    run(b, h, hk, 1, 41, 64, lens=torch.randint(0, 42, (b,), generator=gen))


@pytest.mark.gpu
@pytest.mark.parametrize("nk", [1, 15, 16, 17, 63, 64, 65, 5000])
def test_all_rows_empty_but_one(nk):
    """Nearly nothing to deal out over the runs."""
    run(9, 4, 2, 2, nk, 64, lens=torch.tensor([0, 0, 0, 0, nk, 0, 0, 0, 0]))
    run(3, 2, 2, 1, nk, 72, lens=torch.tensor([0, 0, 0]))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [40, 72, 104])
@pytest.mark.parametrize("nk", [128, 256, 1024, 1100])
@pytest.mark.parametrize("nq", [40, 129])
def test_split_keys(d, nk, nq):
    """One head: the keys are split; lengths that end on a tile, behind its first key and leave splits nothing."""
    run(3, 2, 1, nq, nk, d, "bnhd", lens=torch.tensor([nk, 128, min(nk, 257)]))
