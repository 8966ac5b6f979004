"""Where nothing attends, nothing comes out: keys that are not valid have gradients of zero, and queries without a valid
key o = 0, lse = -inf and dq = 0, whatever the queries and the upstream gradient hold."""
import math

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402
import operators_util as util  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
NUMBER = {BF16: llsa.BF16, F32: llsa.FP32}
# equal heads and shared ones (their rows packed where few), one tile of keys and several, split queries and keys
SIZES = [(3, 2, 2, 150, 90, 64), (3, 2, 2, 150, 90, 72), (3, 4, 2, 150, 300, 64), (3, 4, 2, 70, 300, 128), (3, 8, 2, 1, 300, 64),
         (3, 1, 1, 130, 1100, 64), (3, 4, 1, 40, 100, 128)]


def run(dtype, size, kv_len, key_mask, spoil, repeated=False):
    """One forward and backward; spoil(q, dO) changes the queries and the upstream gradient first.  repeated: one value
    row for all keys by a token stride of zero, which in bf16 too goes to the CUDA-core kernels."""
    b, h, hk, nq, nk, d = size
    gen = torch.Generator().manual_seed(nk + d)
    q, g = (util.tokens(gen, b, h, nq, d, dtype) for _ in range(2))
    k = util.tokens(gen, b, hk, nk, d, dtype)
    v = util.tokens(gen, b, hk, 1, d, dtype).expand(b, hk, nk, d) if repeated else util.tokens(gen, b, hk, nk, d, dtype)
    spoil(q, g)
    op = llsa.CrossAttention(llsa.CrossProblem(b, h, nq, nk, d, kv_heads=hk, dtype=NUMBER[dtype]))
    for t in (op.o, op.lse, op.dq, op.dk, op.dv):
        t.fill_(math.nan)
    if op.work is not None:
        op.work.fill_(255)
    op.forward(q, k, v, kv_len=kv_len, key_mask=key_mask)
    op.backward_pass(q, k, v, g, kv_len=kv_len, key_mask=key_mask)
    torch.cuda.synchronize()
    assert llsa.device_error() == 0
    return op


def keys_of(b, nk, how):
    """kv_len, key_mask: the first batch row has all but some keys, the others none, by length or by mask."""
    gen = torch.Generator().manual_seed(9)
    if how == "length":
        return torch.tensor([nk - nk // 3] + [0] * (b - 1), dtype=torch.int32, device="cuda"), None
    mask = torch.zeros(b, nk, dtype=torch.bool)
    mask[0] = torch.rand(nk, generator=gen) < 0.6
    mask[0, 0] = True
    return None, mask.cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,repeated", [(BF16, False), (BF16, True), (F32, False)])
@pytest.mark.parametrize("how", ["length", "mask"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("size", SIZES)
def test_keys_that_are_not_valid(dtype, repeated, how, value, size):
    """One query of the batch row with keys has a gradient, and another has channels, that are not finite."""
    b, h, hk, nq, nk, d = size

    def spoil(q, g):
        g[0, 0, 0] = value
        q[0, h - 1, nq - 1, 3] = value

    kv_len, key_mask = keys_of(b, nk, how)
    op = run(dtype, size, kv_len, key_mask, spoil, repeated)
    bad = ~util.valid_keys(b, nk, kv_len, key_mask).cuda()
    for t in (op.dk, op.dv):
        assert bool((t.masked_select(bad[:, None, :, None]) == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,repeated", [(BF16, False), (BF16, True), (F32, False)])
@pytest.mark.parametrize("how", ["length", "mask"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("size", SIZES)
def test_queries_without_a_key(dtype, repeated, how, value, size):
    """Batch rows without a valid key, their queries and upstream gradients not finite; the row with keys as the formulas."""
    b, h, hk, nq, nk, d = size

    def spoil(q, g):
        q[1:, :, ::2] = value
        g[1:, :, ::3] = value

    kv_len, key_mask = keys_of(b, nk, how)
    op = run(dtype, size, kv_len, key_mask, spoil, repeated)
    clean = run(dtype, size, kv_len, key_mask, lambda q, g: None, repeated)
    assert bool((op.o[1:] == 0).all()) and bool((op.lse[1:] == -math.inf).all())
    for t in (op.dq, op.dk, op.dv):
        assert bool((t[1:] == 0).all())
    for name in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(getattr(op, name), getattr(clean, name)), name
