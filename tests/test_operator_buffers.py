"""Buffers and sizes that the calls of cross attention and layer norm refuse before any launch (no GPU)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402

GOOD = 1 << 20          # an address that no call here may get as far as using


@pytest.mark.parametrize("kw,needed", [
    (dict(batch=2, heads=4, kv_heads=2, nq=100, nk=50), False),                       # one key split: no workspace
    (dict(batch=2, heads=4, kv_heads=2, nq=100, nk=50, dtype=llsa.FP32), False),
    (dict(batch=2, heads=4, kv_heads=2, nq=1, nk=50), True),                          # few queries
    (dict(batch=1, heads=1, kv_heads=1, nq=100, nk=4096), True),                      # split keys
    (dict(batch=1, heads=1, kv_heads=1, nq=100, nk=4096, dtype=llsa.FP32), True),
])
def test_cross_forward_refuses_a_workspace_it_cannot_use(kw, needed):
    """Misaligned: refused, needed or not; none where one is needed: refused.  Nothing is launched."""
    p = llsa.CrossProblem(**kw)
    need = llsa.cross_query_sizes(p)["fwd_workspace_bytes"]
    assert (need > 0) == needed
    L, r = llsa.lib(), ctypes.byref(p.c())
    before = llsa.kernel_launches()

    def forward(work):
        return L.llsa_cross_attn_fwd(r, GOOD, GOOD, GOOD, None, None, GOOD, GOOD, work, None)

    for off in (1, 4, 8):
        assert forward(GOOD + off) == 3
    if needed:
        assert forward(None) == 1
    assert llsa.kernel_launches() == before


def test_norm_backward_refuses_a_misaligned_workspace():
    """Also where only dx is asked for, which needs none."""
    p = llsa.NormProblem(batch=2, heads=3, n=10, c=64)
    L, r = llsa.lib(), ctypes.byref(p.cp())
    before = llsa.kernel_launches()
    for dw in (GOOD, None):
        assert L.llsa_layer_norm_bwd(r, GOOD, GOOD, GOOD, GOOD, GOOD, GOOD, dw, None, GOOD + 8, None) == 3
    assert llsa.kernel_launches() == before


@pytest.mark.parametrize("heads,nq,status", [
    (4, 1 << 24, 0), (5, 1 << 24, 2),
    (1 << 19, 128, 0), ((1 << 19) + 1, 128, 2),
    (1 << 18, 129, 0), ((1 << 18) + 1, 129, 2),       # two tiles a head, one of them nearly empty
    (1 << 19, 127, 0), (1 << 23, 8, 0),               # heads packed into tiles
])
def test_tiles_of_the_queries_that_share_a_key_head(heads, nq, status):
    """A block takes a key head's query tiles one after the other, and no wait of a good run may give up."""
    assert llsa.cross_validate(llsa.CrossProblem(batch=1, heads=heads, kv_heads=1, nq=nq, nk=200)) == status
