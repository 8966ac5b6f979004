"""The self-attention path with qk_norm takes q and k of any strides; v and dO it reads by their addresses (no GPU)."""
import pytest

torch = pytest.importorskip("torch")

from hierarchical_top_sparse_b200 import llsa  # noqa: E402


def test_v_and_dO_are_checked_before_any_launch():
    p = llsa.Problem(batch=1, heads=2, height=16, width=16, d=64, B=4, L=2, K=4)
    pipe = llsa.Pipeline(p, device="cpu", qk_norm=True)
    good = torch.zeros(1, 2, 256, 64, dtype=torch.bfloat16)
    as_projected = torch.zeros(1, 256, 2, 64, dtype=torch.bfloat16).transpose(1, 2)
    before = llsa.kernel_launches()
    for bad in (as_projected, good.float(), good[:, :1], good[:, :, :255]):
        with pytest.raises(ValueError, match="^v: "):
            pipe.forward(good, good, bad, stream=0)
        with pytest.raises(ValueError, match="^v: "):
            pipe.backward_pass(good, good, bad, good, stream=0)
        with pytest.raises(ValueError, match="^dO: "):
            pipe.backward_pass(good, good, good, bad, stream=0)
    with pytest.raises(ValueError, match="CUDA"):       # q and k as projected are in order: what is refused is the device
        pipe.forward(as_projected, as_projected, good.view(2, 256, 64), stream=0)
    assert llsa.kernel_launches() == before
