"""The dense block's operators where a bound on the whole result hides an error.
Tolerances are derived as in test_gpu_dense.py."""
import pytest
import torch

import tile_level_collective_gb300 as P
from test_gpu_dense import check_clip
from test_gpu_layers import DT

pytestmark = pytest.mark.gpu


# ---- the gradients' norm -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("place", ["in", "out"])
def test_clip_norm_beyond_binary32(dtype, place):
    """A finite set whose norm binary32 cannot hold: the caller reads an infinite norm, and finds scale 1
    and its gradients as they were."""
    t = torch.full((2,), 3e38, dtype=DT[dtype], device="cuda")
    before, out, result = t.clone(), torch.zeros_like(t), torch.zeros(2, device="cuda")
    s = P.Gradients([t], None if place == "in" else [out])
    s.clip(1.0, result, workspace=s.workspace())
    assert result.tolist() == [float("inf"), 1.0]
    assert torch.equal(t, before) and (place == "in" or torch.equal(out, before))


def test_clip_largest_norm():
    """The largest norms that binary32 holds are finite, and limited."""
    check_clip([torch.full((2,), 2.4e38, device="cuda")], None, 1e30)
    check_clip([torch.full((3,), 1.9e38, device="cuda")], [torch.empty(3, device="cuda")], 1e30)
