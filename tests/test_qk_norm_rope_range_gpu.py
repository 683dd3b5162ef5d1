"""Rows whose squares add up beyond fp32 are 0, in the kernel of single rows and in that of groups; others are not touched."""
import pytest
import torch

from .gpu_util import require_gpu
from .test_qk_norm_rope_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,rot", [(5, 66, 66), (5, 128, 94), (600, 128, 94), (5, 128, 128), (5, 64, 0)])
def test_squares_beyond_fp32(T, D, rot):
    require_gpu()
    import selective_state_update_amd as ssu

    c = Case(T, 4, 1, D, rot, seed=1)
    want = c.run(ssu)[0].clone()
    c.q[3, 2] = 1e20
    got, _ = c.run(ssu)
    assert (got[3, 2] == 0).all()
    got[3, 2] = want[3, 2]
    assert torch.equal(got, want)
