"""What one segment of a long prompt hands to the next: states that last over all of it, in workgroups of four and of
eight waves, at every N, and in segments longer than the tokens that one round of decay sums covers."""
import pytest
import torch

from . import seq_carried
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu

# sequences' lengths, H, P, N, G, rate of decay, tokens of a segment (0: uncut)
CASES = [
    ([700], 3, 48, 16, 1, 2e-3, 128), ([700], 3, 48, 32, 3, 2e-3, 128), ([700], 3, 64, 64, 1, 2e-3, 128),
    ([700], 4, 48, 128, 2, 2e-3, 128), ([700, 650], 2, 32, 256, 1, 2e-3, 128), ([700], 2, 128, 128, 1, 2e-3, 128),
    ([900, 5], 3, 96, 128, 1, 1e-3, 128),
    ([800], 255, 16, 16, 1, 2e-3, 288),   # four waves: 256 tokens a round
    ([2112], 128, 80, 128, 1, 5e-4, 544),  # eight: 512
]
UNCUT = [([700] * 20, 16, 32, 64, 1, 2e-3, 0), ([1100, 30], 128, 128, 128, 1, 1e-3, 0)]


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


@pytest.mark.parametrize("case", range(len(CASES + UNCUT)))
def test_state_is_carried(ssu, case):
    lens, H, P, N, G, rate, seg = (CASES + UNCUT)[case]
    a = seq_carried.inputs(lens, H, P, N, G, rate, case, "cuda")
    need = ssu.linear_attention_workspace(len(lens), sum(lens), H, P, N, G)
    assert need == ((sum(lens) // seg + len(lens)) * H * (P * N + 1) * 4 if seg else 0), "not cut as the case says"
    out, state, otol, tol = seq_carried.exact(a)
    got = ssu.linear_attention(**a, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    off = (a["state"].double() - state).abs()
    assert (off <= tol).all(), f"state: {int((off > tol).sum())} of {off.numel()} off, worst {float((off / tol).nan_to_num().max()):.3g} of its bound"
    off = (got.double() - out).abs()
    assert (off <= otol).all(), f"out: {int((off > otol).sum())} of {off.numel()} off, worst {float((off / otol).max()):.3g} of its bound"
