"""The bounds of tests/seq_carried.py see a segment's decay that is rounded to bf16, off by 2^-9 or left out."""
import pytest
import torch

from . import seq_carried
from .test_linear_attention_carried_gpu import CASES


@pytest.mark.parametrize("case", range(len(CASES)))
def test_bounds_see_a_decay_of_16_bits(case):
    lens, H, P, N, G, rate, seg = CASES[case]
    if H * P * N > 1 << 14:  # (the heads' columns are alike: fewer of them, the same decays)
        P, N = 16, 16
    a = seq_carried.inputs(lens, H, P, N, G if H % G == 0 else 1, rate, case, "cpu")
    _, state, _, tol = seq_carried.exact(a)
    # (some heads' decays lie beside a number of 16 bits)
    for bend, enough in ((lambda x: x.to(torch.bfloat16).double(), 1), (lambda x: x * (1 - 2.0 ** -9), H), (torch.zeros_like, H)):
        _, bent, _, _ = seq_carried.exact(a, seg, bend)
        assert int(((bent - state).abs() > tol).flatten(2).any(-1).any(0).sum()) >= enough  # heads


def test_reference_is_the_recurrence():
    a = seq_carried.inputs([70, 3], 2, 4, 5, 1, 0.1, 1, "cpu")
    out, state, otol, tol = seq_carried.exact(a)
    from . import seq_ref
    want = seq_ref.linear_attention(*(seq_ref.f64(a[n]) for n in ("state", "q", "k", "v", "log_decay")), a["cu_seqlens"].numpy(),
                                    a["state_batch_indices"].numpy(), seq_ref.f64(a["beta"]), a["scale"])
    torch.testing.assert_close(out, torch.tensor(want["out"]), rtol=1e-12, atol=0)
    torch.testing.assert_close(state, torch.tensor(want["state"]), rtol=1e-12, atol=0)
    used = a["state_batch_indices"].long()
    assert (tol[used] > 0).all() and (tol[used] < 5e-4 * state[used]).all() and (otol > 0).all()
