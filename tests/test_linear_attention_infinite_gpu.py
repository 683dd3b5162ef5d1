"""Infinite values in prompts: they go through the recurrence as they do token by token, so that a prompt leaves the
state and the outputs that single steps leave, infinities where the formula gives infinities and NaN where it gives NaN."""
import numpy as np
import pytest
import torch

from . import seq_ref
from .gpu_util import require_gpu
from .test_linear_attention_gpu import Case

pytestmark = pytest.mark.gpu
INF = float("inf")

# sequences' lengths, H, P, N, G: uncut in workgroups of four and eight waves, and cut into segments of 128 tokens
LAUNCHES = [([40, 150, 40], 2, 32, 64, 1), ([40, 150, 40], 2, 16, 16, 1), ([40, 150, 40], 2, 80, 128, 2),
            ([40, 150, 40], 2, 48, 256, 1), ([1500], 2, 128, 128, 1), ([1500], 2, 48, 16, 1), ([1500], 2, 32, 128, 2),
            ([1500], 2, 32, 256, 1)]


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def check(ssu, c, steps=True):
    """Against the recurrence in 64 bits, and which values are infinite or NaN against single steps too."""
    with np.errstate(all="ignore"):
        want = c.ref()
    before = c.state.clone()
    out = c.run(ssu)
    rows = np.zeros(c.T, dtype=bool)
    cu = c.cu.tolist()
    for b, i in enumerate(c.idx.tolist()):
        rows[cu[b]:cu[b + 1]] = 0 <= i < before.shape[0]
    for got, exact, tol, what in ((out, want["out"], want["out_tol"], "out"), (c.state, want["state"], want["state_tol"], "state")):
        got = seq_ref.f64(got)
        seen = np.ones(exact.shape, dtype=bool)
        if what == "out":
            seen[~rows] = False
        same = np.where(np.isfinite(exact), np.isfinite(got), np.where(np.isnan(exact), np.isnan(got), got == exact))
        bad = np.argwhere(seen & ~same)
        assert not len(bad), f"{what}: {len(bad)} values, first at {bad[0]}: {got[tuple(bad[0])]}, expected {exact[tuple(bad[0])]}"
        # (the bounds of rows with an infinity in them are infinite or NaN: nothing is left to compare there)
        seq_ref.assert_close(got, np.where(np.isfinite(exact) & np.isfinite(tol), exact, np.nan), np.nan_to_num(tol), what)
    if not steps:
        return
    after, ends = c.state.clone(), out.clone()
    c.state.copy_(before)
    stepped = torch.full_like(out, 7.0)
    for b in range(len(c.lens)):
        for t in range(cu[b], cu[b + 1]):
            g = c.log_decay[t:t + 1] if c.log_decay.dim() == 2 else c.log_decay
            ssu.linear_attention_step(c.state, c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], g, c.idx[b:b + 1],
                                      beta=None if c.beta is None else c.beta[t:t + 1], scale=c.scale, out=stepped[t:t + 1])
    for x, y, what in ((ends, stepped, "out"), (after, c.state, "state")):
        x, y = x.float(), y.float()
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.isinf(), y.isinf()), what
        assert torch.equal(x[x.isinf()], y[y.isinf()]), what


@pytest.mark.parametrize("what", ["v", "k", "q", "beta", "state", "v both signs", "k and v", "two chunks"])
@pytest.mark.parametrize("launch", range(len(LAUNCHES)))
def test_infinity(ssu, what, launch):
    c = Case(*LAUNCHES[launch], seed=launch, rate=0.5)
    H, P, N, G = c.shape
    at = (40 + 77) if len(c.lens) > 1 else 700
    if what == "v":
        c.v[at, 1, 5] = INF
    elif what == "k":
        c.k[at, 0, 9] = -INF
    elif what == "q":
        c.q[at, 0, 9] = INF
    elif what == "beta":
        c.beta[at, 1] = INF
    elif what == "state":
        c.state[c.idx[len(c.lens) // 2].long(), 1, 3, 2] = -INF
    elif what == "v both signs":
        c.v[at, 1, 5], c.v[at + 1, 1, 5] = INF, -INF
        c.k[at + 1, 0] = c.k[at, 0]  # -inf joins +inf in the state
    elif what == "k and v":
        c.k[at, 0, 9], c.v[at, 1, 5], c.v[at, 0, 2] = INF, -INF, 0.0
    else:
        c.v[at, 1, 5], c.v[at + 33, 0, 7], c.q[at + 2, 0, 1] = INF, -INF, -INF
    check(ssu, c, steps=launch in (0, 2, 4))


@pytest.mark.parametrize("launch", range(len(LAUNCHES)))
def test_infinity_in_the_first_and_last_token(ssu, launch):
    c = Case(*LAUNCHES[launch], seed=50 + launch, rate=0.5)
    lo, hi = (40, 190) if len(c.lens) > 1 else (0, 1500)
    c.v[lo, 0, 3], c.k[hi - 1, 0, 8] = INF, INF
    check(ssu, c, steps=False)


@pytest.mark.parametrize("launch", [0, 2, 4, 6])
def test_infinite_state_outlasts_decays(ssu, launch):
    """Every token's decay is positive, their product is not in 32 bits: an infinity stays one. A decay of 0 makes it NaN."""
    c = Case(*LAUNCHES[launch], seed=70 + launch, rate=1.0)
    c.log_decay -= 4.0
    b = len(c.lens) // 2
    c.state[c.idx[b].long(), :, 2, 1] = INF
    at = (40 + 50) if len(c.lens) > 1 else 300
    c.v[at, 0, 6] = -INF
    c.log_decay[at + 20, 1] = -INF
    check(ssu, c, steps=launch == 0)


@pytest.mark.parametrize("launch", [0, 2, 4, 5])
def test_growth_beyond_a_chunk(ssu, launch):
    """Growth that no sum of a chunk or a segment holds in 32 bits, from a state of zeros, with tokens that add nothing,
    and from a state of tiny values: nothing overflows in the recurrence."""
    c = Case(*LAUNCHES[launch], seed=90 + launch, rate=0.01)
    lo, hi = (40, 190) if len(c.lens) > 1 else (0, 1500)
    grow = 64 if len(c.lens) > 1 else 256
    c.log_decay = c.log_decay.clone()
    c.log_decay[lo:lo + grow] = 4.0 if len(c.lens) > 1 else 0.7
    c.v[lo:lo + grow] = 0.0
    c.state[:, 0] = 0.0
    c.state[:, 1] *= 1e-35
    c.log_decay[lo:lo + grow, 1] = 100.0 / grow
    check(ssu, c, steps=False)
