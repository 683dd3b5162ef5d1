"""Values that are not finite in prompts of ssu_gated_delta_rule, in every form of its kernels: with the N of a column
in one, two and four waves, in a tile that is half empty, and with waves that have no column."""
import pytest
import torch

from .test_gated_delta_gpu import Case, ssu  # noqa: F401
from .test_gated_delta_range_gpu import INF, NAN, pair, prompts_and_steps, same

pytestmark = pytest.mark.gpu
VALUES = [("v", INF), ("k", NAN), ("k", -INF), ("q", INF), ("beta", INF), ("log_decay", NAN), ("state", -INF)]


@pytest.mark.parametrize("what,value", VALUES)
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("P,N", [(48, 16), (80, 32), (48, 128), (16, 256)])
def test_not_finite(ssu, P, N, many, normalize, what, value):  # noqa: F811
    """As single tokens leave it. Where finite: values are of order 1, keys of about length 1, and a row of the state of
    about sqrt(N); a token rounds sums of N products with it by (48 + N / 8) 2^-24 sqrt(N), at most 2^-14, and 70 tokens
    whose gains shrink what was off before add up to less than 2^-8 of 1 + |y|; pieces and rounding of out take 2^-7."""
    def change(c):
        t, s = c.T - 70 + 37, c.idx[-1]
        if what == "state":
            c.state[s, 1, 5, 3] = value
        else:
            x = getattr(c, what)
            x[(t, 0) if x.dim() == 2 else (t, 0, 5)] = value

    H = 8 if many else 2
    batch = (64 * 16 // (H * (P // 16)) if many else 1) + 1
    a, b = pair([70] * batch, H, P, N, 2, change, normalize=normalize)
    prompts_and_steps(ssu, a, b)
    ok = b.out.isfinite()
    assert ok.any() and (what == "q" or not ok.all())
    same(a.out, b.out, (2.0 ** -8 + 2.0 ** -7) * (1 + b.out.float().abs()), "out")
    same(a.state, b.state, 2.0 ** -8 * (1 + b.state.abs()), "state")


@pytest.mark.parametrize("N", [64, 128, 256])
def test_every_chunk_by_tokens_and_as_products_in_turn(ssu, N):  # noqa: F811
    """NaN in queries of every second chunk only: the way of a chunk is its own, the state passes through both, and a
    sequence's end inside a chunk that goes by tokens ends it."""
    def change(c):
        for t in list(range(0, 300, 64)) + [299]:
            c.q[t, 0, 7] = NAN

    a, b = pair([300], 2, 64, N, 2, change, normalize=True)
    prompts_and_steps(ssu, a, b)
    assert b.state.isfinite().all()
    same(a.out, b.out, (2.0 ** -8 + 2.0 ** -7) * (1 + b.out.float().abs()), "out")
    same(a.state, b.state, 2.0 ** -8 * (1 + b.state.abs()), "state")
