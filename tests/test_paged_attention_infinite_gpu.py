"""Infinite values in rows of V that a request sees: the formula gives an infinity, or NaN where infinities of both
signs meet or a value is NaN, in that column of that key/value head, and every other value as without it."""
import numpy as np
import pytest
import torch

from . import seq_ref
from .gpu_util import require_gpu
from .test_paged_attention_gpu import BF16, F16, Case

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


@pytest.fixture(params=[0, 1500], ids=["narrow", "wide"], autouse=True)
def width(request, monkeypatch):
    monkeypatch.setattr(Case, "wider", request.param)


def plant(c, b, j, kh, col, value):
    """V's value of token j of request b."""
    page = c.kc.shape[1]
    c.vc[int(c.table[b, j // page]), j % page, kh, col] = value


def check(ssu, c, planted):
    """planted: (request, token, key/value head, column, value). All weights are positive: no score is -inf."""
    want = c.ref()
    per = c.q.shape[1] // c.kc.shape[2]
    hit = np.zeros(want["out"].shape)
    for b, j, kh, col, value in planted:
        plant(c, b, j, kh, col, value)
        with np.errstate(invalid="ignore"):
            hit[b, kh * per:(kh + 1) * per, col] += value
    out, lse = c.run(ssu)
    got = seq_ref.f64(out)
    odd = ~np.isfinite(hit)
    assert np.array_equal(got[odd], hit[odd], equal_nan=True), f"expected {hit[odd]}, got {got[odd]}"
    rest = np.where(odd | (hit != 0), np.nan, want["out"])  # (a column's value replaced)
    assert np.isfinite(got[~np.isnan(rest)]).all()
    seq_ref.assert_close(out, rest, want["out_tol"], "out")
    seq_ref.assert_close(lse, want["lse"], want["lse_tol"], "lse")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [3, 16])
def test_infinite_v(ssu, dtype, D, page):
    """One request's only token (a weight of exactly 1), single infinities among many tokens, both signs in one column,
    and NaN beside them; the same column of the other head stays."""
    lens = [1, 40, 0, 133, 700]
    c = Case(lens, 8, 2, D, page, dtype, seed=D + page)
    check(ssu, c, [(0, 0, 0, 5, INF), (1, 39, 1, D - 1, -INF), (3, 7, 0, 0, INF), (3, 100, 0, 0, INF), (3, 132, 1, 3, INF),
                   (3, 1, 1, 3, -INF), (4, 0, 0, 17, -INF), (4, 699, 0, 17, float("nan")), (4, 650, 1, 40, INF)])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,many", [(64, 1), (128, 1), (256, 1), (128, 300)])
def test_infinite_v_of_small_weight(ssu, dtype, D, many):
    """Its weight is far below 16 bits' (and 32 bits') smallest number, in a step, a wave and a workgroup of its own."""
    c = Case([2500] + [1 + i % 5 for i in range(many - 1)], 4, 1, D, 16, dtype, seed=D, scale=1.0)
    c.q[0] = 0.0
    c.q[0, :, 0] = torch.tensor([2.0, 3.0, 4.0, 5.0], device="cuda")
    page = c.table[0, :157].long()
    c.kc[page, :, 0, 0] = 0.0
    at = 2000  # the row's largest score: 100 (weights of the others e^-80 to e^-200), at one token
    c.kc[page[at // 16], at % 16, 0, 0] = 40.0
    check(ssu, c, [(0, 10, 0, 3, INF), (0, 2499, 0, 9, -INF), (0, 2001, 0, 11, INF), (0, 500, 0, 20, INF), (0, 501, 0, 20, -INF)])


@pytest.mark.parametrize("nq,nk", [(1, 1), (17, 1), (24, 8)])
def test_infinite_v_by_heads(ssu, nq, nk):
    c = Case([300, 9000, 60], nq, nk, 128, 64, seed=nq)
    check(ssu, c, [(0, 299, nk - 1, 127, INF), (1, 4321, 0, 64, -INF), (1, 8999, 0, 1, INF)])


def test_infinite_v_behind_a_score_of_minus_infinity(ssu):
    """Such a token weighs 0, and 0 times an infinity is NaN; a bad page's tokens are not there at all."""
    c = Case([40, 100], 2, 1, 64, 16, seed=5)
    c.q = c.q.abs() + 0.1
    want = c.ref()
    c.kc[c.table[0, 0].long(), 3] = -INF
    plant(c, 0, 3, 0, 7, INF)
    plant(c, 1, 70, 0, 7, INF)
    c.table[1, 70 // 16] = -1
    out, _ = c.run(ssu)
    assert torch.isnan(out[0, :, 7]).all()
    out[0, :, 7] = 0.0
    assert torch.isfinite(out).all()
    c.vc[c.table[0, 0].long(), 3, 0, 7] = 0.0
    want = c.ref()
    want["out"][0, :, 7] = np.nan
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")


def test_infinite_v_repeats_in_a_graph(ssu):
    c = Case([3000, 100], 8, 2, 128, 16, seed=6)
    plant(c, 0, 1234, 1, 50, INF)
    want, lse = c.run(ssu)
    assert (want[0, 4:, 50] == INF).all()
    out = torch.zeros_like(c.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(ssu, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want) and torch.equal(c.run(ssu)[1], lse)
