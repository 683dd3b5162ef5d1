"""ssu_gated_delta_rule where values leave fp32: what a prompt leaves is what single tokens
leave, infinity for infinity and NaN for NaN, in every form of its kernels."""
import pytest
import torch

from .gpu_util import require_gpu
from .test_gated_delta_gpu import Case

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def pair(lens, H, P, N, G, change, **kw):
    """Two cases with the same operands, which `change` has seen."""
    cases = [Case(lens, H, P, N, G, seed=6, **kw) for _ in range(2)]
    for c in cases:
        change(c)
    return cases


def prompts_and_steps(ssu, a, b):
    """a as prompts, b one token after the other (all sequences of one length)."""
    a.run(ssu)
    first, n = b.cu[:-1].long(), b.lens[0]
    assert set(b.lens) == {n}
    for t in range(n):
        at = first + t
        b.out[at] = ssu.gated_delta_rule_step(b.state, b.q[at], b.k[at], b.v[at], b.log_decay[at], None if b.beta is None else b.beta[at],
                                              b.idx, scale=b.scale, normalize=b.normalize)


def same(x, y, off, what):
    """NaN and infinities in the same places, and what is finite in both within `off`."""
    x, y = x.float(), y.float()
    for got, want, name in ((x.isnan(), y.isnan(), "NaN"), (x == INF, y == INF, "inf"), (x == -INF, y == -INF, "-inf")):
        assert torch.equal(got, want), f"{what}: {name} in {int((got != want).sum())} places of {want.numel()} (of {int(want.sum())})"
    ok = y.isfinite()
    assert ((x - y).abs()[ok] <= torch.as_tensor(off, device=y.device).expand(y.shape)[ok]).all(), what


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("P,N", [(64, 64), (48, 16), (32, 32), (64, 128), (32, 256)])
def test_the_recurrence_overflows(ssu, P, N, sparse, many):
    """One key of length 2 again and again, gain 1, no decay: the state grows threefold a token, and fp32 ends within a
    chunk. Rows of the state are powers of 2 times the key, so that all values are powers of about 3 times powers of 2 and
    nothing cancels: each token rounds them by 2^-24 a few times, less than 2^-10 of themselves in all, and none lies within
    1 % of fp32's end."""
    def change(c):
        k = torch.zeros(N, device="cuda") if sparse else torch.full((N,), 2 * N ** -0.5, device="cuda")
        if sparse:
            k[:16] = 0.5  # (zeros: 0 times an infinity is NaN)
        c.k.copy_(k.expand_as(c.k))
        c.q.copy_(c.k)
        c.v.zero_()
        c.state.copy_((2.0 ** -(torch.arange(P, device="cuda") % 4)[:, None] * k).expand_as(c.state))

    H = 2 if not many else 16
    a, b = pair([128] * (1 if not many else 40), H, P, N, 1, change, beta=False, rate=0.0, scale=1.0)
    prompts_and_steps(ssu, a, b)
    assert b.out[:64].isfinite().all() and b.out[70].isfinite().all() and not b.out[127].isfinite().any()
    same(a.out, b.out, 2.0 ** -6 * b.out.float().abs(), "out")
    same(a.state, b.state, 2.0 ** -10 * b.state.abs(), "state")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", [64, 128, 256])
def test_one_gain_overflows(ssu, N, many):
    """A gain times a value beyond fp32 in the middle of a chunk: the tokens before it do not see it."""
    def change(c):
        for b in c.cu[:-1].tolist():
            c.beta[b + 45, 1] = 1e30
            c.v[b + 45, 1, 3] = 1e20

    a, b = pair([70] * (30 if many else 1), 8 if many else 2, 64, N, 2, change)
    prompts_and_steps(ssu, a, b)
    assert b.out[:45].isfinite().all() and not b.out[45, 1, 3].isfinite()
    size = 1 + b.out.float().abs()
    size[45:, 1] = INF  # (the head's other channels take the same gain: their sizes are any)
    state = torch.full_like(b.state, INF)
    state[:, 0] = 2.0 ** -10 * (1 + b.state[:, 0].abs())
    same(a.out, b.out, 2.0 ** -6 * size, "out")
    same(a.state, b.state, state, "state")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", [16, 64, 128])
def test_the_state_leaves_fp32_and_comes_back(ssu, N, many):
    """Decays above 1 take the state beyond fp32 within a chunk, later ones would have taken it back: single tokens keep the
    infinity. Keys and gains of 0, so that nothing else happens."""
    def change(c):
        c.k.zero_()
        for b in c.cu[:-1].tolist():
            c.log_decay[b + 3:b + 13] = 9.0
            c.log_decay[b + 13:b + 23] = -9.0

    a, b = pair([40] * (40 if many else 1), 8 if many else 2, 64, N, 2, change, rate=0.0)
    prompts_and_steps(ssu, a, b)
    assert b.out[:12].isfinite().all() and not b.out[24:40].isfinite().any()
    same(a.out, b.out, 2.0 ** -6 * (1 + b.out.float().abs()), "out")
    same(a.state, b.state, 2.0 ** -10 * (1 + b.state.abs()), "state")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", [64, 128])
def test_a_large_state_decays_before_it_is_asked(ssu, N, many):
    """The state in front of a chunk times q is beyond fp32, the decayed one is not. Keys of 0; q of one value, so that
    nothing cancels: sums of N equal signs."""
    def change(c):
        c.k.zero_()
        c.q.fill_(100.0)
        c.state.abs_().add_(1.0).mul_(1e37)
        c.v.zero_()
        for b in c.cu[:-1].tolist():
            c.log_decay[b] = -30.0

    a, b = pair([40] * (40 if many else 1), 8 if many else 2, 64, N, 2, change)
    prompts_and_steps(ssu, a, b)
    assert b.out.isfinite().all()
    same(a.out, b.out, 2.0 ** -6 * b.out.float().abs(), "out")
    same(a.state, b.state, 2.0 ** -16 * b.state.abs(), "state")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", [16, 32, 64])
def test_infinities_of_one_sign(ssu, N, many):
    """A decay of infinity over a state, keys and queries of one sign, the gain negative: all that single tokens leave are
    infinities of one sign. With N = 16 half of a product's places are no state at all."""
    def change(c):
        c.state.abs_().add_(0.1)
        c.q.abs_().add_(0.1)
        c.k.abs_().add_(0.1)
        c.v.zero_()
        c.beta.mul_(-0.01)
        for b in c.cu[:-1].tolist():
            c.log_decay[b + 37] = INF

    a, b = pair([50] * (40 if many else 1), 8 if many else 2, 64, N, 2, change)
    prompts_and_steps(ssu, a, b)
    assert b.out[:37].isfinite().all() and (b.out[37:50] == INF).all() and (b.state[b.idx.long()] == INF).all()
    # (the chunk of the tokens 0 to 31 is finite; sums of one sign lose nothing)
    same(a.out, b.out, 2.0 ** -6 * b.out.float().abs(), "out")
    same(a.state, b.state, 2.0 ** -10 * b.state.abs(), "state")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("N", [32, 64, 128])
def test_keys_are_normalized_before_they_are_asked(ssu, N, many):
    """A state near fp32's end and long keys that are normalized: S k of the keys as given would be beyond fp32. A NaN in
    one query takes the chunk through the tokens."""
    def change(c):
        c.state.abs_().add_(1.0).mul_(1e36)
        c.k.abs_().add_(0.5).mul_(1000.0)
        c.v.zero_()
        for b in c.cu[:-1].tolist():
            c.q[b + 5, 0, 1] = NAN

    a, b = pair([20] * (40 if many else 1), 8 if many else 2, 64, N, 2, change, normalize=True)
    prompts_and_steps(ssu, a, b)
    assert b.state.isfinite().all() and b.out[:5].isfinite().all() and b.out[6:20].isfinite().all()
    assert b.out[5].isnan().any() and not b.out[5].isnan().all()
    # rows of the state are at most 10e36 sqrt(N) long and no longer behind a token; a token rounds sums of N such products
    # with a key and a query of length 1: 20 N 2^-24 at most
    size = 10e36 * N ** 0.5
    same(a.out, b.out, 2.0 ** -8 * b.out.float().abs() + 2.0 ** -12 * size, "out")
    same(a.state, b.state, 2.0 ** -12 * size, "state")
