"""ssu_gated_delta_rule and ssu_gated_delta_rule_step against the recurrence in fp64
(tests/delta_ref.py), at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest
import torch

from . import delta_ref, seq_ref
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


class Case:
    """Seeded operands on the device: q, k, v as views into one packed tensor, keys
    of about length 1 unless they are normalized, random slots, ragged sequences."""

    def __init__(self, lens, H, P, N, G, seed=0, fixed=False, beta=True, pool=None, rate=1.0, scale=0.7, extra=0,
                 idx_dtype=torch.int32, gap=0, normalize=False):
        g = torch.Generator().manual_seed(seed)
        self.lens = lens
        self.T = T = sum(lens) + extra
        self.shape = (H, P, N, G)
        packed = torch.randn(T, H * P + 2 * G * N + gap, generator=g)
        if not normalize:
            packed[:, H * P:] *= N ** -0.5
        packed = packed.to(torch.bfloat16).cuda()
        self.packed = packed
        self.v = packed[:, :H * P].unflatten(1, (H, P))
        self.q = packed[:, H * P:H * P + G * N].unflatten(1, (G, N))
        self.k = packed[:, H * P + G * N:H * P + 2 * G * N].unflatten(1, (G, N))
        B = len(lens)
        pool = B + 2 if pool is None else pool
        self.state = torch.randn(pool, H, P, N, generator=g).cuda()
        self.idx = torch.randperm(pool, generator=g)[:B].to(idx_dtype).cuda()
        self.cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32).cuda()
        decay = -rate * (torch.rand(H, generator=g) if fixed else torch.rand(T, H, generator=g))
        self.log_decay = decay.float().cuda()
        self.beta = torch.rand(T, H, generator=g).cuda() if beta else None
        self.scale, self.normalize = scale, normalize
        self.out = torch.full((T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")

    def ref(self, state=None, chunk=delta_ref.CHUNK):
        f = seq_ref.f64
        return delta_ref.gated_delta(f(self.state if state is None else state), f(self.q), f(self.k), f(self.v), f(self.log_decay),
                                     self.cu.cpu().numpy(), self.idx.cpu().numpy(), None if self.beta is None else f(self.beta),
                                     self.scale, self.normalize, chunk)

    def run(self, ssu, **kw):
        kw = dict(out=self.out, **kw)
        return ssu.gated_delta_rule(self.state, self.q, self.k, self.v, self.log_decay, self.beta, self.cu, self.idx,
                                    scale=self.scale, normalize=self.normalize, **kw)

    def step(self, ssu, **kw):
        return ssu.gated_delta_rule_step(self.state, self.q, self.k, self.v, self.log_decay, self.beta, self.idx,
                                         scale=self.scale, normalize=self.normalize, out=self.out, **kw)

    def check(self, ssu, step=False, what=""):
        want, before = self.ref(chunk=1 if step else delta_ref.CHUNK), self.state.clone()
        out = self.step(ssu) if step else self.run(ssu)
        assert out is self.out
        seq_ref.assert_close(self.state, want["state"], want["state_tol"], what + " state")
        seq_ref.assert_close(out, want["out"], want["out_tol"], what + " out")
        # rows of no sequence, and slots of none, are as they were
        rest = np.isnan(want["out"])
        assert (seq_ref.f64(out)[rest] == 7.0).all(), what + ": rows of no sequence were written"
        live = [i for i, n in zip(self.idx.tolist(), self.lens) if n and 0 <= i < self.state.shape[0]]
        other = [i for i in range(self.state.shape[0]) if i not in live]
        assert torch.equal(self.state[other], before[other]), what + ": other slots were written"


@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("P", [16, 48, 64, 128, 256])
def test_prompt_shapes(ssu, N, P):
    Case([1, 70, 64, 0, 129], 4, P, N, 2, seed=N + P, normalize=P % 32 == 0).check(ssu)


@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("P", [16, 48, 80, 256])
def test_step_shapes(ssu, N, P):
    Case([1] * 7, 4, P, N, 2, seed=N + P, normalize=P % 32 == 0).check(ssu, step=True)


@pytest.mark.parametrize("N,P,H,B", [(16, 32, 8, 80), (32, 48, 8, 70), (64, 64, 8, 40), (128, 64, 8, 40), (128, 48, 16, 30), (256, 64, 8, 36)])
def test_many_sequences(ssu, N, P, H, B):
    """More columns of heads than the chip has SIMDs: the kernels of two column tiles a wave."""
    Case([(37 * i) % 68 for i in range(B)], H, P, N, 2, seed=B, normalize=True).check(ssu)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 96, 97])
def test_lengths(ssu, n):
    Case([n], 2, 32, 64, 1, seed=n).check(ssu)


@pytest.mark.parametrize("N", [64, 128, 256])
def test_long(ssu, N):
    Case([1500, 3], 2, 32, N, 1, seed=N, normalize=True, rate=0.05).check(ssu)


@pytest.mark.parametrize("kw", [dict(fixed=True), dict(beta=False), dict(idx_dtype=torch.int64), dict(gap=24), dict(gap=1), dict(gap=3),
                                dict(extra=9), dict(rate=0.0), dict(rate=0.0, normalize=True), dict(rate=30.0)])
@pytest.mark.parametrize("step", [False, True])
def test_options(ssu, kw, step):
    Case([1] * 6 if step else [40, 5, 0, 33], 4, 64, 128, 2, seed=3, **(kw if not (step and "extra" in kw) else {})).check(ssu, step=step)


@pytest.mark.parametrize("H,G", [(1, 1), (5, 5), (6, 3), (7, 1), (12, 4)])
def test_heads(ssu, H, G):
    Case([45, 70], H, 32, 64, G, seed=H).check(ssu)


def test_padding(ssu):
    for step in (False, True):
        c = Case([1] * 5 if step else [40, 7, 33, 1, 64], 3, 32, 64, 1, seed=5)
        c.idx[1], c.idx[3] = -1, c.state.shape[0]
        c.check(ssu, step=step)


def test_repeated_keys(ssu):
    """Every token the same key, gain 1, no decay: the triangle is all ones, its inverse has two diagonals."""
    c = Case([100], 2, 32, 64, 1, seed=1, rate=0.0, beta=False, normalize=True)
    c.k.copy_(c.k[:1].expand_as(c.k))
    c.check(ssu)


def test_orthogonal_keys_are_recalled(ssu):
    """Gain 1, no decay, unit keys along the axes: a key's value is what was written last, s + (v - s) with s what the
    key recalled before. s and u = v - s enter out as two bf16 pieces, off by 2^-18 each relative to themselves (half of
    2^-8 twice), and the state as three (2^-24) with a rounding each of the product, the difference, the piece and the sum:
    |s| + |u| <= 2 |s| + |v|. (Not v itself: 2^-18 |s| is more than half a step of a small v.)"""
    N = 64
    c = Case([2 * N], 1, 32, N, 1, seed=2, rate=0.0, beta=False, scale=1.0)
    c.k.copy_(torch.eye(N).repeat(2, 1)[:, None])
    c.q.copy_(c.k)
    slot = c.idx.long()[0]
    v = c.v[:, 0].double()
    size = 2 * torch.cat((c.state[slot, 0].T.double(), v[:N])).abs() + v.abs()
    c.run(ssu)
    assert ((c.out[:, 0].double() - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -17 * size).all()
    assert ((c.state[slot, 0].T.double() - v[N:]).abs() <= 8 * 2.0 ** -24 * size[N:]).all()


@pytest.mark.parametrize("step", [False, True])
def test_resets(ssu, step):
    c = Case([1, 1, 1] if step else [70, 33], 2, 32, 64, 1, seed=4)
    c.log_decay[::3] = -float("inf")
    c.log_decay[1::7] = -3e4
    c.check(ssu, step=step)


def test_growth(ssu):
    c = Case([70], 2, 32, 64, 1, seed=4, rate=-0.1)
    c.check(ssu)


def test_steps_continue_a_prompt(ssu):
    """A prompt, then single tokens, are the whole prompt."""
    whole = Case([75], 4, 64, 128, 2, seed=9, normalize=True)
    want = whole.ref()
    part = Case([75], 4, 64, 128, 2, seed=9, normalize=True)
    kw = dict(scale=part.scale, normalize=True)
    n = 70
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ssu.gated_delta_rule(part.state, part.q[:n], part.k[:n], part.v[:n], part.log_decay[:n], part.beta[:n], cu, part.idx,
                         out=part.out[:n], **kw)
    for t in range(n, 75):
        ssu.gated_delta_rule_step(part.state, part.q[t:t + 1], part.k[t:t + 1], part.v[t:t + 1], part.log_decay[t:t + 1],
                                  part.beta[t:t + 1], part.idx, out=part.out[t:t + 1], **kw)
    seq_ref.assert_close(part.state, want["state"], want["state_tol"], "state")
    seq_ref.assert_close(part.out, want["out"], want["out_tol"], "out")


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what", ["v", "k", "q", "beta", "log_decay", "state"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(ssu, what, value, many):
    """A prompt leaves what single tokens leave, wherever that is not finite, and stays within
    its bounds of them elsewhere."""
    if what == "log_decay" and value == -float("inf"):
        return  # (a reset)
    a, b = (Case([70] * (40 if many else 1), 8 if many else 2, 64, 64, 1, seed=6, normalize=True) for _ in range(2))
    for c in (a, b):
        t, s = c.T - 70 + 37, c.idx[-1]
        if what == "state":
            c.state[s, 1, 5, 3] = value
        else:
            x = getattr(c, what)
            x[(t, 0) if x.dim() == 2 else (t, 0, 5)] = value
    a.run(ssu)
    kw = dict(scale=b.scale, normalize=True)
    first = b.cu[:-1].long()
    for t in range(70):
        at = first + t
        b.out[at] = ssu.gated_delta_rule_step(b.state, b.q[at], b.k[at], b.v[at], b.log_decay[at], b.beta[at], b.idx, **kw)
    for x, y, u in ((a.state, b.state, 2.0 ** -14), (a.out.float(), b.out.float(), 2.0 ** -6)):
        assert torch.equal(x.isnan(), y.isnan()) and torch.equal(x.isinf(), y.isinf())
        assert torch.equal(x[x.isinf()], y[y.isinf()])
        ok = y.isfinite()
        assert ok.any() and not (what != "q" and ok.all())
        # (values of order 1: both sides are held to the fp64 recurrence elsewhere)
        assert ((x - y).abs()[ok] <= u * (1 + y.abs()[ok])).all()


def test_same_bits(ssu):
    a, b = (Case([500, 70, 3], 4, 64, 128, 2, seed=8, normalize=True) for _ in range(2))
    a.run(ssu)
    b.run(ssu, workspace=torch.empty(ssu.gated_delta_rule_workspace(3, 573, 4, 64, 128, 2), dtype=torch.uint8, device="cuda"))
    assert torch.equal(a.state, b.state) and torch.equal(a.out, b.out)


def test_streams_and_graphs(ssu):
    """On a stream of its own, and captured and replayed with eager calls between the replays."""
    a, b = (Case([100, 33], 4, 64, 128, 2, seed=8, normalize=True) for _ in range(2))
    first = a.state.clone()
    a.run(ssu)
    want_state, want = a.state.clone(), a.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.run(ssu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(b.state, want_state) and torch.equal(b.out, want)
    b.state.copy_(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(ssu)
    for i in range(4):
        b.state.copy_(first)
        b.out.fill_(7.0)
        graph.replay()
        a.state.copy_(first)
        a.run(ssu)
        torch.cuda.synchronize()
        assert torch.equal(b.state, want_state) and torch.equal(b.out, want) and torch.equal(a.state, want_state), i


def test_refusals(ssu):
    c = Case([40], 2, 32, 64, 1)
    call = lambda **kw: ssu.gated_delta_rule(**{**dict(  # noqa: E731
        state=c.state, q=c.q, k=c.k, v=c.v, log_decay=c.log_decay, beta=c.beta, cu_seqlens=c.cu, state_batch_indices=c.idx), **kw})
    call()
    for kw, error in ((dict(cu_seqlens=None), ValueError), (dict(q=c.q.float()), TypeError), (dict(k=c.k[:, :, :32]), ValueError),
                      (dict(beta=c.beta[:5]), ValueError), (dict(state=c.state.cpu()), ValueError), (dict(scale=float("nan")), ssu.SSUError),
                      (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), ssu.SSUError),
                      (dict(state_batch_indices=c.idx.float()), TypeError), (dict(normalize=None, beta=c.beta.half()), TypeError)):
        with pytest.raises(error):
            call(**kw)
    with torch.enable_grad(), pytest.raises(ValueError, match="inference only"):
        call(q=c.q.clone().requires_grad_())
    with pytest.raises(ValueError, match="tokens for"):
        ssu.gated_delta_rule_step(c.state, c.q, c.k, c.v, c.log_decay, c.beta, c.idx)
