"""ssu_linear_attention and ssu_linear_attention_step against the recurrence in
fp64 (tests/seq_ref.py), at the sizes, masks and layouts where they can go wrong."""
import numpy as np
import pytest
import torch

from . import seq_ref
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


class Case:
    """Seeded operands on the device: q, k, v as views into one packed tensor with
    rows of its own at both ends, random slots, ragged sequences."""

    def __init__(self, lens, H, P, N, G, seed=0, fixed=False, beta=True, pool=None, rate=1.0, scale=0.7, extra=0,
                 idx_dtype=torch.int32, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.lens = lens
        self.T = T = sum(lens) + extra
        self.shape = (H, P, N, G)
        packed = torch.randn(T, H * P + 2 * G * N + gap, generator=g).to(torch.bfloat16).cuda()
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
        self.scale = scale
        self.out = torch.full((T, H, P), 7.0, dtype=torch.bfloat16, device="cuda")

    def ref(self, state=None):
        c = seq_ref
        return c.linear_attention(c.f64(self.state if state is None else state), c.f64(self.q), c.f64(self.k), c.f64(self.v),
                                  c.f64(self.log_decay), self.cu.cpu().numpy(), self.idx.cpu().numpy(),
                                  None if self.beta is None else c.f64(self.beta), self.scale)

    def run(self, ssu, **kw):
        return ssu.linear_attention(self.state, self.q, self.k, self.v, self.log_decay, self.cu, self.idx, beta=self.beta,
                                    scale=self.scale, out=self.out, **kw)

    def check(self, ssu, step=False, what=""):
        want, before = self.ref(), self.state.clone()
        if step:
            out = ssu.linear_attention_step(self.state, self.q, self.k, self.v, self.log_decay, self.idx, beta=self.beta,
                                            scale=self.scale, out=self.out)
        else:
            out = self.run(ssu)
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
    Case([1, 70, 64, 0, 129], 4, P, N, 2, seed=N + P).check(ssu)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 192, 193, 511, 1000])
def test_prompt_lengths(ssu, length):
    Case([length], 3, 64, 128, 1, seed=length).check(ssu)


@pytest.mark.parametrize("H,G", [(1, 1), (2, 2), (5, 1), (6, 3), (8, 8), (16, 1)])
def test_prompt_heads(ssu, H, G):
    Case([77, 130], H, 32, 64, G, seed=H + G, fixed=True, beta=False).check(ssu)


def test_prompt_many_sequences(ssu):
    rng = np.random.default_rng(3)
    lens = [int(n) for n in rng.integers(0, 90, 200)]
    Case(lens, 2, 16, 32, 1, seed=5, idx_dtype=torch.int64, extra=9).check(ssu)


def test_prompt_long(ssu):
    """Long memory over many chunks: decays near one, and one long next to short ones."""
    Case([3000, 3, 700], 2, 32, 64, 1, seed=11, rate=1e-3).check(ssu)
    Case([5000], 1, 64, 128, 1, seed=12, rate=0.05, beta=False).check(ssu)


@pytest.mark.parametrize("lens,H,P,N", [
    ([700, 300] + [5] * 10, 32, 16, 32),       # whole sequences past the tokens that one round of decay sums covers
    ([600, 40, 1, 0, 3], 32, 128, 128),        # the same in workgroups of eight waves
    ([3 + 7 * i % 40 for i in range(130)], 6, 64, 128),  # more workgroups than three waves per SIMD hold
    ([1500], 2, 128, 128), ([1500, 100], 3, 96, 256), ([1200], 2, 48, 16)])  # cut into segments
def test_prompt_launch_shapes(ssu, lens, H, P, N):
    Case(lens, H, P, N, 1, seed=len(lens) + N).check(ssu)


def test_prompt_unaligned_views(ssu):
    """Odd row pitches and offsets: elements aligned to their size alone."""
    c = Case([50, 81], 3, 32, 64, 1, seed=21, gap=3)
    c.packed = torch.nn.functional.pad(c.packed, (1, 0))
    H, P, N, G = c.shape
    c.v = c.packed[:, 1:1 + H * P].unflatten(1, (H, P))
    c.q = c.packed[:, 1 + H * P:1 + H * P + G * N].unflatten(1, (G, N))
    c.k = c.packed[:, 1 + H * P + G * N:1 + H * P + 2 * G * N].unflatten(1, (G, N))
    assert c.packed.stride(0) % 2 == 1 or c.v.data_ptr() % 4
    c.check(ssu)


def test_prompt_strides(ssu):
    """Head-major tensors, a state inside a larger pool, gains of a strided view."""
    c = Case([40, 100], 4, 32, 64, 2, seed=22)
    H, P, N, G = c.shape
    c.q, c.k, c.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (c.q, c.k, c.v))
    c.state = torch.randn(4, 2, H, P, N, device="cuda")[:, 1]
    c.log_decay = c.log_decay.t().contiguous().t()
    c.beta = torch.rand(c.T, 2 * H, device="cuda")[:, ::2]
    c.out = torch.full((H, c.T, P), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    c.check(ssu)


def test_prompt_padding(ssu):
    c = Case([30, 0, 64, 5], 2, 16, 32, 1, seed=23, extra=3)
    c.idx = torch.tensor([2, -1, 99, 0], dtype=torch.int32, device="cuda")
    c.check(ssu)


def test_prompt_scattered_starts(ssu):
    """cu_seqlens need not start at 0; out-of-range bounds are taken inside [0, T)."""
    c = Case([20, 30], 2, 16, 32, 1, seed=24, extra=14)
    c.cu += 5
    c.check(ssu)
    c.out.fill_(7.0)
    c.cu = torch.tensor([-3, 20, 1 << 30], dtype=torch.int32, device="cuda")
    inside = c.cu
    c.cu = c.cu.clamp(0, c.T)
    want = c.ref()
    c.cu = inside
    c.run(ssu)
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")
    seq_ref.assert_close(c.out, want["out"], want["out_tol"], "out")


def test_prompt_unordered_sequences(ssu):
    """Sequences out of order may share a segment: their values are unspecified, all others are as they were."""
    c = Case([1200, 0, 0, 0], 2, 64, 64, 1, seed=25)
    c.cu = torch.tensor([512, 900, 0, 400, 300], dtype=torch.int32, device="cuda")  # 512 .. 899, none, 0 .. 399, none
    before = c.state.clone()
    for _ in range(3):
        c.run(ssu)
    torch.cuda.synchronize()
    rest = [i for i in range(before.shape[0]) if i not in (c.idx[0].item(), c.idx[2].item())]
    assert torch.equal(c.state[rest], before[rest])
    assert (c.out[400:512] == 7.0).all() and (c.out[900:] == 7.0).all()


@pytest.mark.parametrize("rate", [0.0, 20.0, 300.0])
def test_prompt_decays(ssu, rate):
    """No decay, and decays that leave nothing of the token before."""
    Case([150], 2, 32, 64, 1, seed=31, rate=rate).check(ssu)


def test_prompt_reset(ssu):
    """A log decay of -inf (and one below every exp) resets the state, and what
    follows keeps its digits."""
    c = Case([200], 2, 32, 64, 1, seed=32, rate=0.05)
    c.log_decay[70, 0] = -float("inf")
    c.log_decay[71, 1] = -3e38
    c.log_decay[130] = -1e5
    c.log_decay[10] = -1e3
    c.check(ssu)


def test_prompt_growth(ssu):
    c = Case([90], 2, 16, 32, 1, seed=33)
    c.log_decay = c.log_decay.abs() * 0.1
    c.check(ssu)


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_prompt_nonfinite_reach(ssu, what, value):
    """A value that is not finite reaches its own and later tokens (q: its own), and
    nothing before it or beside it."""
    c = Case([40, 150, 40], 2, 32, 64, 1, seed=41)
    at, H = 40 + 77, c.shape[0]
    want = c.ref()
    if what == "v":
        c.v[at, 1, 5] = value
    else:
        getattr(c, what)[at, 0, 9] = value
    out = c.run(ssu)
    hit = np.zeros(want["out"].shape, dtype=bool)
    if what == "v":
        hit[at:190, 1, 5] = True
    elif what == "k":
        hit[at:190] = True
    else:
        hit[at] = True
    got = seq_ref.f64(out)
    assert not np.isfinite(got[hit]).any(), "a value that is not finite got lost"
    want["out"][hit] = np.nan
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")
    state_hit = np.zeros(want["state"].shape, dtype=bool)
    slot = int(c.idx[1])
    if what == "v":
        state_hit[slot, 1, 5] = True
    elif what == "k":
        state_hit[slot, :, :, 9] = True
    got = seq_ref.f64(c.state)
    assert not np.isfinite(got[state_hit]).any()
    want["state"][state_hit] = np.nan
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")


def test_prompt_neighbours_do_not_leak(ssu):
    """NaN in the rows around a sequence (another request's, or of no request) does not reach it."""
    c = Case([33, 70, 20], 2, 32, 64, 1, seed=42, extra=40)
    c.packed[:33] = float("nan")
    c.packed[103:] = float("nan")
    c.idx[0] = c.idx[2] = -1
    c.check(ssu)


def test_prompt_pieces_match_whole(ssu):
    """A prompt in two calls, and as single steps, within the bounds of the whole."""
    c = Case([150], 2, 32, 64, 1, seed=51)
    want = c.ref()
    cut = 67
    for lo, hi in ((0, cut), (cut, 140)):
        c.cu = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        c.run(ssu)
    for t in range(140, 150):
        ssu.linear_attention_step(c.state, c.q[t:t + 1], c.k[t:t + 1], c.v[t:t + 1], c.log_decay[t:t + 1], c.idx,
                                  beta=c.beta[t:t + 1], scale=c.scale, out=c.out[t:t + 1])
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")
    seq_ref.assert_close(c.out, want["out"], want["out_tol"], "out")


def test_prompt_repeats_bitwise(ssu):
    c = Case([700, 30, 1], 4, 64, 128, 1, seed=52)
    first = c.state.clone()
    a, sa = c.run(ssu).clone(), c.state.clone()
    c.state.copy_(first)
    b = c.run(ssu)
    assert torch.equal(a, b) and torch.equal(sa, c.state)


def test_prompt_then_decode_step(ssu):
    """The prompt's state is the Mamba2 decode step's: a prefill, then ssu_update."""
    H, P, N, G, L = 4, 64, 128, 1, 100
    c = Case([L, L], H, P, N, G, seed=61, extra=2, scale=1.0)
    A = -torch.rand(H, device="cuda") * 4
    delta = torch.rand(c.T, H, device="cuda").to(torch.bfloat16).float()  # the step reads dt as bf16
    c.beta, c.log_decay = delta, A * delta
    c.cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    before = c.state.clone()
    c.run(ssu)
    last = slice(2 * L, 2 * L + 2)
    step = ssu.selective_state_update(c.state, c.v[last], delta[last].to(torch.bfloat16), A, c.k[last], c.q[last],
                                      dt_softplus=False, state_batch_indices=c.idx)
    # the same tokens, each request's last one appended to its prompt
    order = list(range(L)) + [2 * L] + list(range(L, 2 * L)) + [2 * L + 1]
    c.q, c.k, c.v, c.beta, c.log_decay = (x[order] for x in (c.q, c.k, c.v, c.beta, c.log_decay))
    c.cu = torch.tensor([0, L + 1, 2 * L + 2], dtype=torch.int32, device="cuda")
    want = c.ref(before)
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")
    seq_ref.assert_close(step, want["out"][[L, 2 * L + 1]], want["out_tol"][[L, 2 * L + 1]], "step's out")


@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("P,batch", [(16, 1), (48, 7), (64, 33), (80, 5), (128, 2), (256, 3)])
def test_step_shapes(ssu, N, P, batch):
    Case([1] * batch, 4, P, N, 2, seed=N + P, idx_dtype=torch.int64 if batch % 2 else torch.int32).check(ssu, step=True)


@pytest.mark.parametrize("batch", [24, 130, 512])
def test_step_batches(ssu, batch):
    """The sizes at which the launch changes."""
    Case([1] * batch, 16, 64, 128, 1, seed=batch, fixed=True, beta=False).check(ssu, step=True)


def test_step_padding_and_layout(ssu):
    c = Case([1] * 6, 3, 32, 64, 1, seed=71, gap=5)
    c.idx = torch.tensor([3, -1, 0, 1 << 30, 7, 5], dtype=torch.int32, device="cuda")
    c.state = torch.randn(8, 2, 3, 32, 64, device="cuda")[:, 1]
    c.lens = [1, 0, 1, 0, 1, 1]
    want = c.ref()
    c.check(ssu, step=True)
    assert np.isnan(want["out"][[1, 3]]).all()


def test_step_nonfinite(ssu):
    c = Case([1] * 3, 2, 16, 32, 1, seed=72)
    c.log_decay[0, 0] = -float("inf")
    want = c.ref()
    c.v[1, 1, 3] = float("nan")
    out = ssu.linear_attention_step(c.state, c.q, c.k, c.v, c.log_decay, c.idx, beta=c.beta, scale=c.scale, out=c.out)
    assert torch.isnan(out[1, 1, 3]) and torch.isnan(c.state[c.idx[1], 1, 3]).all()
    want["out"][1, 1, 3] = np.nan
    want["state"][int(c.idx[1]), 1, 3] = np.nan
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")


def test_graph_replays(ssu):
    """A captured prompt and step, replayed with eager work between, equal eager runs."""
    c = Case([600, 40], 4, 64, 128, 1, seed=81)
    s = Case([1] * 9, 4, 64, 128, 1, seed=82)

    def both():
        a = c.run(ssu)
        b = ssu.linear_attention_step(s.state, s.q, s.k, s.v, s.log_decay, s.idx, beta=s.beta, scale=s.scale, out=s.out)
        return a, b

    start = c.state.clone(), s.state.clone()
    both()
    want = []
    c.state.copy_(start[0]), s.state.copy_(start[1])
    for _ in range(3):
        a, b = both()
        want.append((a.clone(), b.clone(), c.state.clone(), s.state.clone()))
    c.state.copy_(start[0]), s.state.copy_(start[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    c.state.copy_(start[0]), s.state.copy_(start[1])
    for k in range(3):
        c.out.zero_(), s.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = (c.out, s.out, c.state, s.state)
        assert all(torch.equal(x, y) for x, y in zip(got, want[k])), f"replay {k}"
        Case([100], 4, 64, 128, 1, seed=83).run(ssu)  # eager work with a workspace of its own


def test_two_streams(ssu):
    """Two calls at once on streams of their own."""
    cases = [Case([900], 2, 64, 128, 1, seed=91 + i) for i in range(2)]
    want = [c.ref() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for c, st in zip(cases, streams):
        c.run(ssu, stream=st)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        seq_ref.assert_close(c.state, w["state"], w["state_tol"], "state")
        seq_ref.assert_close(c.out, w["out"], w["out_tol"], "out")


def test_given_workspace_and_new_out(ssu):
    c = Case([400], 2, 32, 64, 1, seed=95)
    want = c.ref()
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    out = ssu.linear_attention(c.state, c.q, c.k, c.v, c.log_decay, c.cu, c.idx, beta=c.beta, scale=c.scale, workspace=ws)
    seq_ref.assert_close(c.state, want["state"], want["state_tol"], "state")
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")


def test_empty(ssu):
    c = Case([0, 0], 2, 16, 32, 1, seed=96)
    before = c.state.clone()
    assert c.run(ssu).shape == (0, 2, 16) and torch.equal(c.state, before)
    z = Case([], 2, 16, 32, 1, seed=97)
    assert z.run(ssu).shape == (0, 2, 16)
    ssu.linear_attention_step(z.state, z.q, z.k, z.v, z.log_decay, z.idx, beta=z.beta, out=z.out)


def test_python_refusals(ssu):
    c = Case([4, 4], 2, 16, 32, 1, seed=98)

    def call(**kw):
        a = dict(state=c.state, q=c.q, k=c.k, v=c.v, log_decay=c.log_decay, cu_seqlens=c.cu, state_batch_indices=c.idx)
        a.update(kw)
        return ssu.linear_attention(**a)

    with pytest.raises(ValueError):
        call(k=c.k[:-1])
    with pytest.raises(ValueError):
        call(cu_seqlens=c.cu[:-1])
    with pytest.raises(TypeError):
        call(q=c.q.half())
    with pytest.raises(TypeError):
        call(cu_seqlens=c.cu.long())
    with pytest.raises(ValueError):
        call(v=c.v.cpu())
    with pytest.raises(ValueError):
        call(log_decay=c.log_decay.clone().requires_grad_())
    with pytest.raises(ssu.SSUError):
        call(scale=float("nan"))
    with pytest.raises(ssu.SSUError):
        call(out=torch.empty(1, 2, 16, dtype=torch.bfloat16, device="cuda").expand(8, 2, 16))
    with pytest.raises(ValueError):
        ssu.linear_attention_step(c.state, c.q, c.k, c.v, c.log_decay, c.idx)
