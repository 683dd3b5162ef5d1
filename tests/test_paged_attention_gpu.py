"""ssu_paged_attention against softmax attention in fp64 (tests/seq_ref.py)."""
import numpy as np
import pytest
import torch

from . import seq_ref
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


@pytest.fixture(params=[0, 1500], ids=["narrow", "wide"], autouse=True)
def width(request, monkeypatch):
    """Tables as wide as the requests need, and wider by that many tokens: short caches have a kernel of their own."""
    monkeypatch.setattr(Case, "wider", request.param)


class Case:
    """Scattered pages; every cache row that no request sees is NaN."""

    wider = 0

    def __init__(self, lens, nq, nk, D, page, dtype=BF16, seed=0, spare=1, gain=1.0, scale=None):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        self.q = (gain * torch.randn(B, nq, D, generator=g)).to(dtype).cuda()
        used = [-(-max(n, 0) // page) for n in lens]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((B, max(used + [0]) + spare + self.wider // page), -7, dtype=torch.int32)
        kc, vc = (torch.randn(pages, page, nk, D, generator=g).to(dtype) for _ in range(2))
        seen = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lens):
            for i in range(used[b]):
                p = order.pop()
                self.table[b, i] = p
                seen[p, :min(page, n - i * page)] = True
        kc[~seen], vc[~seen] = float("nan"), float("nan")
        self.kc, self.vc, self.table = kc.cuda(), vc.cuda(), self.table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.scale = D ** -0.5 if scale is None else scale
        self.dtype = dtype

    def ref(self):
        return seq_ref.paged_attention(seq_ref.f64(self.q), seq_ref.f64(self.kc), seq_ref.f64(self.vc), self.table.cpu().numpy(),
                                       self.lens.cpu().numpy(), self.scale, seq_ref.u_of(self.dtype))

    def run(self, ssu, **kw):
        return ssu.paged_attention(self.q, self.kc, self.vc, self.table, self.lens, scale=self.scale, return_lse=True, **kw)

    def check(self, ssu, **kw):
        want = self.ref()
        out, lse = self.run(ssu, **kw)
        seq_ref.assert_close(out, want["out"], want["out_tol"], "out")
        seq_ref.assert_close(lse, want["lse"], want["lse_tol"], "lse")
        return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 3, 16, 20, 64])
def test_shapes(ssu, dtype, D, page):
    Case([1, 0, 40, 133, 64], 8, 2, D, page, dtype, seed=D + page).check(ssu)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1000, 4097])
def test_lengths(ssu, n):
    Case([n], 4, 1, 128, 16, seed=n).check(ssu)


@pytest.mark.parametrize("nq,nk", [(1, 1), (4, 4), (5, 1), (7, 7), (14, 2), (16, 1), (17, 1), (32, 1), (80, 2), (24, 8)])
def test_heads(ssu, nq, nk):
    Case([100, 37], nq, nk, 64, 16, seed=nq + nk).check(ssu)


@pytest.mark.parametrize("batch", [1, 2, 40, 300])
def test_batches(ssu, batch):
    rng = np.random.default_rng(batch)
    Case([int(n) for n in rng.integers(0, 600, batch)], 4, 2, 64, 16, F16, seed=batch).check(ssu)


def test_long(ssu):
    Case([30011, 5, 9000], 8, 1, 128, 64, seed=3).check(ssu)


def test_sharp_and_flat(ssu):
    """One token far above the others, growing scores, equal scores, scale 0 and a negative scale."""
    Case([700], 4, 1, 128, 16, seed=4, gain=30.0).check(ssu)
    c = Case([900], 4, 1, 128, 16, seed=5)
    base = torch.randn(1, 1, 1, 128, device="cuda")
    pos = torch.zeros(c.kc.shape[0], 16, device="cuda")
    pos[c.table[0, :57].long()] = torch.arange(57 * 16, device="cuda").view(57, 16).float()
    c.kc = (pos[..., None, None] * 0.05 * base).to(BF16)  # scores grow or fall along the sequence
    c.check(ssu)
    Case([333], 4, 2, 64, 16, seed=6, scale=0.0).check(ssu)
    Case([333], 4, 2, 64, 16, seed=7, scale=-0.3).check(ssu)


def test_large_values(ssu):
    """Scores far outside exp's range: the running maximum carries them."""
    c = Case([200, 40], 4, 1, 128, 16, seed=8, gain=1.0, scale=50.0)
    c.check(ssu)


def test_padding_and_empty(ssu):
    c = Case([10, 0, 20, 5], 4, 2, 64, 16, seed=9)
    c.lens[2] = -1
    out = torch.full(c.q.shape, 7.0, dtype=BF16, device="cuda")
    out, lse = c.check(ssu, out=out)
    assert (out[2] == 7.0).all() and (out[1] == 0).all() and (lse[1] == -float("inf")).all()


def test_bad_pages(ssu):
    """Page ids outside the cache hold no visible token; lengths past the table end there."""
    c = Case([100, 50, 80], 4, 2, 64, 16, seed=10, spare=0)
    c.table[0, 2], c.table[0, 6], c.table[1, :] = -1, 1 << 30, c.kc.shape[0]
    c.lens[2] = 5000
    c.table[2, 5:] = -1
    out, _ = c.check(ssu)
    assert (out[1] == 0).all()


def test_infinite_scores(ssu):
    """Keys of -inf score weigh nothing; a row of them alone gives 0."""
    c = Case([40, 20], 2, 1, 64, 16, seed=11)
    c.q = c.q.abs() + 0.1
    first = c.table[0, 0].long()
    c.kc[first, 3] = -float("inf")
    for i in range(2):
        c.kc[c.table[1, i].long()] = -float("inf")
    out, lse = c.check(ssu)
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()


def test_nan_stays_in_its_request(ssu):
    c = Case([40, 50, 60], 4, 2, 64, 16, seed=12)
    want = c.ref()
    c.kc[c.table[1, 0].long(), 2, 1] = float("nan")
    out, _ = c.run(ssu)
    assert torch.isnan(out[1, 2:]).all()
    want["out"][1, 2:] = np.nan
    seq_ref.assert_close(out, want["out"], want["out_tol"], "others")


def test_layouts(ssu):
    """Strided queries, head-major caches with odd pitches, a table inside a larger one."""
    c = Case([100, 17, 64], 6, 2, 64, 16, seed=13)
    big = torch.full((c.kc.shape[0], 2, 16, 131), float("nan"), device="cuda", dtype=BF16)
    big[..., 1:65] = c.kc.transpose(1, 2)
    big[..., 67:131] = c.vc.transpose(1, 2)
    c.kc, c.vc = big[..., 1:65].transpose(1, 2), big[..., 67:131].transpose(1, 2)
    packed = torch.zeros(3, 6 * 64 + 7, device="cuda", dtype=BF16)
    packed[:, 3:3 + 384] = c.q.flatten(1)
    c.q = packed[:, 3:3 + 384].unflatten(1, (6, 64))
    wide = torch.full((3, 2 * c.table.shape[1]), -1, dtype=torch.int32, device="cuda")
    wide[:, 1:1 + c.table.shape[1]] = c.table
    c.table = wide[:, 1:1 + c.table.shape[1]]
    out = torch.zeros(3, 6, 65, device="cuda", dtype=BF16)[..., :64]
    c.check(ssu, out=out)


def test_far_pages(ssu):
    """Cache offsets past 2^31 elements."""
    page, D = 64, 128
    pages = (1 << 31) // (page * D) + 40
    kc = torch.empty(pages, page, 1, D, dtype=BF16, device="cuda")
    vc = torch.empty_like(kc)
    c = Case([150, 64], 4, 1, D, page, seed=14)
    small = c.kc.shape[0]
    kc[pages - small:], vc[pages - small:] = c.kc, c.vc
    want = c.ref()
    c.table = torch.where(c.table >= 0, c.table + (pages - small), c.table)
    c.kc, c.vc = kc, vc
    out, lse = c.run(ssu)
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")
    seq_ref.assert_close(lse, want["lse"], want["lse_tol"], "lse")


def test_repeats_bitwise(ssu):
    c = Case([5000, 300], 8, 2, 128, 16, seed=15)
    a, la = c.run(ssu)
    b, lb = c.run(ssu)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_graph_replays(ssu):
    """Two captured graphs and eager calls, each with a workspace of its own."""
    cases = [Case([3000, 100], 8, 2, 128, 16, seed=16), Case([2000, 700], 8, 2, 128, 16, seed=17)]
    want = [c.run(ssu)[0].clone() for c in cases]
    graphs, outs = [], []
    for c in cases:
        out = torch.zeros_like(c.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(ssu, out=out)
        graphs.append(g), outs.append(out)
    for _ in range(3):
        for i in (0, 1):
            outs[i].zero_()
            graphs[i].replay()
            cases[1 - i].run(ssu)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_short_graph_replays(ssu):
    """Lengths that change between replays of one graph, up to what the table holds."""
    c = Case([500, 400, 450], 8, 2, 128, 16, seed=25)
    out, lens = torch.zeros_like(c.q), c.lens.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(ssu, out=out)
    for n in (0, 1, 17, 256, 257, 400):
        c.lens.fill_(n)
        out.fill_(9.0)
        g.replay()
        assert torch.equal(out, c.run(ssu)[0])
    c.lens.copy_(lens)
    g.replay()
    want = c.ref()
    seq_ref.assert_close(out, want["out"], want["out_tol"], "out")


@pytest.mark.parametrize("D,tokens", [(64, 512), (128, 512), (256, 256)])
@pytest.mark.parametrize("page", [1, 16])
def test_short_limits(ssu, D, tokens, page):
    """On both sides of the longest cache that a workgroup takes alone, with few units and with many."""
    for n in (tokens - 1, tokens, tokens + 1):
        Case([n, 3, 0, n // 2 + 1], 6, 3, D, page, seed=n, spare=0).check(ssu)
    for batch, n in ((127, tokens + 1), (128, tokens + 1), (128, 2048), (128, 2049), (129, 1024), (129, 1025)):
        Case([n] + [1 + 37 * i % 40 for i in range(1, batch)], 2, 2, D, page, seed=batch, spare=0).check(ssu)


@pytest.mark.parametrize("lens,nk,D", [
    ([9000] * 3, 11, 128), ([9000] * 2, 16, 128), ([7000, 9000, 8000, 9500, 100], 8, 128),
    ([1000 + i % 7 for i in range(66)], 2, 256),  # a line per head, more requests than a wave has lanes
    ([2900], 100, 128)])                          # too many heads for that
def test_long_lines(ssu, lens, nk, D):
    """Lines that every second workgroup leaves and that all share, of all heads and of each."""
    Case(lens, nk, nk, D, 64, seed=nk).check(ssu)


def test_two_streams(ssu):
    cases = [Case([4000, 60], 8, 2, 128, 16, seed=18 + i) for i in range(2)]
    want = [c.ref() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [c.run(ssu, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for (out, lse), w in zip(got, want):
        seq_ref.assert_close(out, w["out"], w["out_tol"], "out")
        seq_ref.assert_close(lse, w["lse"], w["lse_tol"], "lse")


@pytest.mark.parametrize("batch", [3, 70])
def test_only_padding(ssu, batch):
    c = Case([20] * batch, 4, 2, 64, 16, seed=26)
    c.lens.fill_(-1)
    out = torch.full(c.q.shape, 7.0, dtype=BF16, device="cuda")
    c.run(ssu, out=out)
    assert (out == 7.0).all()
    c.lens[batch - 1] = 20  # one request behind all the padding
    c.check(ssu, out=out)
    assert (out[:batch - 1] == 7.0).all()


def test_no_requests(ssu):
    c = Case([], 4, 2, 64, 16, seed=20)
    assert c.run(ssu)[0].shape == (0, 4, 64)
    c = Case([0, 0], 4, 2, 64, 16, seed=21, spare=0)
    c.table = c.table[:, :0]
    out, _ = c.check(ssu)
    assert (out == 0).all()


def test_append_then_attend(ssu):
    """The layer as it is used, token after token: norm, rotation and append, then attention over the cache."""
    B, nq, nk, D, page, steps = 3, 4, 2, 64, 16, 20
    g = torch.Generator().manual_seed(22)
    kc, vc = (torch.full((B * 2, page, nk, D), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    blocks = torch.randperm(B * 2, generator=g).view(B, 2).to(torch.int32).cuda()
    angle = torch.arange(64)[:, None].double() * 1e4 ** (-torch.arange(0, D, 2) / D)
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float().cuda()
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(BF16).cuda()
    for t in range(steps):
        qkv = torch.randn(B, (nq + 2 * nk) * D, generator=g).to(BF16).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([nq * D, nk * D, nk * D], 1))
        pos = torch.full((B,), t, device="cuda")
        slots = blocks[:, t // page].long() * page + t % page
        qy, qt = seq_ref.norm_rope(seq_ref.f64(q), seq_ref.f64(w), [t] * B, seq_ref.f64(cos_sin), 1e-6, False, 2.0 ** -8)
        q_out, _ = ssu.qk_norm_rope(q, k, pos, cos_sin, w, w, v=v, k_cache=kc, v_cache=vc, slots=slots)
        seq_ref.assert_close(q_out, qy, qt, "q")
        lens = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        out = ssu.paged_attention(q_out, kc, vc, blocks, lens)
        want = seq_ref.paged_attention(seq_ref.f64(q_out), seq_ref.f64(kc), seq_ref.f64(vc), blocks.cpu().numpy(),
                                       lens.cpu().numpy(), D ** -0.5, 2.0 ** -8)
        seq_ref.assert_close(out, want["out"], want["out_tol"], f"token {t}")


def test_python_refusals(ssu):
    c = Case([20, 20], 4, 2, 64, 16, seed=23)
    with pytest.raises(TypeError):
        ssu.paged_attention(c.q, c.kc.half(), c.vc, c.table, c.lens)
    with pytest.raises(TypeError):
        ssu.paged_attention(c.q, c.kc, c.vc, c.table.long(), c.lens)
    with pytest.raises(ValueError):
        ssu.paged_attention(c.q, c.kc, c.vc[:-1], c.table, c.lens)
    with pytest.raises(ValueError):
        ssu.paged_attention(c.q, c.kc, c.vc, c.table, c.lens[:-1])
    with pytest.raises(ssu.SSUError):
        ssu.paged_attention(c.q[..., :48], c.kc[..., :48], c.vc[..., :48], c.table, c.lens)
    with pytest.raises(ssu.SSUError):
        ssu.paged_attention(c.q[:, :3], c.kc, c.vc, c.table, c.lens)
    with pytest.raises(ValueError):
        ssu.paged_attention(c.q.cpu(), c.kc, c.vc, c.table, c.lens)
