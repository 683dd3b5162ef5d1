"""ssu_shared_prefix_attention against fp64 (tests/shared_ref.py), at the lengths, pages
and layouts where it can go wrong."""
import numpy as np
import pytest
import torch

from . import seq_ref, shared_ref
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


class Case:
    """Seeded operands on the device; page ids all different, tables wider than what is used."""

    def __init__(self, lens, n0, Hq=8, Hk=2, D=64, page=16, dtype=BF16, seed=0, scale=None, spare=1, gap=0):
        g = torch.Generator().manual_seed(seed)
        self.lens_, B = lens, len(lens)
        first, width = max(-(-n0 // page), 0) + spare, max([-(-max(n, 0) // page) for n in lens]) + spare
        pages = first + B * width + 1

        def make(*shape):
            return torch.randn(*shape[:-1], shape[-1] + gap, generator=g).to(dtype).cuda()[..., :shape[-1]]

        self.q, self.kc, self.vc = make(B, Hq, D), make(pages, page, Hk, D), make(pages, page, Hk, D)
        ids = torch.randperm(pages, generator=g).to(torch.int32)
        self.prefix = ids[:first].contiguous().cuda()
        self.table = ids[first:first + B * width].reshape(B, width).contiguous().cuda()
        self.n0 = torch.tensor([n0], dtype=torch.int32).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.scale = D ** -0.5 if scale is None else scale
        self.out = torch.full((B, Hq, D), 7.0, dtype=dtype, device="cuda")

    def run(self, ssu, **kw):
        return ssu.shared_prefix_attention(self.q, self.kc, self.vc, self.prefix, self.n0, self.table, self.lens, scale=self.scale,
                                           out=self.out, return_lse=True, **kw)

    def ref(self):
        f = seq_ref.f64
        return shared_ref.shared_prefix_attention(f(self.q), f(self.kc), f(self.vc), self.prefix.cpu().numpy(), int(self.n0),
                                                  self.table.cpu().numpy(), self.lens.cpu().numpy(), self.scale, seq_ref.u_of(self.q.dtype))

    def check(self, ssu, **kw):
        with np.errstate(invalid="ignore"):
            want = self.ref()
        out, lse = self.run(ssu, **kw)
        seq_ref.assert_close(out, want["out"], want["out_tol"], "out")
        seq_ref.assert_close(lse, want["lse"], want["lse_tol"], "lse")
        assert (seq_ref.f64(out)[np.isnan(want["out"]).all(-1)] == 7.0).all(), "padding was written"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n0", [0, 1, 63, 64, 65, 127, 129, 500])
def test_prefix_lengths(ssu, D, dtype, n0):
    Case([5, 0, 40], n0, D=D, dtype=dtype, seed=n0).check(ssu)


@pytest.mark.parametrize("page", [1, 3, 8, 16, 20, 48, 64, 100, 128, 1000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages(ssu, page, D):
    Case([page + 3, 1, 2 * page], 3 * page + 77, D=D, page=page, seed=page).check(ssu)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (16, 2), (5, 5), (17, 1), (40, 2), (64, 4), (12, 3)])
@pytest.mark.parametrize("B", [1, 2, 7, 33, 70])
def test_heads_and_batches(ssu, Hq, Hk, B):
    """Rows of a key head in less than a wave, in several waves, in several workgroups."""
    Case([(5 * i) % 41 for i in range(B)], 200, Hq, Hk, 64, seed=B + Hq).check(ssu)


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, BF16), (128, F16), (256, F16)])
def test_long(ssu, D, dtype):
    """Many pieces, and own tokens of several runs."""
    Case([700, 3, 0, 1500], 5003, 4, 2, D, dtype=dtype, seed=D).check(ssu)
    Case([9], 20011, 4, 1, D, dtype=dtype, seed=D).check(ssu)


def test_lengths_beyond_the_tables_and_padding(ssu):
    c = Case([30, -1, 10 ** 6, 0, -7, 5], 150, seed=1)
    c.table = c.table[:, :3].contiguous()
    c.prefix = c.prefix[:7].contiguous()
    c.check(ssu)
    c.n0.fill_(-3)
    c.check(ssu)
    c.prefix = c.prefix[:0]
    c.n0.fill_(100)
    c.check(ssu)


def test_empty_tables(ssu):
    c = Case([0, 3, -1], 100, seed=2)
    c.table = c.table[:, :0].contiguous()
    c.check(ssu)
    c.n0.zero_()
    out, lse = c.run(ssu)
    assert (out[:2] == 0).all() and (lse[:2] == -float("inf")).all() and (out[2] == 7.0).all()


def test_no_requests(ssu):
    c = Case([3], 10)
    out = ssu.shared_prefix_attention(c.q[:0], c.kc, c.vc, c.prefix, c.n0, c.table[:0], c.lens[:0])
    assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("D", [64, 128])
def test_bad_pages_and_what_nobody_sees(ssu, D):
    """Tokens of page ids outside the cache are not visible, wherever in a tile they end; rows that
    nobody sees may hold NaN and infinities."""
    for page in (8, 16, 64):
        c = Case([20, 33], 300, D=D, page=page, seed=page)
        bad = [i for i in (0, 3, 4, 9) if i < len(c.prefix)]
        gone = c.prefix[bad].long()
        c.prefix[bad] = torch.tensor([-1, 10 ** 9, c.kc.shape[0], -2 ** 31], dtype=torch.int32)[:len(bad)].cuda()
        c.table[1, 0] = -5
        c.check(ssu)
        out = c.out.clone()
        c.kc[gone], c.vc[gone] = float("nan"), float("inf")
        last = c.prefix[300 // page].long()
        if 0 <= last < c.kc.shape[0]:
            c.kc[last, 300 % page:], c.vc[last, 300 % page:] = float("inf"), float("nan")
        c.run(ssu)
        assert torch.equal(c.out, out)
        c.prefix.fill_(-1)
        c.check(ssu)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_and_nan(ssu, dtype, D):
    """Infinities in visible rows of V give the formula's: an infinity, NaN where both signs meet, also
    where the row's weight is too small for 16 bits. NaN in a query stays in its head."""
    inf = float("inf")
    c = Case([4, 9, 0], 200, 4, 1, D, dtype=dtype, seed=3)
    pg = c.prefix.long()
    c.vc[pg[1], 2, 0, 5] = inf
    c.vc[pg[9], 7, 0, 7], c.vc[pg[3], 1, 0, 7] = inf, -inf
    c.vc[pg[5], 1, 0, 8] = -inf
    c.kc[pg[1], 2] = -4 * c.q[0, 0]  # (far below the others for one row)
    out, _ = c.run(ssu)
    want = c.ref()["out"]
    assert np.array_equal(np.isnan(seq_ref.f64(out)), np.isnan(want)) and np.isnan(want[..., 7]).all()
    assert np.array_equal(np.isinf(seq_ref.f64(out)), np.isinf(want)) and (want[..., 5] == inf).all() and (want[..., 8] == -inf).all()
    rest = np.isfinite(want)
    np.testing.assert_allclose(seq_ref.f64(out)[rest], want[rest], atol=4 * seq_ref.u_of(dtype), rtol=4 * seq_ref.u_of(dtype))
    c = Case([4, 9, 0], 200, 4, 1, D, dtype=dtype, seed=3)
    clean = c.run(ssu)[0].clone()
    c.q[1, 2, 3] = float("nan")
    out, lse = c.run(ssu)
    assert out[1, 2].isnan().all() and lse[1, 2].isnan()
    out[1, 2] = clean[1, 2]
    assert torch.equal(out, clean)


def test_scores_of_minus_infinity(ssu):
    """Keys that no query sees by their scores: they weigh nothing; if all are so, out is 0."""
    c = Case([0, 3], 100, 2, 1, 64, seed=4)
    c.q.fill_(1.0)
    c.kc[c.prefix[:3].long()] = -float("inf")
    c.check(ssu)
    c.kc[c.prefix.long()] = -float("inf")
    out, lse = c.run(ssu)
    assert (out[0] == 0).all() and (lse[0] == -float("inf")).all() and out[1].isfinite().all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(ssu, scale):
    Case([9, 0], 300, seed=5, scale=scale).check(ssu)


def test_growing_scores(ssu):
    """Scores that rise over the prefix: the running maximum changes at every tile."""
    c = Case([0, 5], 700, 2, 1, 64, seed=6)
    c.q.fill_(0.5)
    ramp = torch.linspace(0, 2, 700, device="cuda")
    for j in range(700):
        c.kc[c.prefix[j // 16].long(), j % 16] += ramp[j]
    c.check(ssu)


@pytest.mark.parametrize("gap", [1, 8])
def test_strides(ssu, gap):
    Case([9, 40], 130, 4, 2, 64, seed=7, gap=gap).check(ssu)


def test_agrees_with_paged_attention(ssu):
    """The prefix as the first pages of every request's own table."""
    c = Case([30, 7, 100], 160, 8, 2, 128, seed=8)
    out, lse = c.run(ssu)
    table = torch.cat((c.prefix[:10].expand(3, 10), c.table), 1).contiguous()
    want, want_lse = ssu.paged_attention(c.q, c.kc, c.vc, table, c.lens + 160, scale=c.scale, return_lse=True)
    # two roundings of out, one of the weights: each at most 2^-8 of values of order 1
    assert (out.float() - want.float()).abs().max() <= 3 * 2.0 ** -8 and (lse - want_lse).abs().max() <= 2.0 ** -18


def test_same_bits(ssu):
    a, b = (Case([700, 3, 0, 64], 5003, 8, 2, 128, seed=9) for _ in range(2))
    x = a.run(ssu)
    need = ssu.shared_prefix_attention_workspace(4, 8, 2, 128, 16, a.table.shape[1], a.prefix.shape[0])
    y = b.run(ssu, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("lens", [[700, 3, 0, 64], [20, 3]])
def test_streams_and_graphs(ssu, lens):
    """A captured call reads the prefix's length and the requests' at the replay."""
    c = Case(lens, 1003, 8, 2, 64, seed=10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(ssu, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    got = [x.clone() for x in got]
    want = [x.clone() for x in c.run(ssu)]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.run(ssu)
    for n0, n in ((1003, 3), (0, 2), (77, 0), (1, 20)):
        c.n0.fill_(n0)
        c.lens[-1] = n
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone(), lse.clone()
        eager = c.run(ssu)
        assert torch.equal(replayed[0], eager[0]) and torch.equal(replayed[1], eager[1])


def test_refusals(ssu):
    c = Case([3, 5], 100)
    call = lambda **kw: ssu.shared_prefix_attention(**{**dict(  # noqa: E731
        q=c.q, k_cache=c.kc, v_cache=c.vc, prefix_table=c.prefix, prefix_len=c.n0, block_table=c.table, seq_lens=c.lens), **kw})
    call()
    for kw, error in ((dict(prefix_table=c.prefix.long()), TypeError), (dict(prefix_table=c.prefix[None]), ValueError),
                      (dict(prefix_table=c.prefix.cpu()), ValueError), (dict(prefix_len=c.lens), ValueError),
                      (dict(prefix_len=c.n0[0]), ValueError), (dict(prefix_len=100), TypeError), (dict(prefix_len=c.n0.float()), TypeError),
                      (dict(q=c.q.float()), TypeError), (dict(q=c.q[..., :32]), ValueError), (dict(seq_lens=c.lens[:1]), ValueError),
                      (dict(scale=float("nan")), ssu.SSUError), (dict(prefix_table=c.prefix.repeat_interleave(2)[::2]), ssu.SSUError),
                      (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), ssu.SSUError)):
        with pytest.raises(error):
            call(**kw)
    with torch.enable_grad(), pytest.raises(ValueError, match="inference only"):
        call(q=c.q.clone().requires_grad_())
