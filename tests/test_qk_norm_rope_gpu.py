"""ssu_qk_norm_rope against the definition in fp64 (tests/seq_ref.py)."""
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


def table(rows, rot):
    angle = torch.arange(rows, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    return torch.cat((angle.cos(), angle.sin()), 1).float().cuda()


class Case:
    def __init__(self, T, nq, nk, D, rot, dtype=BF16, inter=False, page=0, seed=0, weights="same", rows=500, gap=0, wide=False):
        g = torch.Generator().manual_seed(seed)
        packed = torch.randn(T, (nq + 2 * nk) * D + gap, generator=g).to(dtype).cuda()
        self.q = packed[:, :nq * D].unflatten(1, (nq, D)) if nq else packed.new_empty(T, 0, D)
        self.k = packed[:, nq * D:(nq + nk) * D].unflatten(1, (nk, D)) if nk else packed.new_empty(T, 0, D)
        self.v = packed[:, (nq + nk) * D:(nq + 2 * nk) * D].unflatten(1, (nk, D)) if nk else packed.new_empty(T, 0, D)
        self.packed, self.inter, self.dtype, self.eps = packed, inter, dtype, 1e-5
        self.cos_sin = table(rows, rot)
        self.pos = torch.randint(0, rows, (T,), generator=g).to(torch.int64 if seed % 2 else torch.int32).cuda()
        w = lambda: (1 + 0.3 * torch.randn(D, generator=g)).to(torch.float32 if weights == "fp32" else dtype).cuda()  # noqa: E731
        self.wq, self.wk = (None, None) if weights == "none" else (w(), w())
        self.cache = {}
        if page:
            pages = -(-T // page) + 2
            kc, vc = (torch.randn(pages, page, nk, D, generator=g).to(dtype).cuda() for _ in range(2))
            slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32 if seed % 2 else torch.int64).cuda()
            self.cache = dict(v=self.v, k_cache=kc, v_cache=vc, slots=slots)

    def ref(self):
        u = seq_ref.u_of(self.dtype)
        return [seq_ref.norm_rope(seq_ref.f64(x), None if w is None else seq_ref.f64(w), self.pos.cpu().numpy(),
                                  seq_ref.f64(self.cos_sin), self.eps, self.inter, u) for x, w in ((self.q, self.wq), (self.k, self.wk))]

    def run(self, ssu, **kw):
        return ssu.qk_norm_rope(self.q, self.k, self.pos, self.cos_sin, self.wq, self.wk, eps=self.eps, interleaved=self.inter,
                                **self.cache, **kw)

    def check(self, ssu, **kw):
        (qy, qt), (ky, kt) = self.ref()
        c = self.cache
        kc, vc = (c["k_cache"].contiguous().clone(), c["v_cache"].contiguous().clone()) if c else (None, None)
        q, k = self.run(ssu, **kw)
        seq_ref.assert_close(q, qy, qt, "q")
        if k is not None:
            seq_ref.assert_close(k, ky, kt, "k")
        if not c:
            return q, k
        pages, page, nk, D = kc.shape
        want, tol = seq_ref.f64(kc).reshape(-1, nk, D), np.zeros((pages * page, nk, D))
        wv = vc.view(-1, nk, D)
        for t, s in enumerate(c["slots"].tolist()):
            if 0 <= s < pages * page and not np.isnan(ky[t]).any():
                want[s], tol[s] = ky[t], kt[t]
                wv[s] = self.v[t]
        seq_ref.assert_close(c["k_cache"].reshape(-1, nk, D), want, tol, "k_cache")
        assert torch.equal(c["v_cache"], vc), "v_cache"
        return q, k


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 64), (256, 256), (80, 32), (96, 96), (192, 64), (512, 512),
                                   (128, 0), (128, 34), (66, 66), (2, 2), (1, 0), (7, 4), (200, 8), (16, 16)])
def test_shapes(ssu, dtype, inter, D, rot):
    Case(5, 6, 2, D, rot, dtype, inter, seed=D + rot).check(ssu)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,D", [(3, 64), (45, 8), (45, 16), (45, 64), (45, 80), (45, 128), (45, 256), (45, 512)])
def test_rotation_widths(ssu, T, D, inter):
    """Every width's last pairs and what lies behind them; nothing beside the rows is written."""
    for rot in sorted({2, 4, 6, 10, 22, 50, D // 2 - 2, D // 2 + 2, D - 6, D - 4, D - 2}):
        if not 0 < rot <= D:
            continue
        c = Case(T, 40, 4, D, rot, BF16, inter, page=2, seed=D + rot, gap=1, weights="fp32" if rot % 4 else "same")
        wide = torch.full((T, 40, D + 3), 9.0, dtype=BF16, device="cuda")
        c.check(ssu, q_out=wide[..., 1:D + 1])
        assert (wide[..., 0] == 9.0).all() and (wide[..., D + 1:] == 9.0).all(), rot


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 22), (64, 32), (66, 30)])
def test_infinity_behind_the_rotated_part(ssu, D, rot, inter):
    """It makes its own row's norm infinite: every other element is 0, its own NaN."""
    c = Case(80, 24, 4, D, rot, inter=inter, seed=3)
    c.q[1, 1, D - 2] = float("inf")
    q, _ = c.run(ssu)
    want = torch.zeros(D, device="cuda")
    want[D - 2] = float("nan")
    assert torch.equal(q[1, 1].isnan(), want.isnan()) and (q[1, 1].nan_to_num() == 0).all()
    q[1, 1] = 0
    assert q.isfinite().all()


@pytest.mark.parametrize("page", [1, 16, 17])
@pytest.mark.parametrize("T", [1, 2, 33, 257])
def test_cache(ssu, T, page):
    Case(T, 4, 2, 128, 128, page=page, seed=T + page).check(ssu)
    Case(T, 3, 1, 64, 32, F16, True, page=page, seed=T + page + 1).check(ssu)


@pytest.mark.parametrize("nq,nk", [(1, 1), (8, 8), (7, 1), (40, 5), (4, 0), (0, 3), (96, 1)])
def test_heads(ssu, nq, nk):
    if nq:
        Case(9, nq, nk, 64, 64, seed=nq, weights="fp32").check(ssu)
    else:
        Case(9, nq, nk, 64, 64, seed=nq, weights="none").check(ssu)


def test_weights(ssu):
    for w in ("none", "fp32", "same"):
        Case(6, 4, 2, 128, 128, seed=3, weights=w).check(ssu)
    c = Case(6, 4, 2, 128, 128, seed=4)
    c.wk = None
    c.check(ssu)


def test_many_tokens(ssu):
    Case(3000, 8, 2, 128, 128, seed=5).check(ssu)


def test_in_place(ssu):
    for D, rot, inter in ((128, 128, False), (128, 64, True), (256, 256, False), (200, 34, False), (512, 512, False)):
        c = Case(40, 4, 2, D, rot, inter=inter, seed=6)
        (qy, qt), (ky, kt) = c.ref()
        q, k = c.run(ssu, q_out=c.q, k_out=c.k)
        assert q is c.q and k is c.k
        seq_ref.assert_close(q, qy, qt, "q")
        seq_ref.assert_close(k, ky, kt, "k")


def test_cache_and_k_out(ssu):
    c = Case(20, 4, 2, 128, 128, page=16, seed=7)
    k_out = torch.empty_like(c.k)
    _, k = c.check(ssu, k_out=k_out)
    assert k is k_out


def test_padding(ssu):
    """Positions outside the table skip the token, slots outside the cache the copy."""
    c = Case(12, 4, 2, 128, 128, page=16, seed=9)
    c.pos[2], c.pos[5] = -1, 500
    c.cache["slots"][3], c.cache["slots"][4] = -1, 1 << 40 if c.cache["slots"].dtype == torch.int64 else 1 << 30
    q_out = torch.full(c.q.shape, 7.0, dtype=BF16, device="cuda")
    q, _ = c.check(ssu, q_out=q_out)
    assert (q[[2, 5]] == 7.0).all()


def test_layouts(ssu):
    """Odd pitches and offsets, head-major operands, caches with room between heads."""
    c = Case(10, 3, 1, 64, 64, seed=11, gap=5)
    c.check(ssu)
    c = Case(10, 4, 2, 128, 128, page=8, seed=12)
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    c.packed = torch.nn.functional.pad(c.packed, (3, 0))
    c.k = c.packed[:, 3 + 4 * 128:3 + 6 * 128].unflatten(1, (2, 128))
    c.cache["v"] = c.v = c.packed[:, 3 + 6 * 128:3 + 8 * 128].unflatten(1, (2, 128))
    big = torch.randn(5, 2, 8, 129 * 2, device="cuda").to(BF16)  # [pages, heads, rows, wider than D]
    c.cache["k_cache"] = big[..., 1:129].transpose(1, 2)
    c.cache["v_cache"] = big[..., 130:258].transpose(1, 2)
    c.cache["slots"] = torch.randperm(40)[:10].cuda()
    c.check(ssu)


def test_extreme_rows(ssu):
    """Zero rows, rows whose squares leave fp16's range, infinities and NaN stay in their row."""
    c = Case(8, 2, 1, 128, 128, seed=13)
    c.q[1] = 0
    c.q[2] = 60000.0
    c.q[3] *= 1e-4
    c.check(ssu)
    (qy, qt), _ = c.ref()
    c.q[5, 1, 3] = float("inf")
    c.q[6, 0, 7] = float("nan")
    q, _ = c.run(ssu)
    assert torch.isnan(q[5, 1, 3]) and torch.isnan(q[6, 0]).all()
    qy[5, 1], qy[6, 0] = np.nan, np.nan
    seq_ref.assert_close(q, qy, qt, "other rows")


def test_graph_replays(ssu):
    c = Case(33, 4, 2, 128, 128, page=16, seed=15)
    eager, _ = c.run(ssu)
    eager = eager.clone()
    kc = c.cache["k_cache"].clone()
    out = torch.zeros_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ssu, q_out=out)
    for _ in range(3):
        out.zero_()
        c.cache["k_cache"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
        written = c.cache["slots"].long()
        assert torch.equal(c.cache["k_cache"].view(-1, 2, 128)[written], kc.view(-1, 2, 128)[written])


def test_stream_and_empty(ssu):
    c = Case(50, 4, 2, 128, 128, seed=16)
    (qy, qt), _ = c.ref()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    q, _ = c.run(ssu, stream=s)
    s.synchronize()
    seq_ref.assert_close(q, qy, qt, "q")
    e = Case(0, 4, 2, 128, 128, seed=17)
    assert e.run(ssu)[0].shape == (0, 4, 128)


def test_python_refusals(ssu):
    c = Case(4, 4, 2, 64, 64, page=4, seed=18)
    with pytest.raises(ValueError):
        ssu.qk_norm_rope(c.q, c.k, c.pos, c.cos_sin, k_cache=c.cache["k_cache"])
    with pytest.raises(TypeError):
        ssu.qk_norm_rope(c.q.float(), c.k, c.pos, c.cos_sin)
    with pytest.raises(TypeError):
        ssu.qk_norm_rope(c.q, c.k.half(), c.pos, c.cos_sin)
    with pytest.raises(ValueError):
        ssu.qk_norm_rope(c.q, c.k, c.pos[:-1], c.cos_sin)
    with pytest.raises(ssu.SSUError):
        ssu.qk_norm_rope(c.q, c.k, c.pos, c.cos_sin[:, :3])
    with pytest.raises(ssu.SSUError):
        ssu.qk_norm_rope(c.q, c.k, c.pos, c.cos_sin, eps=-1.0)
    with pytest.raises(ValueError):
        ssu.qk_norm_rope(c.q, c.k, c.pos, c.cos_sin, q_weight=c.wq.clone().float().requires_grad_())
    with torch.no_grad():
        ssu.qk_norm_rope(c.q, c.k, c.pos, c.cos_sin, q_weight=c.wq.clone().float().requires_grad_())
