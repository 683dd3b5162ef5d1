"""ssu_add_rms_norm against fp64 (tests/delta_ref.py), at the widths, types and layouts
where it can go wrong."""
import numpy as np
import pytest
import torch

from . import delta_ref, seq_ref
from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
TINY = 2.0 ** -126


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def operands(T, D, dtype=BF16, res=None, wtype=None, seed=0, gap=0):
    g = torch.Generator().manual_seed(seed)

    def make(dtype, size=1.0):
        return (size * torch.randn(T, D + gap, generator=g)).to(dtype).cuda()[:, :D]

    x = make(dtype)
    residual = None if res is None else make(res, 3.0)
    weight = None if wtype is None else (1 + 0.3 * torch.randn(D, generator=g)).to(wtype).cuda()
    return x, residual, weight


def check(ssu, x, residual, weight, eps=1e-6, quantize=False, group=0, **kw):
    """fp32 in between: a sum of D squares, a root, a division, two products; each output rounded once."""
    f = seq_ref.f64
    T, D = x.shape
    before = None if residual is None else f(residual)
    s, y = delta_ref.add_rms_norm(f(x), before, None if weight is None else f(weight), eps)
    got = ssu.add_rms_norm(x, residual, weight, eps=eps, quantize=quantize, group=group, **kw)
    if residual is not None:
        u = 0.0 if residual.dtype == F32 else seq_ref.u_of(residual.dtype)
        least = 2.0 ** -25 if residual.dtype == F16 else 0.0
        size = np.abs(f(x)) + np.abs(before) if T else 0
        seq_ref.assert_close(residual, s, u * np.abs(s) + 2 * seq_ref.EPS32 * size + least, "residual")
    rough = (D + 16) * seq_ref.EPS32 * np.abs(y)  # (x + residual that cancel are rounded relative to what is left: exact in 16 bits)
    if residual is not None and residual.dtype == F32:
        rough = rough + 4 * seq_ref.EPS32 * np.abs(y)
    if not quantize:
        u = seq_ref.u_of(x.dtype)
        seq_ref.assert_close(got, y, u * np.abs(y) + rough + (2.0 ** -25 if x.dtype == F16 else 1e-38), "out")
        return got
    q, scales = got
    n = group or D
    assert q.dtype == E4M3 and q.shape == (T, D) and scales.shape == (T, D // n)
    most = np.abs(y).reshape(T, D // n, n).max(-1)
    seq_ref.assert_close(scales, np.maximum(most / 448, TINY), (D + 20) * seq_ref.EPS32 * most / 448 + 1e-44, "scales")
    v, unit = y.reshape(T, D // n, n), np.maximum(most / 448, TINY)[..., None]
    ratio = (v / unit).reshape(T, D)
    # half a step of three bits of fraction, 2^-9 below 2^-6
    seq_ref.assert_close(q.float(), ratio, np.maximum(2.0 ** -4 * np.abs(ratio), 2.0 ** -10) * (1 + 2.0 ** -10)
                         + 2 * (D + 20) * seq_ref.EPS32 * np.abs(ratio), "8 bits")
    return got


@pytest.mark.parametrize("D", [1, 2, 7, 8, 9, 16, 31, 64, 100, 256, 511, 512, 513, 520, 1000, 1024, 2048, 4096, 4100, 5120, 8192, 16384,
                               16392, 24000, 32760, 32768])
@pytest.mark.parametrize("quantize", [False, True])
def test_widths(ssu, D, quantize):
    for i, (dtype, res) in enumerate(((BF16, BF16), (F16, F32), (BF16, None))):
        check(ssu, *operands(3, D, dtype, res, dtype, seed=D + i), quantize=quantize)


@pytest.mark.parametrize("T", [0, 1, 2, 3, 5, 63, 64, 65, 257, 1000])
@pytest.mark.parametrize("D", [24, 1000])
def test_rows(ssu, T, D):
    check(ssu, *operands(T, D, BF16, BF16, F32, seed=T))
    check(ssu, *operands(T, D, BF16, F32, None, seed=T), quantize=True)


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("many", [1, 2, 3, 5, 7, 16, 33, 100])
@pytest.mark.parametrize("res", [None, F16, F32])
def test_groups(ssu, group, many, res):
    check(ssu, *operands(5, group * many, F16, res, F16, seed=many), quantize=True, group=group)


@pytest.mark.parametrize("gap", [1, 2, 3, 8])
@pytest.mark.parametrize("D", [33, 1016])
def test_strides(ssu, gap, D):
    """Rows that begin anywhere, and what lies between them stays."""
    x, r, w = operands(9, D, BF16, BF16, BF16, seed=gap, gap=gap)
    base = torch.full((9, D + gap), 7.0, dtype=BF16, device="cuda")
    check(ssu, x, r, w, out=base[:, :D])
    assert (base[:, D:] == 7.0).all()
    bytes_ = torch.full((9, D + gap), 7, dtype=torch.uint8, device="cuda")
    wide = torch.full((9, 3), 7.0, device="cuda")
    check(ssu, *operands(9, D, BF16, F32, BF16, seed=gap, gap=gap), quantize=True, out=bytes_.view(E4M3)[:, :D], scales=wide[:, 1:2])
    assert (bytes_[:, D:] == 7).all() and (wide[:, ::2] == 7.0).all()


@pytest.mark.parametrize("D", [40, 2000, 9000])
def test_in_place(ssu, D):
    x, r, w = operands(130, D, BF16, BF16, BF16, seed=1)
    want_r = r.clone()
    want = ssu.add_rms_norm(x, want_r, w)
    got = ssu.add_rms_norm(x, r, w, out=x)
    assert got is x and torch.equal(x, want) and torch.equal(r, want_r)


@pytest.mark.parametrize("D,group", [(256, 0), (256, 64), (8192, 0), (8192, 128)])
def test_special_rows(ssu, D, group):
    """Zeros, values near fp32's least, infinities and NaN: each in its own row, the other rows untouched by it."""
    x, _, _ = operands(6, D, BF16, None, None, seed=2)
    clean = ssu.add_rms_norm(x, quantize=True, group=group)
    y = x.clone()
    y[0] = 0
    y[1] = 1e-38
    y[2, 5] = float("nan")
    y[3, 5] = float("inf")
    y[4] = 3e38
    q, scales = ssu.add_rms_norm(y, quantize=True, group=group)
    assert (q[0].float() == 0).all() and (scales[0] == np.float32(TINY)).all()
    assert q[1].float().isfinite().all()
    assert q[2].float().isnan().all() and scales[2].isnan().all()
    assert q[3, 5].float().isnan() and scales[3, 0].isnan()  # infinity over infinity; the rest of the row is 0
    assert group == 0 or (q[3, group:].float() == 0).all()
    assert (q[4].float() == 0).all()  # (its squares are beyond fp32)
    assert torch.equal(q[5].view(torch.uint8), clean[0][5].view(torch.uint8)) and torch.equal(scales[5], clean[1][5])
    out = ssu.add_rms_norm(y)
    assert out[2].isnan().all() and out[3, 5].isnan() and (out[3, 6:] == 0).all() and (out[4] == 0).all() and (out[0] == 0).all()


def test_a_nan_in_the_weight_stays_in_its_group(ssu):
    x, _, w = operands(3, 256, BF16, None, F32, seed=3)
    w[70] = float("nan")
    q, scales = ssu.add_rms_norm(x, weight=w, quantize=True, group=64)
    assert scales[:, 1].isnan().all() and q[:, 64:128].float().isnan().all()
    assert scales[:, [0, 2, 3]].isfinite().all() and q[:, :64].float().isfinite().all()


def test_small_values_keep_the_least_scale(ssu):
    """A weight that makes the norm smaller than 448 times the least scale."""
    x, _, _ = operands(2, 64, BF16, None, None, seed=3)
    w = torch.full((64,), 2.0 ** -120, device="cuda")
    q, scales = ssu.add_rms_norm(x, weight=w, quantize=True)
    assert (scales == np.float32(TINY)).all()
    y = delta_ref.add_rms_norm(seq_ref.f64(x), None, seq_ref.f64(w), 1e-6)[1] / TINY
    seq_ref.assert_close(q.float(), y, np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) * 1.001, "8 bits")


@pytest.mark.parametrize("T,D,quantize", [(3, 100, False), (40, 8192, True)])
def test_streams_and_graphs(ssu, T, D, quantize):
    x, r, w = operands(T, D, BF16, BF16, BF16, seed=4)
    first = r.clone()

    def bits(y):
        return [t.view(torch.uint8) for t in (y if quantize else (y,))]

    want = bits(ssu.add_rms_norm(x, r, w, quantize=quantize))
    s = torch.cuda.Stream()
    r.copy_(first)
    s.wait_stream(torch.cuda.current_stream())
    got = bits(ssu.add_rms_norm(x, r, w, quantize=quantize, stream=s))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bits(ssu.add_rms_norm(x, r, w, quantize=quantize))
    for _ in range(3):
        r.copy_(first)
        graph.replay()
        other = first.clone()
        eager = bits(ssu.add_rms_norm(x, other, w, quantize=quantize))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, e) for a, b, e in zip(got, want, eager)) and torch.equal(r, other)


def test_refusals(ssu):
    x, r, w = operands(3, 64, BF16, BF16, BF16)
    for kw, error in ((dict(x=x.float()), TypeError), (dict(x=x[0]), ValueError), (dict(residual=r[:2]), ValueError),
                      (dict(residual=r.half()), TypeError), (dict(weight=w[:5]), ValueError), (dict(group=32), ValueError),
                      (dict(quantize=True, group=48), ValueError), (dict(quantize=True, group=16), ssu.SSUError),
                      (dict(scales=torch.empty(3, 1, device="cuda")), ValueError), (dict(eps=-1.0), ssu.SSUError),
                      (dict(quantize=True, out=torch.empty_like(x)), TypeError), (dict(x=x.cpu()), ValueError),
                      (dict(x=x.T.contiguous().T, residual=None), ssu.SSUError), (dict(residual=r[:1].expand(3, 64)), ssu.SSUError),
                      (dict(quantize=True, group=-1), ValueError)):
        with pytest.raises(error):
            ssu.add_rms_norm(**{**dict(x=x, residual=r, weight=w), **kw})
    with torch.enable_grad(), pytest.raises(ValueError, match="inference only"):
        ssu.add_rms_norm(x.clone().requires_grad_())
