"""Tensors that the delta rule, the residual norm and attention over a shared prefix would not read
as torch does are refused, whichever operand they are; and a run of a hybrid model's layers."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from . import delta_ref, seq_ref, shared_ref
from .gpu_util import require_gpu
from .test_seq_tensors_gpu import attention, linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def norm():
    h = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(x=h(3, 64), residual=h(3, 64), weight=h(64), out=h(3, 64))


def shared():
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(attention(), prefix_table=i(1, 0), prefix_len=i(20))


CALLS = [("gated_delta_rule", linear), ("add_rms_norm", norm), ("shared_prefix_attention", shared)]
FLOATS = [(f, make, name) for f, make, names in
          (("gated_delta_rule", linear, ("state", "q", "k", "v", "log_decay", "beta")),
           ("add_rms_norm", norm, ("x", "residual", "weight", "out")),
           ("shared_prefix_attention", shared, ("q", "k_cache", "v_cache", "out"))) for name in names]


@pytest.mark.parametrize("f,make", CALLS)
def test_plain_tensors_run(ssu, f, make):
    getattr(ssu, f)(**make())


@pytest.mark.parametrize("f,make,name", FLOATS)
def test_dual_tensors(ssu, f, make, name):
    a = make()
    with fwd.dual_level():
        a[name] = fwd.make_dual(a[name], torch.ones_like(a[name]))
        with torch.no_grad(), pytest.raises(ValueError, match=f"no tangent is carried for {name}"):
            getattr(ssu, f)(**a)
        a[name] = fwd.unpack_dual(a[name]).primal
        getattr(ssu, f)(**a)


@pytest.mark.parametrize("f,make,name", FLOATS)
def test_negated_views(ssu, f, make, name):
    a = make()
    a[name] = torch._neg_view(a[name])
    with pytest.raises(ValueError, match=f"{name} is a view of negated memory"):
        getattr(ssu, f)(**a)
    a[name] = a[name].resolve_neg()
    getattr(ssu, f)(**a)


@pytest.mark.parametrize("f,make", CALLS)
def test_streams_of_their_own(ssu, f, make):
    """Two calls at once, each with memory of its own, are the same calls one after the other."""
    torch.manual_seed(3)
    first, second = make(), make()
    copy = lambda a: {k: v.clone() for k, v in a.items()}  # noqa: E731
    want = [getattr(ssu, f)(**copy(a)) for a in (first, second)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    operands = [copy(first), copy(second)]
    torch.cuda.synchronize()
    got = [getattr(ssu, f)(**a, stream=s) for a, s in zip(operands, streams)]
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_a_decode_step_of_a_hybrid_model(ssu):
    """norm -> delta rule -> norm -> rotation into the cache -> attention behind the shared prefix, one token for
    each of five requests, each result against fp64 on the operator's own inputs."""
    torch.manual_seed(5)
    B, D, H, P, N, Hq, Hk, page, n0 = 5, 256, 4, 64, 64, 4, 2, 16, 100
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    h = lambda *s: r(*s).to(torch.bfloat16)  # noqa: E731
    f = seq_ref.f64
    x, residual, w = h(B, D), r(B, D), h(D)
    s, y = delta_ref.add_rms_norm(f(x), f(residual), f(w), 1e-6)
    hidden = ssu.add_rms_norm(x, residual, w)
    seq_ref.assert_close(hidden, y, 2.0 ** -8 * abs(y) + (D + 20) * seq_ref.EPS32 * abs(y), "norm")
    seq_ref.assert_close(residual, s, 2 * seq_ref.EPS32 * (abs(f(x)) + abs(s) + abs(s - f(x))), "residual")

    packed = (hidden @ (h(D, 3 * H * N) / 16)).to(torch.bfloat16).view(B, 3, H, N)
    q, k, v = packed.unbind(1)
    state, idx = r(B + 2, H, P, N), torch.randperm(B + 2, device="cuda")[:B]
    decay, beta = -r(B, H).abs(), torch.rand(B, H, device="cuda")
    want = delta_ref.gated_delta(f(state), f(q), f(k), f(v), f(decay), list(range(B + 1)), idx.cpu().numpy(), f(beta), 0.125, True, 1)
    out = ssu.gated_delta_rule_step(state, q, k, v, decay, beta, idx, scale=0.125, normalize=True)
    seq_ref.assert_close(out, want["out"], want["out_tol"], "rule")
    seq_ref.assert_close(state, want["state"], want["state_tol"], "state")

    hidden8, scales = ssu.add_rms_norm(out.reshape(B, H * P), residual, w, quantize=True, group=128)
    again = (hidden8.float().view(B, -1, 128) * scales[..., None]).view(B, D)
    packed = (again.to(torch.bfloat16) @ (h(D, (Hq + 2 * Hk) * N) / 16)).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (-1, N)) for t in packed.split((Hq * N, Hk * N, Hk * N), 1))
    kc, vc = h(30, page, Hk, N), h(30, page, Hk, N)
    prefix, table = torch.arange(7, dtype=torch.int32, device="cuda"), torch.arange(10, 25, dtype=torch.int32, device="cuda").view(B, 3)
    lens = torch.tensor([1, 16, 17, 33, 48], dtype=torch.int32, device="cuda")
    at = lens.long() - 1
    slots = table.long()[torch.arange(B), at // page] * page + at % page
    angle = torch.arange(200, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, N, 2, device="cuda") / N)
    q, _ = ssu.qk_norm_rope(q, k, n0 + at, torch.cat((angle.cos(), angle.sin()), 1).float(), v=v, k_cache=kc, v_cache=vc, slots=slots)
    n = torch.tensor([n0], dtype=torch.int32, device="cuda")
    out, lse = ssu.shared_prefix_attention(q, kc, vc, prefix, n, table, lens, return_lse=True)
    want = shared_ref.shared_prefix_attention(f(q), f(kc), f(vc), prefix.cpu().numpy(), n0, table.cpu().numpy(), lens.cpu().numpy(), N ** -0.5,
                                              2.0 ** -8)
    seq_ref.assert_close(out, want["out"], want["out_tol"], "attention")
    seq_ref.assert_close(lse, want["lse"], want["lse_tol"], "lse")
