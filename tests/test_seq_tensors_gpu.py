"""Tensors that the sequence operators would not read as torch does are refused, whichever operand they are."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def linear():
    r = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    h = lambda *s: r(*s).to(torch.bfloat16)  # noqa: E731
    return dict(state=r(3, 2, 16, 32), q=h(8, 1, 32), k=h(8, 1, 32), v=h(8, 2, 16), log_decay=-r(8, 2).abs(),
                cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"),
                state_batch_indices=torch.tensor([1], device="cuda"), beta=r(8, 2))


def rope():
    h = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(q=h(4, 2, 64), k=h(4, 1, 64), positions=torch.arange(4, device="cuda"), cos_sin=torch.randn(8, 64, device="cuda"),
                q_weight=h(64), k_weight=h(64), v=h(4, 1, 64), k_cache=h(2, 4, 1, 64), v_cache=h(2, 4, 1, 64),
                slots=torch.arange(4, device="cuda"))


def attention():
    h = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)  # noqa: E731
    return dict(q=h(2, 2, 64), k_cache=h(2, 16, 1, 64), v_cache=h(2, 16, 1, 64),
                block_table=torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"),
                seq_lens=torch.tensor([3, 16], dtype=torch.int32, device="cuda"), out=h(2, 2, 64))


CALLS = [("linear_attention", linear), ("qk_norm_rope", rope), ("paged_attention", attention)]
FLOATS = [(f, make, name) for f, make, names in
          (("linear_attention", linear, ("state", "q", "k", "v", "log_decay", "beta")),
           ("qk_norm_rope", rope, ("q", "k", "cos_sin", "q_weight", "k_weight", "v", "k_cache", "v_cache")),
           ("paged_attention", attention, ("q", "k_cache", "v_cache", "out"))) for name in names]


@pytest.mark.parametrize("f,make", CALLS)
def test_plain_tensors_run(ssu, f, make):
    getattr(ssu, f)(**make())


@pytest.mark.parametrize("f,make,name", FLOATS)
def test_dual_tensors(ssu, f, make, name):
    """A forward-mode tangent would be dropped without a word, also under no_grad."""
    a = make()
    with fwd.dual_level():
        a[name] = fwd.make_dual(a[name], torch.ones_like(a[name]))
        with torch.no_grad(), pytest.raises(ValueError, match=f"no tangent is carried for {name}"):
            getattr(ssu, f)(**a)
        a[name] = fwd.unpack_dual(a[name]).primal
        getattr(ssu, f)(**a)


@pytest.mark.parametrize("f,make,name", FLOATS)
def test_negated_views(ssu, f, make, name):
    """Their memory holds the values' negatives (a conjugate's imaginary part is one)."""
    a = make()
    a[name] = torch._neg_view(a[name])
    with pytest.raises(ValueError, match=f"{name} is a view of negated memory"):
        getattr(ssu, f)(**a)
    a[name] = a[name].resolve_neg()
    getattr(ssu, f)(**a)
