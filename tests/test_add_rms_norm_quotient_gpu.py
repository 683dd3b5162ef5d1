"""ssu_add_rms_norm to 8 bits: out is y / scale, divided in fp32 and then rounded once, also where the quotient
lies halfway between two 8-bit values."""
import pytest
import torch

from .gpu_util import require_gpu

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def halves(unit):
    """Values whose quotient by `unit` is, in fp32, halfway between two 8-bit values, or one fp32 step beside that."""
    steps = torch.arange(0, 126, dtype=torch.uint8).view(E4M3).float()
    middle = (steps[1:] + steps[:-1]) / 2  # exact in fp32
    y = middle * unit
    near = torch.stack([torch.nextafter(y, torch.zeros(())), y, torch.nextafter(y, torch.full((), 1e30))], 1).flatten()
    return near


@pytest.mark.parametrize("size", [1.0, 2.0 ** -85, 2.0 ** -113, 2.0 ** 100])
@pytest.mark.parametrize("D,group", [(4096, 0), (4096, 128), (4096, 32), (391, 0), (384, 64)])
def test_halfway(ssu, D, group, size):
    """x of +-1 and eps = 0: the norm is the weight, exactly, and so is what is divided."""
    g = torch.Generator().manual_seed(D + group)
    n = group or D
    w = torch.empty(D // n, n)
    for i in range(D // n):
        most = 448 * size * torch.exp2(4 * torch.rand((), generator=g) - 2)
        unit = most / 448
        y = halves(unit)
        w[i] = y[torch.randint(0, len(y), (n,), generator=g)].minimum(most)
        w[i, 0] = most
    w = w.reshape(-1)
    x = (2.0 * torch.randint(0, 2, (3, D), generator=g) - 1).to(torch.bfloat16)
    q, scales = ssu.add_rms_norm(x.cuda(), weight=w.cuda(), eps=0.0, quantize=True, group=group)
    y = (x.float() * w).reshape(3, D // n, n)
    unit = y.abs().amax(-1, keepdim=True) / 448
    assert torch.equal(scales.cpu(), unit[..., 0])
    want = (y / unit).reshape(3, D).to(E4M3)
    assert torch.equal(q.cpu().view(torch.uint8), want.view(torch.uint8))
    # (the product with a rounded reciprocal is another value: the operands tell the two apart)
    assert not torch.equal((y * (1 / unit)).reshape(3, D).to(E4M3).view(torch.uint8), want.view(torch.uint8))
