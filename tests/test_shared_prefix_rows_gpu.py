"""ssu_shared_prefix_attention where rows hold what no result comes of: padding requests' queries, whatever they hold,
and queries that are NaN."""
import pytest
import torch

from .gpu_util import require_gpu
from .test_shared_prefix_gpu import BF16, F16, Case

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def ssu():
    require_gpu()
    import selective_state_update_amd as m

    return m


def workspace(ssu, c):
    B, Hq, D = c.q.shape
    need = ssu.shared_prefix_attention_workspace(B, Hq, c.kc.shape[2], D, c.kc.shape[1], c.table.shape[1], c.prefix.shape[0])
    return torch.full((need,), 85, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("D,dtype", [(64, BF16), (128, F16), (256, BF16)])
@pytest.mark.parametrize("lens", [[5, -1, 9], [-1] * 9 + [3] * 40 + [-1] * 30, [-3, -1]])
def test_queries_of_padding_requests(ssu, D, dtype, lens):
    """What they hold is not read into anything: the same bits everywhere, the workspace included."""
    results = []
    for value in (0.5, NAN, INF):
        c = Case(lens, 500, 8, 2, D, dtype=dtype, seed=D)
        c.q[c.lens < 0] = value
        c.check(ssu)
        ws = workspace(ssu, c)
        c.out.fill_(7.0)
        out, lse = c.run(ssu, workspace=ws)
        live = c.lens >= 0
        results.append((out, lse[live], ws))
    for other in results[1:]:
        for x, y in zip(results[0], other):
            assert torch.equal(x, y)


def least_time(f):
    for _ in range(2):
        f()
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


@pytest.mark.parametrize("row", ["padding", "live"])
def test_time_of_nan(ssu, row):
    """A NaN in a query does not hold the other requests up. (Token by token, 20 to 100 times as long, would go only rows
    that infinities of V reach.)"""
    c = Case([5, -1, 9, 3], 8000, 8, 2, 128, seed=1)
    ws = workspace(ssu, c)
    finite = least_time(lambda: c.run(ssu, workspace=ws))
    c.q[1 if row == "padding" else 0] = NAN
    assert least_time(lambda: c.run(ssu, workspace=ws)) <= 4 * finite


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("D,tokens", [(64, 400), (128, 12000), (256, 3000)])
def test_time_of_nan_among_own_tokens(ssu, D, tokens, shared):
    """The same for a request's own tokens, here and in paged_attention, in a workgroup of its own and in several."""
    c = Case([5, tokens, 9], 100, 4, 2, D, seed=2)
    ws = workspace(ssu, c)

    def call():
        if shared:
            return c.run(ssu, workspace=ws)
        return ssu.paged_attention(c.q, c.kc, c.vc, c.table, c.lens, scale=c.scale, out=c.out, return_lse=True, workspace=ws)

    finite, clean = least_time(call), [x.clone() for x in call()]
    c.q[1, 2, 3] = NAN
    slow = least_time(call)
    out, lse = call()
    assert out[1, 2].isnan().all() and lse[1, 2].isnan()
    out[1, 2], lse[1, 2] = clean[0][1, 2], clean[1][1, 2]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    assert slow <= 4 * finite, (slow, finite)
