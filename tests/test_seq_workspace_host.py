"""The sizes of workspaces from Python are the C ABI's."""
import pytest

from .test_seq_host import ATTN, LINEAR, change, lib, pack, ssu  # noqa: F401


@pytest.mark.parametrize("batch,ntokens,H,P,N,G", [(1, 5000, 16, 64, 128, 1), (1, 37, 16, 64, 128, 1), (4, 3000, 32, 128, 256, 4),
                                                   (3, 9000, 5, 80, 16, 5), (0, 0, 1, 16, 16, 1)])
def test_linear(ssu, lib, batch, ntokens, H, P, N, G):
    want = lib.ssu_linear_attention_workspace(pack("linear", change(LINEAR, dict(batch=batch, ntokens=ntokens, nheads=H, headdim=P,
                                                                                 dstate=N, ngroups=G))))
    assert want >= 0 and ssu.linear_attention_workspace(batch, ntokens, H, P, N, G) == want
    assert (want > 0) == (ntokens > 1000)


@pytest.mark.parametrize("batch,nq,nk,D,page,pages", [(1, 16, 2, 128, 16, 100), (64, 32, 8, 128, 64, 128), (3, 8, 1, 64, 1, 300),
                                                      (2, 4, 4, 256, 16, 17)])
def test_attention(ssu, lib, batch, nq, nk, D, page, pages):
    want = lib.ssu_paged_attention_workspace(pack("attn", change(ATTN, dict(batch=batch, nq=nq, nk=nk, headdim=D, page_size=page,
                                                                            max_pages=pages))))
    assert want >= 0 and ssu.paged_attention_workspace(batch, nq, nk, D, page, pages) == want


def test_refusals(ssu):
    with pytest.raises(ValueError, match="headdim 24"):
        ssu.linear_attention_workspace(1, 100, 4, 24, 64)
    with pytest.raises(ValueError, match="ngroups 3"):
        ssu.linear_attention_workspace(1, 100, 4, 64, 64, 3)
    with pytest.raises(ValueError, match="headdim 96"):
        ssu.paged_attention_workspace(1, 4, 2, 96, 16, 4)
    with pytest.raises(ValueError, match="batch is too large"):
        ssu.paged_attention_workspace(1 << 40, 4, 2, 64, 16, 4)
    with pytest.raises(TypeError):
        ssu.paged_attention_workspace(1.5, 4, 2, 64, 16, 4)
    with pytest.raises(TypeError):
        ssu.linear_attention_workspace(1, 100, 4)
