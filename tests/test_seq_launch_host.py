"""The sequence operators' launches are counted in 64 bits: what a launch does not
hold (2^32 threads) is refused before the GPU is touched, never cut to the bits that fit."""
import pytest

from .test_seq_host import ATTN, BF16, F32, LINEAR, NONE, QK, UNSUPPORTED, change, lib, pack, ssu, view  # noqa: F401


def step(**kw):
    """One token of each request, most of them padding: the pool holds few states."""
    P, N, H = kw["headdim"], kw["dstate"], kw["nheads"]
    return change(LINEAR, {"cu": NONE, "ws": 0, "ws_bytes": 0, "ntokens": kw["batch"], "ngroups": 1,
                           "state": view(F32, H * P * N, P * N, N, 1), "q": view(BF16, N, N, 1), "k": view(BF16, N, N, 1),
                           "v": view(BF16, H * P, P, 1), "out": view(BF16, H * P, P, 1), "decay": view(F32, H, 1),
                           "beta": view(F32, H, 1), **kw})


@pytest.mark.parametrize("kw", [
    dict(batch=1 << 26, nheads=1, headdim=256, dstate=256),           # 2^32 workgroups, 0 in 32 bits
    dict(batch=(1 << 26) + 1, nheads=1, headdim=256, dstate=256),     # 64 more
    dict(batch=1 << 22, nheads=16, headdim=256, dstate=128),          # 2^31: negative in 32 bits
    dict(batch=1 << 20, nheads=1, headdim=256, dstate=256),           # 2^26 of 64 threads
    dict(batch=1 << 24, nheads=4, headdim=16, dstate=16)])            # one workgroup a head, 2^26 again
def test_step(lib, kw):
    assert lib.ssu_linear_attention_step(pack("linear", step(**kw)), None) == UNSUPPORTED, lib.ssu_last_error()


def test_prompts(lib):
    kw = dict(batch=1 << 24, ntokens=1 << 20)  # 2^26 workgroups of 256 threads
    assert lib.ssu_linear_attention(pack("linear", change(LINEAR, kw)), None) == UNSUPPORTED, lib.ssu_last_error()


@pytest.mark.parametrize("kw", [
    dict(ntokens=1 << 23, headdim=66, rot=66),                        # 2^26 head rows, a wave each
    dict(ntokens=1 << 28, headdim=64),                                # groups of 8 lanes
    dict(ntokens=1 << 33, headdim=8, rot=8),
    dict(nq=(1 << 31) - 1), dict(nq=1 << 30, nk=1 << 30)])
def test_qk(lib, kw):
    assert lib.ssu_qk_norm_rope(pack("qk", change(QK, kw)), None) == UNSUPPORTED, lib.ssu_last_error()


def test_attention(lib):
    kw = dict(batch=1 << 23, max_pages=8)  # a workgroup of 256 threads for each of 2^24 units
    assert lib.ssu_paged_attention(pack("attn", change(ATTN, kw)), None) == UNSUPPORTED, lib.ssu_last_error()
