"""Attention over a shared prefix on the host: its C struct, what is refused before the GPU
is touched, and the oracle against brute force. No test here launches a kernel."""
import ctypes
import os
import re
import struct
import subprocess

import numpy as np
import pytest

from .test_seq_host import ATTN, ATTN_BAD, I32, I64, INVALID, MISALIGNED, OK, ROOT, UNSUPPORTED, VIEW, change, flat, view

LAYOUT = struct.Struct("6i2qfi" + VIEW * 7 + "Qq" + VIEW * 2 + "q")
SHARED = {**ATTN, "prefix": view(I32, 1), "prefix_len": view(I32, 1), "prefix_pages": 50}


def pack(d):
    out = []
    for v in d.values():
        out.extend(flat(v) if isinstance(v, dict) else (v,))
    return LAYOUT.pack(*out)


@pytest.fixture(scope="module")
def ssu():
    import selective_state_update_amd as m

    return m


@pytest.fixture(scope="module")
def lib(ssu):
    lib = ctypes.CDLL(ssu.library_path())
    lib.ssu_shared_prefix_attention.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.ssu_shared_prefix_attention_workspace.argtypes = [ctypes.c_void_p]
    lib.ssu_shared_prefix_attention_workspace.restype = ctypes.c_int64
    lib.ssu_last_error.restype = ctypes.c_char_p
    return lib


def test_struct_layout_matches_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) { printf("%zu %zu %zu\\n", '
                   "sizeof(ssu_shared_args), offsetof(ssu_shared_args, prefix_table), offsetof(ssu_shared_args, prefix_pages)); return 0; }\n")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(rocm, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [LAYOUT.size, LAYOUT.size - 8 - 96, LAYOUT.size - 8]
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssu.h")).read(), flags=re.S)
    body = re.search(r"typedef struct ssu_shared_args \{(.*?)\}", text, flags=re.S).group(1)
    assert re.findall(r"(\w+)\s*(?=[,;])", body) == ["attn", "prefix_table", "prefix_len", "prefix_pages"]


@pytest.mark.parametrize("kw,code", ATTN_BAD + [
    (dict(prefix_pages=-1), INVALID), (dict(prefix_pages=1 << 62), INVALID), ({"prefix.ptr": 0}, INVALID), ({"prefix.dtype": I64}, INVALID),
    ({"prefix_len.ptr": 0}, INVALID), ({"prefix_len.dtype": I64}, INVALID), ({"prefix.reserved": 1}, INVALID), ({"prefix.0": -1}, INVALID),
    ({"prefix.0": 2}, UNSUPPORTED), ({"prefix.0": 0}, UNSUPPORTED), ({"prefix.ptr": 0x10002}, MISALIGNED), ({"prefix_len.ptr": 0x10002}, MISALIGNED)])
def test_refusals(lib, kw, code):
    assert lib.ssu_shared_prefix_attention(pack(change(SHARED, kw)), None) == code, lib.ssu_last_error()
    assert lib.ssu_last_error()


def test_nothing_to_do(lib):
    assert lib.ssu_shared_prefix_attention(pack(change(SHARED, dict(batch=0))), None) == OK
    assert lib.ssu_shared_prefix_attention(None, None) == INVALID and lib.ssu_shared_prefix_attention_workspace(None) == -1


def test_launches(lib):
    """A workgroup of 256 threads for each of 2^24 units, of the requests' own tokens and of the prefix's."""
    assert lib.ssu_shared_prefix_attention(pack(change(SHARED, dict(batch=1 << 23, max_pages=8, ws_bytes=1 << 62))), None) == UNSUPPORTED
    assert lib.ssu_last_error()


def test_workspace(ssu, lib):
    for batch, nq, nk, D, page, pages, first in ((1, 16, 2, 128, 16, 100, 40), (64, 32, 8, 128, 64, 128, 500), (3, 8, 1, 64, 1, 300, 0),
                                                 (2, 4, 4, 256, 16, 17, 1 << 40)):
        want = lib.ssu_shared_prefix_attention_workspace(pack(change(SHARED, dict(batch=batch, nq=nq, nk=nk, headdim=D, page_size=page,
                                                                                  max_pages=pages, prefix_pages=first))))
        assert want >= batch * nq * (D + 2) * 4 and ssu.shared_prefix_attention_workspace(batch, nq, nk, D, page, pages, first) == want
        assert want >= ssu.paged_attention_workspace(batch, nq, nk, D, page, pages)
    with pytest.raises(ValueError, match="headdim 96"):
        ssu.shared_prefix_attention_workspace(1, 4, 2, 96, 16, 4, 4)
    with pytest.raises(ValueError, match="prefix_pages"):
        ssu.shared_prefix_attention_workspace(1, 4, 2, 64, 16, 4, -1)


def test_python_wants_the_gpu(ssu):
    import torch

    z = torch.zeros
    with pytest.raises(ValueError):
        ssu.shared_prefix_attention(z(1, 1, 64), z(1, 1, 1, 64), z(1, 1, 1, 64), z(1), z(1), z(1, 1), z(1))


def test_oracle_agrees_with_brute_force():
    import torch

    from . import seq_ref, shared_ref

    rng = np.random.default_rng(1)
    q, kc, vc = rng.normal(size=(2, 2, 4)), rng.normal(size=(4, 2, 1, 4)), rng.normal(size=(4, 2, 1, 4))
    a = shared_ref.shared_prefix_attention(q, kc, vc, np.array([2, 0, 9]), 5, np.array([[1], [3]]), np.array([1, 0]), 0.3, 2.0 ** -8)
    for b, rows in ((0, [(2, 0), (2, 1), (0, 0), (0, 1), (1, 0)]), (1, [(2, 0), (2, 1), (0, 0), (0, 1)])):
        K, V = (torch.tensor(np.stack([x[i, j, 0] for i, j in rows])) for x in (kc, vc))
        s = torch.tensor(q[b]) @ K.T * 0.3
        np.testing.assert_allclose(a["out"][b], torch.softmax(s, -1) @ V, atol=1e-14)
        np.testing.assert_allclose(a["lse"][b], torch.logsumexp(s, -1), atol=1e-14)
    # the prefix as a request's first pages is paged attention
    one = shared_ref.shared_prefix_attention(q, kc, vc, np.array([2, 0]), 4, np.array([[1], [3]]), np.array([2, 1]), 0.3, 2.0 ** -8)
    two = seq_ref.paged_attention(q, kc, vc, np.array([[2, 0, 1], [2, 0, 3]]), np.array([6, 5]), 0.3, 2.0 ** -8)
    np.testing.assert_allclose(one["out"], two["out"], atol=1e-14)
    assert (one["out_tol"] > two["out_tol"]).all()
