"""The gated delta rule and the residual norm on the host: their C structs, what is
refused before the GPU is touched, and the oracle against brute force. No test here
launches a kernel."""
import ctypes
import os
import re
import struct
import subprocess

import numpy as np
import pytest

from .test_seq_host import BF16, F16, F32, I32, I64, INVALID, LINEAR, LINEAR_BAD, MISALIGNED, NONE, OK, ROOT, UNSUPPORTED, VIEW, change, \
    flat, view

E4M3 = 5
DELTA_LAYOUT, NORM_LAYOUT = struct.Struct("6i2qfi" + VIEW * 9 + "Qq"), struct.Struct("q3if" + VIEW * 5)
DELTA = {("normalize" if k == "reserved" else k): v for k, v in LINEAR.items()}
NORM = dict(ntokens=3, width=256, group=0, device=-1, eps=1e-6, x=view(BF16, 256, 1), residual=view(F32, 256, 1), weight=view(BF16, 1),
            out=view(BF16, 256, 1), scales=NONE)


def eight():
    return {"out": view(E4M3, 256, 1), "scales": view(F32, 2, 1)}


def pack(layout, d):
    out = []
    for v in d.values():
        out.extend(flat(v) if isinstance(v, dict) else (v,))
    return layout.pack(*out)


@pytest.fixture(scope="module")
def ssu():
    import selective_state_update_amd as m

    return m


@pytest.fixture(scope="module")
def lib(ssu):
    lib = ctypes.CDLL(ssu.library_path())
    for name in ("ssu_gated_delta_rule", "ssu_gated_delta_rule_step", "ssu_add_rms_norm"):
        getattr(lib, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.ssu_gated_delta_rule_workspace.argtypes = [ctypes.c_void_p]
    lib.ssu_gated_delta_rule_workspace.restype = ctypes.c_int64
    lib.ssu_last_error.restype = ctypes.c_char_p
    return lib


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) { printf("%zu %zu %zu %zu %d\\n", '
                   "sizeof(ssu_delta_args), sizeof(ssu_norm_args), offsetof(ssu_delta_args, workspace), offsetof(ssu_norm_args, x), "
                   "SSU_E4M3); return 0; }\n")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(rocm, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [DELTA_LAYOUT.size, NORM_LAYOUT.size, DELTA_LAYOUT.size - 16, 24, E4M3]


def test_field_order_matches_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssu.h")).read(), flags=re.S)
    for name, want in (("ssu_delta_args", DELTA), ("ssu_norm_args", NORM)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        fields = re.findall(r"(\w+)\s*(?=[,;])", body)
        short = {"cu_seqlens": "cu", "log_decay": "decay", "workspace": "ws", "workspace_bytes": "ws_bytes"}
        assert [short.get(f, f) for f in fields] == list(want)


@pytest.mark.parametrize("kw,code", [(kw, code) for kw, code in LINEAR_BAD if "reserved" not in kw]
                         + [(dict(normalize=2), INVALID), (dict(normalize=-1), INVALID), (dict(ws=0), INVALID),
                            (dict(ws_bytes=1000), INVALID), (dict(ws=0x20008), MISALIGNED), ({"q.0": 1 << 24}, UNSUPPORTED)])
def test_delta_refusals(lib, kw, code):
    assert lib.ssu_gated_delta_rule(pack(DELTA_LAYOUT, change(DELTA, kw)), None) == code, lib.ssu_last_error()
    step = change(DELTA, {"cu": NONE, "ws": 0, "ws_bytes": 0, "batch": 10, **kw})
    if not {"batch", "ntokens", "ws", "ws_bytes", "q.0"} & set(kw):
        assert lib.ssu_gated_delta_rule_step(pack(DELTA_LAYOUT, step), None) == code
    assert lib.ssu_last_error()


def test_delta_nothing_to_do(lib):
    assert lib.ssu_gated_delta_rule(pack(DELTA_LAYOUT, change(DELTA, dict(batch=0))), None) == OK
    assert lib.ssu_gated_delta_rule(pack(DELTA_LAYOUT, change(DELTA, dict(ntokens=0, ws=0))), None) == OK
    assert lib.ssu_gated_delta_rule_step(pack(DELTA_LAYOUT, change(DELTA, {"batch": 0, "ntokens": 0, "cu": NONE, "ws": 0, "ws_bytes": 0})),
                                         None) == OK
    assert lib.ssu_gated_delta_rule_step(pack(DELTA_LAYOUT, DELTA), None) == INVALID  # (prompts are not steps)
    assert lib.ssu_gated_delta_rule(None, None) == INVALID and lib.ssu_gated_delta_rule_step(None, None) == INVALID


def test_delta_workspace(ssu, lib):
    for batch, T, H, P, N, G in ((1, 5000, 16, 64, 128, 1), (4, 37, 32, 128, 256, 4), (3, 9000, 5, 80, 16, 5)):
        want = lib.ssu_gated_delta_rule_workspace(pack(DELTA_LAYOUT, change(DELTA, dict(batch=batch, ntokens=T, nheads=H, headdim=P, dstate=N,
                                                                                        ngroups=G))))
        assert want >= 8192 * H * ((T + 31) // 32) and ssu.gated_delta_rule_workspace(batch, T, H, P, N, G) == want
    assert ssu.gated_delta_rule_workspace(0, 0, 1, 16, 16) == 0
    with pytest.raises(ValueError, match="headdim 24"):
        ssu.gated_delta_rule_workspace(1, 100, 4, 24, 64)
    assert lib.ssu_gated_delta_rule_workspace(None) == -1


@pytest.mark.parametrize("kw", [dict(batch=1 << 22, nheads=16, headdim=256, dstate=128), dict(batch=1 << 20, nheads=1, headdim=256, dstate=256),
                                dict(batch=1 << 24, nheads=4, headdim=16, dstate=16)])
def test_delta_step_launches(lib, kw):
    P, N, H = kw["headdim"], kw["dstate"], kw["nheads"]
    d = change(DELTA, {"cu": NONE, "ws": 0, "ws_bytes": 0, "ntokens": kw["batch"], "ngroups": 1, "state": view(F32, H * P * N, P * N, N, 1),
                       "q": view(BF16, N, N, 1), "k": view(BF16, N, N, 1), "v": view(BF16, H * P, P, 1), "out": view(BF16, H * P, P, 1),
                       "decay": view(F32, H, 1), "beta": view(F32, H, 1), **kw})
    assert lib.ssu_gated_delta_rule_step(pack(DELTA_LAYOUT, d), None) == UNSUPPORTED, lib.ssu_last_error()


def test_delta_prompt_launches(lib):
    for kw in (dict(batch=1 << 24, ntokens=1 << 20), dict(batch=1, ntokens=0x7fff0000, nheads=1, ngroups=1)):
        d = change(DELTA, {**kw, "ws_bytes": 1 << 62})
        code = lib.ssu_gated_delta_rule(pack(DELTA_LAYOUT, d), None)
        assert code == UNSUPPORTED, lib.ssu_last_error()


NORM_BAD = [
    (dict(ntokens=-1), INVALID), (dict(width=0), INVALID), (dict(width=32769), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(group=32), INVALID), (dict(group=-1), INVALID),
    ({"scales": view(F32, 2, 1)}, INVALID), ({**eight(), "group": 48}, INVALID), ({**eight(), "group": 16}, UNSUPPORTED),
    ({**eight(), "group": 512, "width": 1024}, UNSUPPORTED), ({**eight(), "scales": NONE}, INVALID), ({**eight(), "scales.0": 0}, INVALID),
    ({**eight(), "scales.1": 0, "group": 128}, INVALID), ({**eight(), "scales.ptr": 0x10002}, MISALIGNED), ({**eight(), "scales.dtype": BF16}, INVALID),
    ({"x.ptr": 0}, INVALID), ({"out.ptr": 0}, INVALID), ({"x.dtype": F32}, INVALID), ({"x.dtype": E4M3}, INVALID), ({"residual.dtype": F16}, INVALID),
    ({"weight.dtype": F16}, INVALID), ({"out.dtype": F32}, INVALID), ({"x.reserved": 1}, INVALID), ({"x.0": -1}, INVALID),
    ({"residual.0": 0}, INVALID), ({"out.0": 0}, INVALID), ({"x.1": 2}, UNSUPPORTED), ({"residual.1": 0}, UNSUPPORTED),
    ({"out.1": 2}, UNSUPPORTED), ({"weight.0": 2}, UNSUPPORTED), ({"x.ptr": 0x10001}, MISALIGNED), ({"residual.ptr": 0x10002}, MISALIGNED),
    (dict(ntokens=1 << 40), UNSUPPORTED), (dict(ntokens=1 << 25, width=1024), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", NORM_BAD)
def test_norm_refusals(lib, kw, code):
    assert lib.ssu_add_rms_norm(pack(NORM_LAYOUT, change(NORM, kw)), None) == code, lib.ssu_last_error()
    assert lib.ssu_last_error()


def test_norm_nothing_to_do(lib):
    assert lib.ssu_add_rms_norm(pack(NORM_LAYOUT, change(NORM, {"ntokens": 0, "x.ptr": 0, "out.ptr": 0})), None) == OK
    assert lib.ssu_add_rms_norm(None, None) == INVALID


def test_python_wants_the_gpu(ssu):
    import torch

    z = torch.zeros
    with pytest.raises(ValueError):
        ssu.gated_delta_rule(z(1, 1, 16, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1), None, z(2), z(1))
    with pytest.raises(ValueError):
        ssu.gated_delta_rule_step(z(1, 1, 16, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1), None, z(1))
    with pytest.raises(ValueError):
        ssu.add_rms_norm(z(1, 16))


def test_oracles_agree_with_brute_force():
    """tests/delta_ref.py itself: the rule as products of whole matrices, a reflection's fixed points, and bounds that
    hold what fp32 does."""
    from . import delta_ref

    rng = np.random.default_rng(1)
    T, H, P, N = 40, 2, 3, 8
    q, k, v, S0 = rng.normal(size=(T, 1, N)), rng.normal(size=(T, 1, N)), rng.normal(size=(T, H, P)), rng.normal(size=(2, H, P, N))
    g, beta = -rng.random((T, H)), rng.random((T, H))
    for norm in (False, True):
        kk, qq = ((x / np.sqrt((x ** 2).sum(-1, keepdims=True) + 1e-6) if norm else 0.4 * x) for x in (k, q))
        r = delta_ref.gated_delta(S0, q if norm else qq, k if norm else kk, v, g, [0, T], [1], beta, 0.5, norm)
        one = delta_ref.gated_delta(S0, q if norm else qq, k if norm else kk, v, g, [0, T], [1], beta, 0.5, norm, chunk=1)
        low = S0.astype(np.float32)
        for h in range(H):
            S = S0[1, h]
            s = low[1, h]
            for t in range(T):
                M = np.exp(g[t, h]) * (np.eye(N) - beta[t, h] * np.outer(kk[t, 0], kk[t, 0]))
                S = S @ M + beta[t, h] * np.outer(v[t, h], kk[t, 0])
                np.testing.assert_allclose(r["out"][t, h], 0.5 * S @ qq[t, 0], rtol=1e-10, atol=1e-12)
                f = np.float32
                s = s * f(np.exp(g[t, h]))
                s = s + np.outer(f(beta[t, h]) * (v[t, h].astype(f) - s @ kk[t, 0].astype(f)), kk[t, 0].astype(f)).astype(f)
            np.testing.assert_allclose(r["state"][1, h], S, rtol=1e-10, atol=1e-12)
            assert (np.abs(s - S) <= one["state_tol"][1, h]).all() and (np.abs(s - S) <= r["state_tol"][1, h]).all()
        assert np.array_equal(r["state"][0], S0[0])
        # the bounds tell bf16 (2^-9 of values of order 1) from fp32
        assert r["state_tol"][1].max() < 2.0 ** -12
