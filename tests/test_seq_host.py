"""The sequence operators' C ABI on the host: bad arguments are refused before the
GPU is touched. The structs are packed here as include/ssu.h declares them.

No test here launches a kernel: every call carries an invalid field or nothing
to do. The pointer values are never dereferenced on the host."""
import ctypes
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
F32, BF16, I32, I64, F16 = range(5)


VIEW = "Qii4q"  # ptr, dtype, reserved, strides
LAYOUTS = {"linear": struct.Struct("6i2qfi" + VIEW * 9 + "Qq"), "qk": struct.Struct("q6ifi2q" + VIEW * 12),
           "attn": struct.Struct("6i2qfi" + VIEW * 7 + "Qq")}


@pytest.fixture(scope="module")
def ssu():
    import selective_state_update_amd as m

    return m


@pytest.fixture(scope="module")
def lib(ssu):
    lib = ctypes.CDLL(ssu.library_path())
    for name in ("ssu_linear_attention", "ssu_linear_attention_step", "ssu_qk_norm_rope", "ssu_paged_attention"):
        getattr(lib, name).argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    for name in ("ssu_linear_attention_workspace", "ssu_paged_attention_workspace"):
        getattr(lib, name).argtypes = [ctypes.c_void_p]
        getattr(lib, name).restype = ctypes.c_int64
    lib.ssu_last_error.restype = ctypes.c_char_p
    return lib


def view(dtype, *strides, ptr=0x10000, reserved=0):
    return dict(ptr=ptr, dtype=dtype, reserved=reserved, strides=tuple(strides) + (0,) * (4 - len(strides)))


NONE = view(0, ptr=0)


def flat(v):
    return (v["ptr"], v["dtype"], v["reserved"]) + v["strides"]


def change(d, kw):
    """`d` with fields replaced; "q.dtype" names a field of view q, "q.2" a stride."""
    d = {k: dict(v) if isinstance(v, dict) else v for k, v in d.items()}
    for name, value in kw.items():
        head, _, field = name.partition(".")
        if not field:
            d[head] = value
        elif field.isdigit():
            s = list(d[head]["strides"])
            s[int(field)] = value
            d[head]["strides"] = tuple(s)
        else:
            d[head][field] = value
    return d


LINEAR = dict(batch=2, nheads=4, headdim=64, dstate=128, ngroups=2, device=-1, ntokens=10, pool_slots=5, scale=1.0, reserved=0,
              state=view(F32, 32768, 8192, 128, 1), idx=view(I32, 1), cu=view(I32, 1), q=view(BF16, 512, 128, 1),
              k=view(BF16, 512, 128, 1), v=view(BF16, 256, 64, 1), decay=view(F32, 4, 1), beta=view(F32, 4, 1),
              out=view(BF16, 256, 64, 1), ws=0x20000, ws_bytes=1 << 40)
QK = dict(ntokens=3, nq=4, nk=2, headdim=64, rot=64, interleaved=0, device=-1, eps=1e-6, page_size=16, max_pos=100, num_pages=8,
          q=view(BF16, 256, 64, 1), k=view(BF16, 128, 64, 1), q_weight=view(BF16, 1), k_weight=view(F32, 1),
          positions=view(I64, 1), cos_sin=view(F32, 64, 1), q_out=view(BF16, 256, 64, 1), k_out=view(BF16, 128, 64, 1),
          v=view(BF16, 128, 64, 1), k_cache=view(BF16, 2048, 128, 64, 1), v_cache=view(BF16, 2048, 128, 64, 1), slots=view(I64, 1))
ATTN = dict(batch=2, nq=4, nk=2, headdim=64, page_size=16, device=-1, num_pages=8, max_pages=100, scale=0.1, reserved=0,
            q=view(BF16, 256, 64, 1), k_cache=view(BF16, 2048, 128, 64, 1), v_cache=view(BF16, 2048, 128, 64, 1),
            table=view(I32, 4, 1), lens=view(I32, 1), out=view(BF16, 256, 64, 1), lse=view(F32, 4, 1), ws=0x20000, ws_bytes=1 << 40)


def pack(layout, d):
    out = []
    for v in d.values():
        out.extend(flat(v) if isinstance(v, dict) else (v,))
    return LAYOUTS[layout].pack(*out)


def test_struct_layouts_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ssu.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu\\n", '
                   "sizeof(ssu_linear_args), sizeof(ssu_qk_args), sizeof(ssu_attn_args), offsetof(ssu_linear_args, state), "
                   "offsetof(ssu_qk_args, q), offsetof(ssu_attn_args, workspace)); return 0; }\n")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = tmp_path / "sizes"
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(rocm, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [LAYOUTS["linear"].size, LAYOUTS["qk"].size, LAYOUTS["attn"].size, 48, 56, LAYOUTS["attn"].size - 16]


def test_field_order_matches_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssu.h")).read(), flags=re.S)
    for name, want in (("ssu_linear_args", LINEAR), ("ssu_qk_args", QK), ("ssu_attn_args", ATTN)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % name, text, flags=re.S).group(1)
        fields = re.findall(r"(\w+)\s*(?=[,;])", body)
        short = {"cu_seqlens": "cu", "log_decay": "decay", "block_table": "table", "seq_lens": "lens", "workspace": "ws",
                 "workspace_bytes": "ws_bytes"}
        assert [short.get(f, f) for f in fields] == list(want)


LINEAR_BAD = [
    (dict(batch=-1), INVALID), (dict(ntokens=-1), INVALID), (dict(pool_slots=-1), INVALID), (dict(nheads=0), INVALID),
    (dict(ngroups=3), INVALID), (dict(ngroups=0), INVALID), (dict(reserved=1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID),
    (dict(headdim=8), UNSUPPORTED), (dict(headdim=24), UNSUPPORTED), (dict(headdim=272), UNSUPPORTED),
    (dict(dstate=48), UNSUPPORTED), (dict(dstate=512), UNSUPPORTED), (dict(ntokens=1 << 33), UNSUPPORTED),
    (dict(batch=1 << 30, nheads=4), UNSUPPORTED),
    ({"state.ptr": 0}, INVALID), ({"idx.ptr": 0}, INVALID), ({"q.ptr": 0}, INVALID), ({"k.ptr": 0}, INVALID),
    ({"v.ptr": 0}, INVALID), ({"decay.ptr": 0}, INVALID), ({"out.ptr": 0}, INVALID),
    ({"state.dtype": BF16}, INVALID), ({"idx.dtype": F32}, INVALID), ({"q.dtype": F16}, INVALID), ({"v.dtype": F32}, INVALID),
    ({"decay.dtype": BF16}, INVALID), ({"beta.dtype": I32}, INVALID), ({"out.dtype": F32}, INVALID),
    ({"q.reserved": 1}, INVALID), ({"v.0": -256}, INVALID), ({"decay.1": -1}, INVALID), ({"out.0": 0}, INVALID),
    ({"state.2": 0}, INVALID),
    ({"state.3": 2}, UNSUPPORTED), ({"q.2": 2}, UNSUPPORTED), ({"k.2": 0}, UNSUPPORTED), ({"v.2": 2}, UNSUPPORTED),
    ({"out.2": 2}, UNSUPPORTED), ({"idx.0": 2}, UNSUPPORTED),
    ({"state.ptr": 0x10004}, MISALIGNED), ({"state.2": 130}, MISALIGNED), ({"q.ptr": 0x10001}, MISALIGNED),
    ({"beta.ptr": 0x10002}, MISALIGNED), ({"idx.ptr": 0x10004, "idx.dtype": I64}, MISALIGNED),
]


@pytest.mark.parametrize("kw,code", LINEAR_BAD)
def test_linear_refusals(lib, kw, code):
    prompt = change(LINEAR, kw)
    assert lib.ssu_linear_attention(pack("linear", prompt), None) == code, lib.ssu_last_error()
    assert lib.ssu_last_error()
    step = change(LINEAR, {"cu": NONE, "ws": 0, "ws_bytes": 0, "batch": 10, **kw})
    if "batch" not in kw and "ntokens" not in kw:
        assert lib.ssu_linear_attention_step(pack("linear", step), None) == code


@pytest.mark.parametrize("kw,code", [({"cu.ptr": 0}, INVALID), ({"cu.dtype": I64}, INVALID), ({"cu.0": 2}, UNSUPPORTED),
                                     ({"v.0": 1 << 24}, UNSUPPORTED), ({"out.0": 1 << 24}, UNSUPPORTED),
                                     ({"cu.ptr": 0x10002}, MISALIGNED)])
def test_linear_prompt_refusals(lib, kw, code):
    assert lib.ssu_linear_attention(pack("linear", change(LINEAR, kw)), None) == code


@pytest.mark.parametrize("kw", [dict(batch=9), dict(cu=view(I32, 1)), dict(ws=0x20000)])
def test_linear_step_refusals(lib, kw):
    d = change(LINEAR, {"cu": NONE, "ws": 0, "ws_bytes": 0, "batch": 10, **kw})
    assert lib.ssu_linear_attention_step(pack("linear", d), None) == INVALID


def test_linear_nothing_to_do(lib):
    assert lib.ssu_linear_attention(pack("linear", change(LINEAR, dict(batch=0))), None) == OK
    empty = {k: 0 for k in ("q.ptr", "k.ptr", "v.ptr", "decay.ptr", "out.ptr")}
    assert lib.ssu_linear_attention(pack("linear", change(LINEAR, dict(ntokens=0, **empty))), None) == OK
    step = change(LINEAR, {"cu": NONE, "ws": 0, "ws_bytes": 0, "batch": 0, "ntokens": 0})
    assert lib.ssu_linear_attention_step(pack("linear", step), None) == OK
    for fn in (lib.ssu_linear_attention, lib.ssu_linear_attention_step, lib.ssu_qk_norm_rope,
               lib.ssu_paged_attention):
        assert fn(None, None) == INVALID
    assert lib.ssu_linear_attention_workspace(None) == lib.ssu_paged_attention_workspace(None) == -1


QK_BAD = [
    (dict(ntokens=-1), INVALID), (dict(nq=-1), INVALID), (dict(nk=-1), INVALID), (dict(max_pos=-1), INVALID),
    (dict(num_pages=-1), INVALID), (dict(headdim=0), INVALID), (dict(rot=3), INVALID), (dict(rot=66), INVALID),
    (dict(rot=-2), INVALID), (dict(interleaved=2), INVALID), (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(page_size=0), INVALID), (dict(num_pages=1 << 62), INVALID), (dict(headdim=514), UNSUPPORTED),
    (dict(ntokens=1 << 40), UNSUPPORTED),
    ({"q.ptr": 0}, INVALID), ({"k.ptr": 0}, INVALID), ({"q_out.ptr": 0}, INVALID), ({"positions.ptr": 0}, INVALID),
    ({"cos_sin.ptr": 0}, INVALID), ({"v.ptr": 0}, INVALID), ({"k_cache.ptr": 0}, INVALID), ({"v_cache.ptr": 0}, INVALID),
    ({"slots.ptr": 0}, INVALID), ({"q.dtype": F32}, INVALID), ({"k.dtype": F16}, INVALID), ({"q_out.dtype": F16}, INVALID),
    ({"q_weight.dtype": F16}, INVALID), ({"k_cache.dtype": F16}, INVALID), ({"positions.dtype": F32}, INVALID),
    ({"slots.dtype": BF16}, INVALID), ({"q.0": -1}, INVALID), ({"k_out.0": 0}, INVALID), ({"v_cache.1": 0}, INVALID),
    ({"cos_sin.reserved": 5}, INVALID),
    ({"q.2": 2}, UNSUPPORTED), ({"v.2": 2}, UNSUPPORTED), ({"k_cache.3": 2}, UNSUPPORTED), ({"cos_sin.1": 2}, UNSUPPORTED),
    ({"positions.0": 2}, UNSUPPORTED), ({"slots.0": 0}, UNSUPPORTED), ({"k_weight.0": 2}, UNSUPPORTED),
    ({"q.ptr": 0x10001}, MISALIGNED), ({"v_cache.ptr": 0x10001}, MISALIGNED), ({"cos_sin.ptr": 0x10002}, MISALIGNED),
    ({"slots.ptr": 0x10004}, MISALIGNED), ({"k_weight.ptr": 0x10002}, MISALIGNED),
]


@pytest.mark.parametrize("kw,code", QK_BAD)
def test_qk_refusals(lib, kw, code):
    assert lib.ssu_qk_norm_rope(pack("qk", change(QK, kw)), None) == code, lib.ssu_last_error()


def test_qk_nothing_to_do(lib):
    for kw in (dict(ntokens=0), dict(nq=0, nk=0), dict(max_pos=0)):
        assert lib.ssu_qk_norm_rope(pack("qk", change(QK, kw)), None) == OK


ATTN_BAD = [
    (dict(batch=-1), INVALID), (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(page_size=0), INVALID),
    (dict(nk=0), INVALID), (dict(nq=3), INVALID), (dict(nq=0), INVALID), (dict(reserved=1), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=3e38), INVALID), (dict(headdim=96), UNSUPPORTED), (dict(headdim=512), UNSUPPORTED),
    (dict(batch=1 << 30), UNSUPPORTED),
    ({"q.ptr": 0}, INVALID), ({"k_cache.ptr": 0}, INVALID), ({"v_cache.ptr": 0}, INVALID), ({"table.ptr": 0}, INVALID),
    ({"lens.ptr": 0}, INVALID), ({"out.ptr": 0}, INVALID), ({"q.dtype": F32}, INVALID), ({"k_cache.dtype": F16}, INVALID),
    ({"v_cache.dtype": F16}, INVALID), ({"out.dtype": F32}, INVALID), ({"table.dtype": I64}, INVALID),
    ({"lens.dtype": I64}, INVALID), ({"lse.dtype": BF16}, INVALID), ({"out.1": 0}, INVALID), ({"lse.0": 0}, INVALID),
    ({"q.0": -1}, INVALID), ({"lse.reserved": 1}, INVALID),
    ({"q.2": 2}, UNSUPPORTED), ({"out.2": 2}, UNSUPPORTED), ({"k_cache.3": 0}, UNSUPPORTED), ({"table.1": 2}, UNSUPPORTED),
    ({"lens.0": 2}, UNSUPPORTED), ({"q.ptr": 0x10001}, MISALIGNED), ({"table.ptr": 0x10002}, MISALIGNED),
    ({"lse.ptr": 0x10002}, MISALIGNED), (dict(ws=0), INVALID), (dict(ws_bytes=64), INVALID), (dict(ws=0x20008), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", ATTN_BAD)
def test_attention_refusals(lib, kw, code):
    assert lib.ssu_paged_attention(pack("attn", change(ATTN, kw)), None) == code, lib.ssu_last_error()


def test_attention_nothing_to_do(lib):
    assert lib.ssu_paged_attention(pack("attn", change(ATTN, dict(batch=0))), None) == OK


def test_attention_workspace(lib):
    """None for short caches: a workgroup takes each unit."""
    def need(**kw):
        return lib.ssu_paged_attention_workspace(pack("attn", change(ATTN, kw)))

    assert need(max_pages=32) == 0 and need(max_pages=33) > 0
    assert need(max_pages=16, headdim=256) == 0 and need(max_pages=17, headdim=256) > 0
    assert need(max_pages=33, batch=127) > 0 and need(max_pages=33, batch=128) == 0  # two units a request
    assert need(max_pages=128, batch=128) == 0 and need(max_pages=129, batch=128) > 0
    assert need(max_pages=128, batch=128, headdim=256) == 0 and need(max_pages=129, batch=128, headdim=256) > 0
    assert need(max_pages=64, batch=129, headdim=256) == 0 and need(max_pages=65, batch=129, headdim=256) > 0
    assert need(max_pages=0) == 0 and need(nk=0) == -1


def test_stream_of_another_device():
    """Refused: the call would run on the operands' own current stream instead."""
    import types

    import torch

    import selective_state_update_amd as ssu

    operand = types.SimpleNamespace(device=torch.device("cuda", 0))
    stream = types.SimpleNamespace(cuda_stream=0, device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:1"):
        ssu._on(stream, operand)


def test_python_wants_the_gpu(ssu):
    import torch

    z = torch.zeros
    with pytest.raises(ValueError):
        ssu.linear_attention(z(1, 1, 16, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1), z(2), z(1))
    with pytest.raises(ValueError):
        ssu.linear_attention_step(z(1, 1, 16, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1, 16), z(1, 1), z(1))
    with pytest.raises(ValueError):
        ssu.qk_norm_rope(z(1, 1, 8), z(1, 1, 8), z(1), z(4, 8))
    with pytest.raises(ValueError):
        ssu.paged_attention(z(1, 1, 64), z(1, 1, 1, 64), z(1, 1, 1, 64), z(1, 1), z(1))


def test_oracles_agree_with_brute_force():
    """tests/seq_ref.py itself: linear attention by its sum over pairs of tokens, the rotation by complex
    numbers, attention by torch's softmax."""
    import numpy as np
    import torch

    from . import seq_ref

    rng = np.random.default_rng(1)
    T, H, P, N = 9, 2, 3, 4
    q, k, v = rng.normal(size=(T, 1, N)), rng.normal(size=(T, 1, N)), rng.normal(size=(T, H, P))
    g, beta, S0 = -rng.random((T, H)), rng.random((T, H)), rng.normal(size=(2, H, P, N))
    r = seq_ref.linear_attention(S0, q, k, v, g, [0, T], [1], beta, 0.5)
    L = g.cumsum(0)
    for t in range(T):
        for h in range(H):
            y = np.exp(L[t, h]) * S0[1, h] @ q[t, 0]
            for j in range(t + 1):
                y = y + np.exp(L[t, h] - L[j, h]) * beta[j, h] * (q[t, 0] @ k[j, 0]) * v[j, h]
            np.testing.assert_allclose(r["out"][t, h], 0.5 * y, rtol=1e-12, atol=1e-12)
    assert np.array_equal(r["state"][0], S0[0]) and r["state_tol"][1].min() > 0
    x, pos = rng.normal(size=(2, 1, 8)), [1, 2]
    angle = np.arange(4)[:, None] * np.array([1.0, 0.1])
    y, _ = seq_ref.norm_rope(x, None, pos, np.concatenate([np.cos(angle), np.sin(angle)], 1), 0.0, True, 2.0 ** -8)
    n = x / np.sqrt((x ** 2).mean(-1, keepdims=True))
    for t in range(2):
        z = (n[t, 0, 0:4:2] + 1j * n[t, 0, 1:4:2]) * np.exp(1j * angle[pos[t]])
        np.testing.assert_allclose(y[t, 0], np.concatenate([np.stack([z.real, z.imag], 1).ravel(), n[t, 0, 4:]]), atol=1e-14)
    q, kc, vc = rng.normal(size=(1, 2, 4)), rng.normal(size=(3, 2, 1, 4)), rng.normal(size=(3, 2, 1, 4))
    a = seq_ref.paged_attention(q, kc, vc, np.array([[2, 0]]), np.array([3]), 0.3, 2.0 ** -8)
    K, V = torch.tensor(np.stack([kc[2, 0, 0], kc[2, 1, 0], kc[0, 0, 0]])), torch.tensor(np.stack([vc[2, 0, 0], vc[2, 1, 0], vc[0, 0, 0]]))
    s = torch.tensor(q[0]) @ K.T * 0.3
    np.testing.assert_allclose(a["out"][0], torch.softmax(s, -1) @ V, atol=1e-14)
    np.testing.assert_allclose(a["lse"][0], torch.logsumexp(s, -1), atol=1e-14)
