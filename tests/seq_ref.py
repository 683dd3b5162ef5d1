"""The sequence operators (linear attention, norm and rotation, paged attention)
in fp64 from their definitions, one row at a time, with the magnitudes that
their error bounds are stated in, and the bounds.

A rounding to a type is off by at most half a step, finfo(type).eps / 2 relative
(u below: bf16 2^-8, fp16 2^-11); fp32 by 2^-24. A value split into a 16-bit pair
(rounded value and rounded remainder) is off by at most u^2.
"""
from __future__ import annotations

import numpy as np
import torch

EPS32 = 2.0 ** -24


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def linear_attention(state, q, k, v, log_decay, cu, idx, beta=None, scale=1.0):
    """state [pool,H,P,N], q, k [T,G,N], v [T,H,P], log_decay [T,H] or [H], beta
    [T,H] or None (fp64 arrays). Returns a dict: `state` and `out` (nan in rows
    that are not written), and their bounds `state_tol`, `out_tol`.

    A bounds |S| (the recurrence on magnitudes). E collects what each fp32
    step can add: E_t = a (E_{t-1} + (1 + |log_decay|) A_{t-1}) + A_t, one
    2^-24 of it for each rounding a token meets. A token meets at most 64 of
    them (the partial sums of a chunk's products, the decay's and the gain's
    factors). out carries the state's error through q, the split of the state
    and of the weights into bf16 pairs (2^-16 each, of sum |q| A), a sum over N
    and the output's rounding."""
    T, H, P = v.shape
    N, G = q.shape[2], q.shape[1]
    state = state.copy()
    tol = np.zeros_like(state)
    out, otol = np.full((T, H, P), np.nan), np.zeros((T, H, P))
    if log_decay.ndim == 1:
        log_decay = np.broadcast_to(log_decay, (T, H))
    beta = np.ones((T, H)) if beta is None else beta
    group = np.arange(H) // (H // G)
    for b in range(len(idx)):
        if not 0 <= idx[b] < state.shape[0]:
            continue
        S = state[idx[b]]
        A, E = np.abs(S), np.zeros_like(S)
        for t in range(cu[b], cu[b + 1]):
            g = np.maximum(log_decay[t], -1e4)[:, None, None]
            a = np.exp(g)
            new = beta[t][:, None, None] * v[t][:, :, None] * k[t][group][:, None, :]
            S = S * a + new
            E = a * (E + (1 + np.abs(g)) * A)
            A = a * A + np.abs(new)
            E += A
            qt = q[t][group][:, None, :]
            out[t] = scale * (S * qt).sum(-1)
            otol[t] = 2.0 ** -8 * np.abs(out[t]) + abs(scale) * (
                (2.0 ** -15 + N * EPS32) * (A * np.abs(qt)).sum(-1) + 64 * EPS32 * (E * np.abs(qt)).sum(-1))
        state[idx[b]] = S
        tol[idx[b]] = 64 * EPS32 * E
    return dict(state=state, out=out, state_tol=tol, out_tol=otol + 1e-30)


def norm_rope(x, weight, positions, cos_sin, eps, interleaved, u):
    """x [T, heads, D]; rows of positions outside the table are nan."""
    T, _, D = x.shape
    rot = cos_sin.shape[1]
    y, tol = np.full(x.shape, np.nan), np.zeros(x.shape)
    for t in range(T):
        if not 0 <= positions[t] < cos_sin.shape[0]:
            continue
        c, s = cos_sin[positions[t]][:rot // 2], cos_sin[positions[t]][rot // 2:]
        n = x[t] / np.sqrt((x[t] ** 2).mean(-1, keepdims=True) + eps)
        n = n if weight is None else n * weight
        mag = np.abs(n)
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z, m = n.copy(), mag.copy()
        z[:, a], z[:, b] = n[:, a] * c - n[:, b] * s, n[:, b] * c + n[:, a] * s
        m[:, a] = mag[:, a] * np.abs(c) + mag[:, b] * np.abs(s)
        m[:, b] = mag[:, b] * np.abs(c) + mag[:, a] * np.abs(s)
        y[t] = z
        # a sum of D squares, a root, a division and four products
        tol[t] = u * np.abs(z) + (D + 16) * EPS32 * m
    return y, tol + (2.0 ** -25 if u == 2.0 ** -11 else 1e-38)  # half of the smallest fp16 step below 2^-14


def paged_attention(q, kc, vc, table, lens, scale, u):
    """q [B, Hq, D], caches [pages, page, Hk, D]. Returns dict(out, lse, out_tol,
    lse_tol); nan where nothing is written."""
    B, Hq, D = q.shape
    pages, page, Hk, _ = kc.shape
    out, lse = np.full((B, Hq, D), np.nan), np.full((B, Hq), np.nan)
    otol, ltol = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        if lens[b] < 0:
            continue
        n = min(int(lens[b]), table.shape[1] * page)
        j = np.arange(n)
        pg = table[b][j // page].astype(np.int64)
        ok = (pg >= 0) & (pg < pages)
        pg, off = pg[ok], j[ok] % page
        for h in range(Hq):
            K, V = kc[pg, off, h // (Hq // Hk)], vc[pg, off, h // (Hq // Hk)]
            s = K @ q[b, h] * scale
            if not len(s) or s.max() == -np.inf:
                out[b, h], lse[b, h] = 0.0, -np.inf
                continue
            w = np.exp(s - s.max())
            out[b, h] = w @ V / w.sum()
            lse[b, h] = s.max() + np.log(w.sum())
            # a score: a sum of D products and the scale's; its weight: the
            # exponent's argument (rounded relative to its size) and the power
            size = (np.abs(K) @ np.abs(q[b, h])) * abs(scale)
            delta = (EPS32 * ((D + 8) * size + 4 * np.abs(s - s.max()) + 16)).max()
            # sums over n weights, rescaled as the maximum grows
            sums = 64 * EPS32
            otol[b, h] = u * np.abs(out[b, h]) + (4 * u * u + 2 * delta + 2 * sums) * (w @ np.abs(V)) / w.sum()
            ltol[b, h] = 2 * delta + sums + 4 * EPS32 * abs(lse[b, h])
    return dict(out=out, lse=lse, out_tol=otol + (2.0 ** -25 if u == 2.0 ** -11 else 1e-38), lse_tol=ltol)


def assert_close(got, want, tol, what):
    got = f64(got) if torch.is_tensor(got) else np.asarray(got, dtype=np.float64)
    seen = ~np.isnan(want)
    with np.errstate(invalid="ignore"):  # infinities are compared by themselves
        bad = seen & ~((np.abs(got - want) <= tol) | (got == want))
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        worst = np.nanmax(np.where(seen, np.abs(got - want) / np.maximum(tol, 1e-300), 0))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} values off, first at {i}: {got[i]!r}, expected "
                             f"{want[i]!r} within {np.broadcast_to(tol, want.shape)[i]!r}; worst {worst:.3g} of its bound")
