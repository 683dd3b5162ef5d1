"""The gated delta rule in fp64 from its definition, with bounds of what fp32 and the
prompts' chunks can add, and the residual norm in fp64.

Bounds of the rule, for each row p of a head's state (a vector s over n, 2-norms), in
units of 2^-24, chunks of C tokens (steps: C = 1). L, X: the chunk's triangle and the
inverse of 1 + L; m_i = |v_i| + exp(L_i) |s| |k_i| bounds what enters u_i.

  r_i = v_i - exp(L_i) s . k_i: a sum of N products on matrix units (32 a time) or of
      lanes, three pieces of 2^-24, the decay and its difference: (48 + N / 8 + |L_i|) m_i
  u = X r: the sum's roundings 48 (|X| m), and X's own: |X| |L| |X| m, 48 roundings of
      L's entries (a product of N, as above, three factors) and of the substitution
  s behind the chunk: what was off before it, carried by the decay and by
      prod_j max(1, |1 - beta_j |k_j|^2|), and sum_j |late_j| |k_j| (du_j + 48 |u_j|) + 48 exp(L_C) |s|
  out_i: 2^-8 of itself; the state's error through q and through u; the pieces of the
      state, of the weights and of u in two (2^-16 each); sums as above.
"""
from __future__ import annotations

import numpy as np

from .seq_ref import EPS32

FAINT = 1e-6
CHUNK = 32


def gated_delta(state, q, k, v, log_decay, cu, idx, beta=None, scale=1.0, normalize=False, chunk=CHUNK):
    """state [pool,H,P,N], q, k [T,G,N], v [T,H,P], log_decay [T,H] or [H], beta
    [T,H] or None (fp64 arrays, finite). Returns a dict as seq_ref.linear_attention."""
    T, H, P = v.shape
    N, G = q.shape[2], q.shape[1]
    state = state.copy()
    tol = np.zeros_like(state)
    out, otol = np.full((T, H, P), np.nan), np.zeros((T, H, P))
    if log_decay.ndim == 1:
        log_decay = np.broadcast_to(log_decay, (T, H))
    log_decay = np.maximum(log_decay, -1e4)
    beta = np.ones((T, H)) if beta is None else beta
    if normalize:
        q, k = (x / np.sqrt((x ** 2).sum(-1, keepdims=True) + FAINT) for x in (q, k))
    for b in range(len(idx)):
        if not 0 <= idx[b] < state.shape[0]:
            continue
        for h in range(H):
            S = state[idx[b], h]
            err = np.zeros(P)
            for t0 in range(cu[b], cu[b + 1], chunk):
                t1 = min(t0 + chunk, cu[b + 1])
                K, Q, V = k[t0:t1, h // (H // G)], q[t0:t1, h // (H // G)], v[t0:t1, h]
                B, g = beta[t0:t1, h], log_decay[t0:t1, h]
                C = t1 - t0
                L = np.cumsum(g)
                with np.errstate(over="ignore"):
                    between = np.tril(np.exp(np.minimum(L[:, None] - L[None], 700)))
                low = np.tril((K @ K.T) * between * B[:, None], -1)
                X = np.linalg.inv(np.eye(C) + low)
                kn, qn, sn = np.linalg.norm(K, axis=1), np.linalg.norm(Q, axis=1), np.linalg.norm(S, axis=1)
                grow = np.exp(L)
                # the recurrence itself
                s, U = S.copy(), np.zeros((C, P))
                for i in range(C):
                    s = s * np.exp(g[i])
                    U[i] = B[i] * (V[i] - s @ K[i])
                    s = s + U[i][:, None] * K[i][None]
                    out[t0 + i, h] = scale * (s @ Q[i])
                # bounds
                aX, steps = np.abs(X) * np.abs(B)[None], (48 + N / 8 + np.abs(L))[:, None]
                m = np.abs(V) + grow[:, None] * kn[:, None] * sn[None]
                du = EPS32 * (aX @ (steps * m) + 48 * (aX @ m) + np.abs(X) @ ((48 + N / 8) * np.abs(low)) @ (aX @ m))
                through = aX @ (grow[:, None] * kn[:, None] * err[None])  # of what was off before, in u
                weight = np.abs(scale) * np.abs(np.tril((Q @ K.T) * between))
                # the products of q and k that cancel are off by their own sums
                wsize = np.abs(scale) * np.tril((np.abs(Q) @ np.abs(K).T) * between)
                otol[t0:t1, h] = (2.0 ** -8 * np.abs(out[t0:t1, h])
                                  + np.abs(scale) * grow[:, None] * qn[:, None] * (err + (2.0 ** -16 + steps * EPS32) * sn[None])
                                  + weight @ (du + through + (2.0 ** -15 + 64 * EPS32) * np.abs(U))
                                  + (64 + N / 8) * EPS32 * (wsize @ np.abs(U)))
                late = np.exp(L[-1] - L)
                carried = grow[-1] * np.prod(np.maximum(1.0, np.abs(1 - B * kn ** 2)))
                err = carried * err + (late * kn) @ (du + (48 + np.abs(L[-1] - L))[:, None] * EPS32 * np.abs(U)) \
                    + (48 + np.abs(L[-1])) * EPS32 * grow[-1] * sn
                S = s
            state[idx[b], h] = S
            tol[idx[b], h] = err[:, None] + 1e-37
    return dict(state=state, out=out, state_tol=tol, out_tol=otol + 1e-30)


def add_rms_norm(x, residual, weight, eps):
    """Returns s (x + residual) and y, fp64 [T, D]."""
    s = x if residual is None else x + residual
    y = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + eps)
    return s, y if weight is None else y * weight
