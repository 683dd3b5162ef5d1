"""Attention behind a shared prefix in fp64 from its definition: one row of keys per
request, the prefix's and then its own, with the bounds of seq_ref.paged_attention and
one rounding of the prefix's weights to 16 bits more (u relative; fp16 weights, scaled
by 2^14, are off by 2^-25 more where they are too small for that)."""
from __future__ import annotations

import numpy as np

from .seq_ref import EPS32


def rows_of(table, n, page, pages):
    j = np.arange(min(max(int(n), 0), len(table) * page))
    pg = table[j // page].astype(np.int64) if len(j) else j
    ok = (pg >= 0) & (pg < pages)
    return pg[ok], j[ok] % page


def shared_prefix_attention(q, kc, vc, prefix, prefix_len, table, lens, scale, u):
    """q [B, Hq, D], caches [pages, page, Hk, D], prefix [pages0], table [B, width].
    Returns dict(out, lse, out_tol, lse_tol); nan where nothing is written."""
    B, Hq, D = q.shape
    pages, page, Hk, _ = kc.shape
    out, lse = np.full((B, Hq, D), np.nan), np.full((B, Hq), np.nan)
    otol, ltol = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    pg0, off0 = rows_of(prefix, prefix_len, page, pages)
    for b in range(B):
        if lens[b] < 0:
            continue
        pg1, off1 = rows_of(table[b], lens[b], page, pages)
        pg, off = np.concatenate((pg0, pg1)), np.concatenate((off0, off1))
        for h in range(Hq):
            K, V = kc[pg, off, h // (Hq // Hk)], vc[pg, off, h // (Hq // Hk)]
            s = K @ q[b, h] * scale
            if not len(s) or s.max() == -np.inf:
                out[b, h], lse[b, h] = 0.0, -np.inf
                continue
            w = np.exp(s - s.max())
            out[b, h] = w @ V / w.sum()
            lse[b, h] = s.max() + np.log(w.sum())
            size = (np.abs(K) @ np.abs(q[b, h])) * abs(scale)
            delta = (EPS32 * ((D + 8) * size + 4 * np.abs(s - s.max()) + 16)).max()
            sums = 64 * EPS32
            small = len(pg0) * 2.0 ** -39 * np.abs(V).max(0) if u == 2.0 ** -11 else 0.0
            otol[b, h] = u * np.abs(out[b, h]) + ((u + 4 * u * u + 2 * delta + 2 * sums) * (w @ np.abs(V)) + small) / w.sum()
            ltol[b, h] = 2 * delta + sums + 4 * EPS32 * abs(lse[b, h])
    return dict(out=out, lse=lse, out_tol=otol + (2.0 ** -25 if u == 2.0 ** -11 else 1e-38), lse_tol=ltol)
