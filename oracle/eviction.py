"""Float64 CPU oracle of the cache-eviction calls: attention mass of the cached
tokens, the choice of those that stay, compaction of the paged cache to them.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, written from
the definitions in include/mla.h; nothing here is shared with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from .mla import DEFAULT_THETA, gather_cache, rope


def attention_mass(q_lat, pool, page_table, lens, lse, scale, mass, decay=1.0, mass_lens=None):
    """The updated mass [B, width] after one step.

    Query token i of sequence b sits at cache index lens[b] - nq + i and sees the
    indices up to its own; its weight for key n and head h is exp(scale q . row_n - lse).
    q_lat [B, nq, H, R], lse [B, nq, H]; rows with lse = -inf saw no key.
    """
    q_lat = np.asarray(q_lat, dtype=np.float64)
    lse = np.asarray(lse, dtype=np.float64)
    B, nq = q_lat.shape[:2]
    out = np.array(mass, dtype=np.float64)
    for b in range(B):
        n = int(lens[b])
        rows = np.asarray(gather_cache(pool, page_table[b], n), dtype=np.float64)
        w = np.zeros(n)
        for i in range(nq):
            seen = n - nq + i + 1
            s = scale * (rows[:seen] @ q_lat[b, i].T)            # [seen, H]
            some = lse[b, i] > -np.inf
            w[:seen] += np.exp(s[:, some] - lse[b, i, some]).sum(axis=1)
        old = n - nq if mass_lens is None else int(mass_lens[b])
        old = max(0, min(old, n))
        if decay != 0:
            w[:old] += decay * out[b, :old]
        out[b, :n] = w
    return out


def select(mass, lens, budgets, n_sink, n_recent):
    """Per sequence, the ascending cache indices that stay: first n_sink, last
    n_recent, then the largest masses (ties: lowest index; NaN above +inf)."""
    kept = []
    for b in range(len(lens)):
        n = int(lens[b])
        k = min(n, int(budgets[b]))
        s = min(n_sink, k)
        r = min(n_recent, k - s)
        m = np.asarray(mass[b][:n], dtype=np.float64)
        if k == n:
            kept.append(np.arange(n))
            continue
        middle = list(range(s, n - r))
        # Python's sort is stable: equal masses keep their index order
        middle.sort(key=lambda j: (not np.isnan(m[j]), -m[j] if not np.isnan(m[j]) else 0.0))
        kept.append(np.array(sorted(list(range(s)) + middle[: k - s - r] + list(range(n - r, n))), dtype=np.int64))
    return kept


def compact(pool, page_table, kept, d_c, mass=None, rerotate=True, theta=DEFAULT_THETA):
    """(pool, mass) after row j of sequence b became [c_n || RoPE(k_n^R, j - n)],
    n = kept[b][j]; rows that stay where they are keep their values exactly."""
    before = np.asarray(pool, dtype=np.float64)
    after = before.copy()
    page = before.shape[1]
    new_mass = None if mass is None else np.array(mass, dtype=np.float64)
    for b, idx in enumerate(kept):
        idx = np.asarray(idx, dtype=np.int64)
        if len(idx) == 0:
            continue
        j = np.arange(len(idx))
        rows = before[page_table[b][idx // page], idx % page].copy()
        if rerotate:
            rows[:, d_c:] = rope(rows[:, d_c:], j - idx, theta)
        after[page_table[b][j // page], j % page] = rows
        if mass is not None:
            new_mass[b, : len(idx)] = np.asarray(mass, dtype=np.float64)[b, idx]
    return after, new_mass
