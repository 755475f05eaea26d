"""fp64 oracle of a step of speculative decoding: tree attention, the verdict, the rows that stand.

TEST INFRASTRUCTURE ONLY, like the decode oracle: plain numpy arrays in and out, no code
shared with the CUDA path.  Every function is pinned by ``tests/test_oracle_tree.py``.
"""
from __future__ import annotations

import numpy as np


def ancestors(parents):
    """Boolean [n, n]: row i marks node i and its ancestors."""
    sees = np.zeros((len(parents), len(parents)), dtype=bool)
    for i, up in enumerate(parents):
        if i:
            sees[i] = sees[up]
        sees[i, i] = True
    return sees


def tree_reference(q, k, v, seqlens, sees):
    """out [T, Hq, d] and lse [T, Hq] of the last len(sees[b]) tokens of every sequence; sees[b] is a
    boolean [n, n] of the nodes that each node sees.  k, v [N, Hkv, d], sequences back to back."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    at = t = 0
    for L, s in zip(seqlens, sees):
        n = len(s)
        for i in range(n):
            rows = at + np.flatnonzero(np.concatenate((np.ones(L - n, dtype=bool), s[i])))
            if rows.size == 0:
                continue
            for h in range(Hq):
                x = k[rows, h // G] @ q[t + i, h] / np.sqrt(d)
                w = np.exp(x - x.max())
                out[t + i, h] = w @ v[rows, h // G] / w.sum()
                lse[t + i, h] = x.max() + np.log(w.sum())
        at, t = at + L, t + n
    return out, lse


def weights(p):
    """Probabilities as they count: NaN and negative values 0, at most 1."""
    return np.clip(np.nan_to_num(np.asarray(p, dtype=np.float64), nan=0.0, posinf=1.0, neginf=0.0), 0.0, 1.0)


def verify_walk(target, tokens, uniform, parents=None, draft=None):
    """(path, emitted) of one sequence of n >= 1 nodes: target [n, V], draft [n, V] or None."""
    n, V = target.shape
    u = np.asarray(uniform, dtype=np.float64)
    path, emitted = [0], []
    while True:
        node = path[-1]
        p = weights(target[node])
        left, mass, tried, went = p.copy(), 1.0, False, None
        for i in range(node + 1, n):
            if (parents[i] if parents is not None else i - 1) != node:
                continue
            x = int(tokens[i])
            there = 0 <= x < V
            if draft is not None:
                q = weights(draft[i])
                if there and p[x] > 0 and u[i] * q[x] < p[x]:
                    went = i
                    break
                left = np.maximum(p - q, 0.0)
            else:
                w = left[x] if there else 0.0
                if w > 0 and u[i] * mass < w:
                    went = i
                    break
                mass -= w
                if there:
                    left[x] = 0.0
            tried = True
        if went is None:
            break
        path.append(went)
        emitted.append(int(tokens[went]))
    if tried and left.sum() == 0:
        left = p
    sums = np.cumsum(left)
    emitted.append(int(np.searchsorted(sums, u[0] * sums[-1], side="right")) if sums[-1] > 0 else -1)
    return path, emitted


def keep_rows(rows, path):
    """rows [n, ...] after row i took row path[i], as far as the path ascends within [0, n)."""
    new = rows.copy()
    for i, x in enumerate(path):
        if not 0 <= x < len(rows) or (i and x <= path[i - 1]):
            break
        new[i] = rows[x]
    return new
