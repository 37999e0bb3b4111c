"""Verification of drafted tokens in fp64 (test infrastructure; see ``oracle/__init__``).

Drafted token x_t is kept when u_t q_t(x_t) < p_t(x_t); at the first that is not, a token is drawn from
max(p_t - q_t, 0) (from p_t where that has no mass), after the last one from the next row of p, at the
lowest index whose cumulative sum passes u times the total. Values that are not positive and finite
count as zero.
"""
from __future__ import annotations

import numpy as np


def clean(x) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    return np.where(np.isfinite(x) & (x > 0), x, 0.0)


def sample(w: np.ndarray, u: float) -> int:
    cum = np.cumsum(w)
    over = np.nonzero(cum > u * cum[-1])[0]
    mass = np.nonzero(w > 0)[0]
    if len(mass) == 0:
        return -1
    return int(over[0]) if len(over) else int(mass[-1])


def verify_one(x, p, q, u, n):
    """One request: x [T] drafted ids, p [T + 1, V], q [T, V] or None, u [T + 1], n drafted.
    Returns (tokens [T + 1], accepted)."""
    T, V = len(x), p.shape[1]
    p = clean(p)
    q = None if q is None else clean(q)
    tokens = np.full(T + 1, -1, dtype=np.int64)
    a = 0
    while a < n:
        if not 0 <= x[a] < V:
            break
        if not float(u[a]) * (1.0 if q is None else q[a, x[a]]) < p[a, x[a]]:
            break
        tokens[a] = x[a]
        a += 1
    w = p[a]
    if a < n:
        rest = w.copy()
        if q is not None:
            rest = np.maximum(w - q[a], 0.0)
        elif 0 <= x[a] < V:
            rest[x[a]] = 0.0
        w = rest if rest.sum() > 0 else w
    tokens[a] = sample(w, float(u[-1]))
    return tokens, a
