"""Shared prefixes, weights and eviction, in plain fp64 NumPy.

TEST INFRASTRUCTURE ONLY, like oracle/attention.py: one sequence, logical cache.

* shared prefix: nothing but full attention over prefix rows and own rows;
* cross attention: every query row attends to all N_b states;
* weights: the probability of every row, summed over a KV head's query heads,
  added to an accumulator; the current token's row starts from its own;
* eviction: of n weighed rows the recent ones stay (position >= seen - recent),
  then those of largest weight, ties to the lower row, `budget` in all; the kept
  rows at or behind the budget move into the freed rows before it, in order.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64


def attend_all(q, K, V):
    """q [T, H_q, d], K, V [N, H_kv, d] -> (out [T, H_q, d], p [T, H_q, N], sum p|V| like out)."""
    q, K, V = _f64(q), _f64(K), _f64(V)
    T, n_q, d = q.shape
    n_kv = K.shape[1]
    out, mag = np.zeros((T, n_q, d)), np.zeros((T, n_q, d))
    p = np.zeros((T, n_q, K.shape[0]))
    if K.shape[0] == 0:
        return out, p, mag
    for h in range(n_q):
        j = h // (n_q // n_kv)
        s = q[:, h] @ K[:, j].T / math.sqrt(d)
        e = np.exp(s - s.max(-1, keepdims=True))
        p[:, h] = e / e.sum(-1, keepdims=True)
        out[:, h] = p[:, h] @ V[:, j]
        mag[:, h] = p[:, h] @ np.abs(V[:, j])
    return out, p, mag


def add_weights(mass, pos, p, n_t: int, protect: int, seen: int, n_kv: int):
    """mass, pos [H_kv, rows] after a step with probabilities p [H_q, N_t]."""
    mass, pos = _f64(mass).copy(), np.array(np.asarray(pos), dtype=np.int64)
    w = _f64(p).reshape(n_kv, -1, n_t).sum(1)
    for r in range(protect, n_t):
        i = r - protect
        if i >= mass.shape[1]:
            break
        if r == n_t - 1:
            mass[:, i] = w[:, r]
            pos[:, i] = seen - 1
        else:
            mass[:, i] += w[:, r]
    return mass, pos


def evict_moves(mass, pos, n: int, seen: int, budget: int, recent: int):
    """One KV head: (rows that stay ascending, [(from, to), ...]) of rows 0 .. n-1."""
    mass = [float(x) for x in mass[:n]]

    def order(r):   # a NaN is smaller than any number
        nan = math.isnan(mass[r])
        return (int(pos[r]) < seen - recent, nan, 0.0 if nan else -mass[r], r)

    best = sorted(range(n), key=order)
    stay = sorted(best[:min(n, budget)])
    keep = len(stay)
    kept = set(stay)
    holes = [r for r in range(keep) if r not in kept]
    late = [r for r in stay if r >= keep]
    return stay, list(zip(late, holes))
