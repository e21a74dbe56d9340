"""Attention with a sliding window and sinks in float64 from its definition, one
sequence and head at a time, with its gradients written out and the cache as a
list of positions.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""
from __future__ import annotations

import numpy as np


def sees(p, j, window, sinks):
    """Whether the token at position p sees the one at position j (arrays broadcast)."""
    return (j <= p) & ((p - j < window) | (j < sinks))


def slot(t, window, sinks):
    """Row of a cache that holds the token at position t."""
    return t if t < sinks else sinks + (t - sinks) % window


def cached_positions(length, window, sinks):
    """Positions that a cache holds after `length` tokens, ascending."""
    return [t for t in range(length) if t < sinks or t >= length - window]


def keep(cache, rows, length, window, sinks):
    """cache [sinks + window, ...] after the tokens `rows` at positions length, length + 1, ..."""
    cache = cache.copy()
    for i, r in enumerate(rows):
        cache[slot(length + i, window, sinks)] = r
    return cache


def attend(q, k, v, pq, pk, window, sinks, scale):
    """One head: q [n, dk] at positions pq, k [m, dk], v [m, dv] at positions pk.
    Returns o [n, dv], lse [n], weights p [n, m]."""
    m = sees(pq[:, None], pk[None, :], window, sinks)
    s = np.where(m, scale * (q @ np.where(m.any(0)[:, None], k, 0.0).T), -np.inf)
    top = s.max(1)
    e = np.exp(s - top[:, None])
    z = e.sum(1)
    p = e / z[:, None]
    return p @ np.where(m.any(0)[:, None], v, 0.0), top + np.log(z), p


def attend_backward(q, k, v, o, lse, d_o, pq, pk, window, sinks, scale):
    """dq, dk, dv of one head, for the forward's o and lse as they are given."""
    m = sees(pq[:, None], pk[None, :], window, sinks)
    p = np.where(m, np.exp(np.where(m, scale * (q @ k.T), 0.0) - lse[:, None]), 0.0)
    ds = p * (d_o @ v.T - (d_o * o).sum(1)[:, None])
    return scale * ds @ k, scale * ds.T @ q, p.T @ d_o
