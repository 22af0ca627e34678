"""Attention over spans in plain numpy float64: forward, backward and document spans by brute force."""
from __future__ import annotations

import numpy as np


def document_spans(bounds, B, s, prefix=None):
    """(lo, hi, positions) [B*s], token by token from the definition."""
    lo, hi, pos = (np.zeros(B * s, dtype=np.int32) for _ in range(3))
    for t in range(B * s):
        for d in range(len(bounds) - 1):
            if bounds[d] <= t < bounds[d + 1]:
                first = max(bounds[d], t // s * s)
                end = min(bounds[d + 1], t // s * s + s)
                lo[t] = first - t // s * s
                hi[t] = min(end, max(t + 1, first + (prefix[d] if prefix is not None else 0))) - t // s * s
                pos[t] = t - first
    return lo, hi, pos


def visible(lo, hi, s):
    """Boolean [s, s]: which key columns each query row of one sequence sees."""
    j = np.arange(s)
    return (j >= np.asarray(lo)[:, None]) & (j < np.asarray(hi)[:, None])


def scores(q, k, vis, scale, cap=0.0, slope=0.0):
    """(z with -inf where nothing is seen, dz / d(scale q.k)) for one head: q [n, d], k [m, d]."""
    z = scale * (q @ k.T)
    dz = np.ones_like(z)
    if cap:
        t = np.tanh(z / cap)
        z, dz = cap * t, 1 - t * t
    z = z - slope * np.abs(np.arange(len(q))[:, None] - np.arange(len(k)))
    return np.where(vis, z, -np.inf), dz


def forward(q, k, v, vis, scale, cap=0.0, slope=0.0):
    """(o, lse, p) for one head; lse in log2 units; an empty row gives 0 and -inf."""
    z, _ = scores(q, k, vis, scale, cap, slope)
    m = z.max(axis=1, keepdims=True, initial=-np.inf)
    m = np.where(np.isfinite(m), m, 0.0)
    e = np.exp(z - m)
    l = e.sum(axis=1, keepdims=True)
    p = e / np.where(l == 0, 1.0, l)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(l))[:, 0] / np.log(2.0)
    return p @ v, lse, p


def backward(q, k, v, vis, scale, do, cap=0.0, slope=0.0, o=None, lse=None):
    """(dq, dk, dv, p, ds) for one head. With o and lse the probabilities and row sums are taken from
    them, as a backward pass that is handed the forward's rounded results does."""
    z, dz = scores(q, k, vis, scale, cap, slope)
    if lse is None:
        o, _, p = forward(q, k, v, vis, scale, cap, slope)
    else:
        p = np.exp(z - np.where(np.isfinite(lse), lse, 0.0)[:, None] * np.log(2.0))
    ds = p * (do @ v.T - (do * o).sum(axis=1, keepdims=True)) * dz
    return scale * (ds @ k), scale * (ds.T @ q), p.T @ do, p, ds
