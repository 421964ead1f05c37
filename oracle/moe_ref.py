"""Float64 CPU oracle of the operators between a router's choice and the
optimizer step: tokens sorted by expert, dispatched to their experts' rows and
combined from them, the gradients of both, and the norm of all gradients.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA path and imports
nothing from it.  The definitions are those of ``include/muon.h``.
"""
from __future__ import annotations

import math

import numpy as np


def sort(chosen, experts, mask=None, rows=None):
    """(offsets [experts + 1], order, place [T, K], bad): copy after copy into its
    expert's list; the lists one after the other, cut to `rows` rows.  bad: whether a
    choice was neither an expert nor -1, or copies did not fit."""
    chosen = np.asarray(chosen)
    T, K = chosen.shape
    rows = T * K if rows is None else rows
    lists, bad = [[] for _ in range(experts)], False
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        for k in range(K):
            e = int(chosen[t, k])
            if 0 <= e < experts:
                lists[e].append(t * K + k)
            elif e != -1:
                bad = True
    order = [i for copies in lists for i in copies]
    ends = np.cumsum([0] + [len(c) for c in lists])
    bad = bad or len(order) > rows
    order = order[:rows]
    place = np.full(T * K, -1, dtype=np.int64)
    place[order] = np.arange(len(order))
    return np.minimum(ends, rows), np.array(order, dtype=np.int64), place.reshape(T, K), bad


def dispatch(x, place, rows):
    """xs [rows, D]; rows without a copy are NaN."""
    x = np.asarray(x, dtype=np.float64)
    xs = np.full((rows, x.shape[1]), np.nan)
    for t, at in enumerate(place):
        for r in at:
            if 0 <= r < rows:
                xs[r] = x[t]
    return xs


def combine(ys, place, weights=None):
    """(out [T, D], mass): mass is the sum of the terms' magnitudes.  No weights: 1."""
    ys = np.asarray(ys, dtype=np.float64)
    out = np.zeros((len(place), ys.shape[1]))
    mass = np.zeros_like(out)
    for t, at in enumerate(place):
        for k, r in enumerate(at):
            if 0 <= r < len(ys):
                term = ys[r] * (1.0 if weights is None else float(weights[t][k]))
                out[t] += term
                mass[t] += np.abs(term)
    return out, mass


def combine_grad(dout, ys, weights, place):
    """(dys [rows, D], dweights [T, K], mass of dweights); rows without a copy are NaN."""
    dout, ys = np.asarray(dout, dtype=np.float64), np.asarray(ys, dtype=np.float64)
    dys = np.full(ys.shape, np.nan)
    dw, mass = np.zeros(np.shape(place)), np.zeros(np.shape(place))
    for t, at in enumerate(place):
        for k, r in enumerate(at):
            if 0 <= r < len(ys):
                dys[r] = float(weights[t][k]) * dout[t]
                dw[t, k] = np.sum(dout[t] * ys[r])
                mass[t, k] = np.sum(np.abs(dout[t] * ys[r]))
    return dys, dw, mass


def grad_norm(tensors, max_norm=math.inf):
    """(norm, scale) of a list of arrays; scale is NaN where norm is not finite."""
    norm = math.sqrt(math.fsum(float(np.sum(np.square(np.asarray(t, dtype=np.float64)))) for t in tensors))
    if not math.isfinite(norm):
        return norm, math.nan
    return norm, min(1.0, max_norm / (norm + 1e-6))
