"""Float64 CPU oracle of the operators that produce a mixture-of-experts step's
gradients: the router balance loss, 8-bit activation checkpoints, the gated
activation on them and the experts' weight gradients.

TEST INFRASTRUCTURE ONLY.  It shares no code with the CUDA path and imports
nothing from it.  The definitions are those of ``include/muon.h``; the pages
the optimizer follows do not describe these operators.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 32


# ---- balance loss -----------------------------------------------------------
def sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    z = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + z), z / (1.0 + z))


def probabilities(logits, score):
    """Rows of probabilities; a row whose scores are all 0 gives 0."""
    x = np.asarray(logits, dtype=np.float64)
    if score == "sigmoid":
        a = sigmoid(x)
    else:
        top = np.max(x, axis=1, keepdims=True) if x.shape[0] else np.zeros((0, 1))
        a = np.exp(x - np.where(np.isneginf(top), 0.0, top))
    z = a.sum(axis=1, keepdims=True)
    return np.divide(a, z, out=np.zeros_like(a), where=z != 0)


def balance(logits, chosen, seq_begin=None, mask=None, score="softmax", coef=1e-2):
    """dict(loss, counts, load [S, E] = coef/N f, grad, mass): mass is
    coef/N p (f + sum f p), the size of the gradient's terms."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    K = np.asarray(chosen).shape[1]
    begin = [0, T] if seq_begin is None else [int(v) for v in seq_begin]
    S = len(begin) - 1
    valid = np.zeros(T, dtype=bool)
    for b, e in zip(begin[:-1], begin[1:]):
        valid[b:e] = True
    if mask is not None:
        valid &= np.asarray(mask).astype(bool)
    N = int(valid.sum())
    counts = np.zeros(E, dtype=np.int64)
    load = np.zeros((S, E))
    grad, mass = np.zeros((T, E)), np.zeros((T, E))
    loss = 0.0
    for s, (b, e) in enumerate(zip(begin[:-1], begin[1:])):
        rows = np.nonzero(valid[b:e])[0] + b
        if len(rows) == 0:
            continue
        ids = np.asarray(chosen)[rows].ravel()
        c = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        counts += c
        load[s] = coef / N * (E / (K * len(rows))) * c
        p = probabilities(x[rows], score)
        loss += float((load[s] * p.sum(axis=0)).sum())
        dot = (p * load[s]).sum(axis=1, keepdims=True)
        slope = 1.0 - sigmoid(x[rows]) if score == "sigmoid" else 1.0
        grad[rows] = p * slope * (load[s] - dot)
        mass[rows] = p * slope * (load[s] + dot)
    return dict(loss=loss, counts=counts, load=load, grad=grad, mass=mass)


# ---- 8-bit checkpoints ------------------------------------------------------
def _exponent(amax: float) -> int:
    """Least e >= -126 with 127 * 2^e >= amax."""
    if amax == 0.0:
        return -126
    e = math.frexp(amax)[1] - 9
    while math.ldexp(127.0, e) < amax:
        e += 1
    return max(e, -126)


def act8_encode(x):
    """(codes int8 [rows, blocks*32], bytes uint8 [rows, blocks])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    codes = np.zeros((rows, nb * BLOCK), dtype=np.int8)
    exps = np.zeros((rows, nb), dtype=np.uint8)
    for r in range(rows):
        for b in range(nb):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.all(np.isfinite(v)):
                exps[r, b] = 255
                continue
            e = _exponent(float(np.max(np.abs(v))))
            q = np.rint(v * math.ldexp(1.0, -e)) if e > -1000 else v
            if e == 122:
                q = np.clip(q, -63, 63)
            codes[r, b * BLOCK:b * BLOCK + len(v)] = q
            exps[r, b] = e + 127
    return codes, exps


def act8_decode(codes, exps, cols):
    step = np.ldexp(1.0, exps.astype(np.int64) - 127)
    step = np.where(exps == 255, np.nan, step)
    rows, nb = exps.shape
    v = codes.astype(np.float64).reshape(rows, nb, BLOCK) * step[:, :, None]
    return v.reshape(rows, nb * BLOCK)[:, :cols]


# ---- gated activation -------------------------------------------------------
def swiglu(gate, up):
    return gate * sigmoid(gate) * up


def swiglu_grad(dh, gate, up):
    """(dgate, dup) of sum(dh * silu(gate) * up)."""
    s = sigmoid(gate)
    return dh * up * s * (1.0 + gate * (1.0 - s)), dh * gate * s


# ---- weight gradients -------------------------------------------------------
def weight_grads(dy, x, offsets):
    """([E, out, in] gradients, the same sums of absolute products)."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    pairs = list(zip(offsets[:-1], offsets[1:]))
    g = np.stack([dy[a:b].T @ x[a:b] for a, b in pairs])
    size = np.stack([np.abs(dy[a:b]).T @ np.abs(x[a:b]) for a, b in pairs])
    return g, size
