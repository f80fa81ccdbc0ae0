"""Float64 oracle of the experts' operators: the sort of a batch's choices by
expert, the rows' way to the experts and back, and products over groups of
rows with bias, activation and residual, with their gradients.  Plain numpy,
no code shared with the kernels."""

from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[float])
_erfc = np.vectorize(math.erfc, otypes=[float])


def sort(ids, experts):
    """(offsets, order, place) of the choices ids (tokens, top)."""
    flat = np.asarray(ids).reshape(-1)
    place = np.full(flat.size, -1)
    order = np.full(flat.size, -1)
    offsets = [0]
    at = 0
    for e in range(experts):
        for s in np.nonzero(flat == e)[0]:
            place[s], order[at] = at, s
            at += 1
        offsets.append(at)
    return np.array(offsets), order, place.reshape(np.shape(ids))


def gather(x, place, into):
    """`into` with every token's row at its places."""
    out = np.array(into, dtype=np.float64)
    for t, row in enumerate(place):
        for p in row:
            if p >= 0:
                out[p] = x[t]
    return out


def combine(ys, place, weights=None, residual=None):
    y = np.zeros((len(place), ys.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    for t, row in enumerate(place):
        for j, p in enumerate(row):
            if p >= 0:
                y[t] += ys[p] * (1.0 if weights is None else weights[t, j])
    return y


def combine_grad(dy, ys, weights, place, into):
    dys, dw = np.array(into, dtype=np.float64), np.zeros(np.shape(weights))
    for t, row in enumerate(place):
        for j, p in enumerate(row):
            if p >= 0:
                dys[p] = dy[t] * weights[t, j]
                dw[t, j] = float(np.dot(dy[t], ys[p]))
    return dys, dw


# Activations: z times a distribution function of z.  The logistic function
# is evaluated from the side where its exponential is small.
def _logistic(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1.0, e) / (1.0 + e)


def activation(name, z):
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z
    if name == "relu":
        return np.maximum(z, 0.0)
    if name == "silu":
        return z * _logistic(z)
    if name == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    return z * _logistic(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))


def slope(name, z):
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return np.ones_like(z)
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "silu":
        return _logistic(z) * (1.0 + z * _logistic(-z))
    if name == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(8.0 / math.pi)
    u = k * (z + 0.044715 * z ** 3)
    return _logistic(u) + z * _logistic(u) * _logistic(-u) * k * (1.0 + 3 * 0.044715 * z * z)


def _bounds(offsets, rows):
    return [0, rows] if offsets is None else list(offsets)


def linear(x, w, bias=None, act="none", residual=None, offsets=None, y=None, pre=None):
    """(y, pre): w (groups, out, in), bias (groups, out); rows of no group as in the given y and pre."""
    b = _bounds(offsets, len(x))
    y = np.zeros((len(x), w.shape[1])) if y is None else np.array(y, dtype=np.float64)
    pre = y.copy() if pre is None else np.array(pre, dtype=np.float64)
    for g in range(len(w)):
        r = slice(b[g], b[g + 1])
        z = x[r] @ w[g].T + (0.0 if bias is None else bias[g])
        pre[r] = z
        y[r] = activation(act, z) + (0.0 if residual is None else residual[r])
    return y, pre


def linear_grad(dy, x, w, act="none", pre=None, offsets=None, x_act="none", x_pre=None, dx=None, dw=None, db=None):
    """(dx, dw, db): dw and db are added to the given ones."""
    b = _bounds(offsets, len(dy))
    dx = np.zeros(x.shape) if dx is None else np.array(dx, dtype=np.float64)
    dw = np.zeros(w.shape) if dw is None else np.array(dw, dtype=np.float64)
    db = np.zeros(w.shape[:2]) if db is None else np.array(db, dtype=np.float64)
    for g in range(len(w)):
        r = slice(b[g], b[g + 1])
        dz = dy[r] * (1.0 if act == "none" else slope(act, pre[r]))
        dx[r] = (dz @ w[g]) * (1.0 if x_act == "none" else slope(x_act, x_pre[r]))
        dw[g] += dz.T @ x[r]
        db[g] += dz.sum(0)
    return dx, dw, db
