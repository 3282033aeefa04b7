"""fp64 reference of the head's losses and of the routing to experts.

TEST INFRASTRUCTURE ONLY (tests/). Written from the formulas in
include/dmuon.h, one token at a time where that is plainest; shares no code
with the library.
"""

from __future__ import annotations

import numpy as np


def log_softmax(z):
    """(log p, lse) of the rows of z."""
    top = z.max(axis=1, keepdims=True)
    lse = top + np.log(np.exp(z - top).sum(axis=1, keepdims=True))
    return z - lse, lse[:, 0]


def xent(hidden, weight, targets, grad_loss=None):
    """dict(loss, lse[, dz, dhidden, dweight]) of the softmax cross entropy."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    z = h @ w.T
    logp, lse = log_softmax(z)
    loss = np.zeros(len(h))
    dz = np.zeros_like(z)
    for t, y in enumerate(np.asarray(targets)):
        if not 0 <= y < len(w):
            continue
        others = np.delete(z[t], y) - z[t, y]
        # -log p of a sure token from the others' ratio to it
        loss[t] = np.log1p(np.exp(others).sum()) if others.size and others.max() < 50 else -logp[t, y]
        if grad_loss is not None:
            dz[t] = np.exp(logp[t])
            dz[t, y] -= 1.0
            dz[t] *= float(grad_loss[t])
    out = dict(loss=loss, lse=lse, z=z)
    if grad_loss is not None:
        out.update(dz=dz, dhidden=dz @ w, dweight=dz.T @ h)
    return out


def teacher(top_ids, top_logits, vocab, temperature):
    """The teacher's distribution over the vocabulary, row by row (a list of {id: probability})."""
    rows = []
    for ids, lg in zip(np.asarray(top_ids), np.asarray(top_logits, np.float64)):
        on = [(int(i), x) for i, x in zip(ids, lg) if 0 <= i < vocab and x != -np.inf]
        row = []
        if on:
            best = max(x for _, x in on)
            e = [np.exp((x - best) / temperature) for _, x in on]
            row = [(i, v / sum(e)) for (i, _), v in zip(on, e)]
        rows.append(row)
    return rows


def distill(hidden, weight, top_ids, top_logits, temperature, grad_loss=None):
    """dict(loss, lse[, dz, dhidden, dweight]) of the divergence from a teacher's top logits."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    z = h @ w.T / temperature
    logp, lse = log_softmax(z)
    loss = np.zeros(len(h))
    dz = np.zeros_like(z)
    for t, row in enumerate(teacher(top_ids, top_logits, len(w), temperature)):
        for i, q in row:
            if q > 0:
                loss[t] += temperature ** 2 * q * (np.log(q) - logp[t, i])
        if grad_loss is not None and row:
            dz[t] = np.exp(logp[t])
            for i, q in row:
                dz[t, i] -= q
            dz[t] *= float(grad_loss[t]) * temperature
    out = dict(loss=loss, lse=lse, z=z)
    if grad_loss is not None:
        out.update(dz=dz, dhidden=dz @ w, dweight=dz.T @ h)
    return out


def route(expert_ids, experts):
    """(dest, source, offsets): rows by expert, then by assignment."""
    ids = np.asarray(expert_ids)
    flat = ids.reshape(-1)
    order = [i for e in range(experts) for i in np.nonzero(flat == e)[0]]
    dest = np.full(flat.size, -1, np.int64)
    source = np.full(flat.size, -1, np.int64)
    for r, i in enumerate(order):
        dest[i], source[r] = r, i
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(experts)])])
    return dest.reshape(ids.shape), source, offsets


def dispatch(x, source, top):
    x = np.asarray(x, np.float64)
    xs = np.zeros((len(source), x.shape[1]))
    for r, i in enumerate(source):
        if i >= 0:
            xs[r] = x[i // top]
    return xs


def combine(ys, weights, dest):
    ys = np.asarray(ys, np.float64)
    y = np.zeros((dest.shape[0], ys.shape[1]))
    for t in range(dest.shape[0]):
        for k in range(dest.shape[1]):
            if dest[t, k] >= 0:
                y[t] += (1.0 if weights is None else float(weights[t, k])) * ys[dest[t, k]]
    return y


def combine_backward(dy, ys, weights, dest):
    dy, ys = np.asarray(dy, np.float64), np.asarray(ys, np.float64)
    dys, dw = np.zeros_like(ys), np.zeros(dest.shape)
    for t in range(dest.shape[0]):
        for k in range(dest.shape[1]):
            r = dest[t, k]
            if r >= 0:
                dys[r] = float(weights[t, k]) * dy[t]
                dw[t, k] = dy[t] @ ys[r]
    return dys, dw
