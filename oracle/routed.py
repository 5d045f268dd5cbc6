"""Routed fields and distillation, in float64 from their definitions: pairs
sorted by expert, rows moved there and back, one linear layer per expert, the
loss against a teacher's top logits, and every gradient."""
from __future__ import annotations

import numpy as np


def plan(ids, n_experts):
    """offsets, order, place of ids [n, k]; ids outside [0, n_experts) last."""
    flat = np.asarray(ids, np.int64).reshape(-1)
    key = np.where((flat >= 0) & (flat < n_experts), flat, n_experts)
    order = np.argsort(key, kind="stable")
    place = np.empty_like(order)
    place[order] = np.arange(order.size)
    offsets = np.array([(key < e).sum() for e in range(n_experts + 1)], np.int64)
    return offsets, order, place.reshape(np.shape(ids))


def gather(x, offsets, place):
    n, k = place.shape
    rows = np.zeros((n * k, x.shape[1]))
    for t in range(n):
        for j in range(k):
            if place[t, j] < offsets[-1]:
                rows[place[t, j]] = x[t]
    return rows


def combine(y, offsets, place, weights=None):
    n, k = place.shape
    out = np.zeros((n, y.shape[1]))
    for t in range(n):
        for j in range(k):
            if place[t, j] < offsets[-1]:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * np.asarray(y[place[t, j]], np.float64)
    return out


def combine_grad(dout, y, offsets, place, weights=None):
    n, k = place.shape
    dy, dw = np.zeros(y.shape), np.zeros((n, k))
    for t in range(n):
        for j in range(k):
            s = place[t, j]
            if s < offsets[-1]:
                w = 1.0 if weights is None else float(weights[t, j])
                dy[s] = w * np.asarray(dout[t], np.float64)
                dw[t, j] = np.dot(np.asarray(y[s], np.float64), np.asarray(dout[t], np.float64))
    return dy, dw


def expert_linear(x, weight, bias, offsets, slots, rows=None, relu=False):
    """x rows per slot (or x[rows[s]])."""
    x, weight = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    xs = x if rows is None else x[rows]
    y = np.zeros((slots, weight.shape[1]))
    for e in range(weight.shape[0]):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi] = xs[lo:hi] @ weight[e].T
        if bias is not None:
            y[lo:hi] += np.asarray(bias[e], np.float64)
    return np.maximum(y, 0.0) if relu else y


def expert_linear_grad(dz, x, weight, offsets, rows=None, relu_x=False):
    dz, x, weight = (np.asarray(a, np.float64) for a in (dz, x, weight))
    xs = x if rows is None else x[rows]
    E, d_out, d_in = weight.shape
    dx, dw, db = np.zeros((dz.shape[0], d_in)), np.zeros(weight.shape), np.zeros((E, d_out))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        dx[lo:hi] = dz[lo:hi] @ weight[e]
        dw[e] = dz[lo:hi].T @ xs[lo:hi]
        db[e] = dz[lo:hi].sum(0)
    if relu_x:
        live = offsets[-1]
        dx[:live] *= xs[:live] > 0
    return dx, dw, db


def distill(logits, t_logits, t_ids, temperature, row_scale=None):
    """loss [n], lse [n], grad [n, classes] row by row."""
    logits, t_logits = np.asarray(logits, np.float64), np.asarray(t_logits, np.float64)
    n, V = logits.shape
    T = float(temperature)
    loss, lse, grad = np.zeros(n), np.zeros(n), np.zeros((n, V))
    with np.errstate(all="ignore"):
        for r in range(n):
            z = logits[r] / T
            m = z.max()
            none = np.isneginf(m)
            total = 0.0 if none else np.exp(z - m).sum()  # (kept apart from m, which may be too large to add it to)
            lse[r] = m if none else m + np.log(total)
            logq = np.full(V, -np.inf) if none else (z - m) - np.log(total)
            q = np.zeros(V) if none else np.exp(z - m) / total
            ok = (t_ids[r] >= 0) & (t_ids[r] < V)
            t, idx = t_logits[r][ok] / T, t_ids[r][ok]
            if t.size == 0 or np.isneginf(t.max()):
                continue
            logp = t - t.max() - np.log(np.exp(t - t.max()).sum())
            p = np.exp(logp)
            for pj, lp, v in zip(p, logp, idx):
                if pj != 0:  # (a NaN counts)
                    loss[r] += pj * (lp - logq[v])
            loss[r] *= T * T
            g = q * p.sum()
            np.subtract.at(g, idx, p)
            grad[r] = T * g * (1.0 if row_scale is None else float(row_scale[r]))
    return loss, lse, grad
