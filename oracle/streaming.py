"""Streaming routed fields, in float64 from their definitions: the gate and its
gradient, the whole routed layer sample by sample, the gated linear recurrence
step by step and its gradient, and the norm of a list of gradients."""
from __future__ import annotations

import numpy as np


def gate(logits, k, renorm):
    """ids [n, k] (largest first, lowest index among equals, -1: none left) and weights."""
    z = np.asarray(logits, np.float64)
    n, E = z.shape
    ids, w = np.full((n, k), -1, np.int64), np.zeros((n, k))
    for t in range(n):
        order = np.argsort(-z[t], kind="stable")[:k]
        live = [v for v in order if z[t, v] != -np.inf]
        if not live:
            continue
        e = np.exp(z[t] - z[t, live[0]])
        total = e[live].sum() if renorm else e.sum()
        for j, v in enumerate(live):
            ids[t, j], w[t, j] = v, e[v] / total
    return ids, w


def gate_grad(dweights, logits, ids, weights, n_experts, renorm):
    n, k = ids.shape
    out = np.zeros((n, n_experts))
    for t in range(n):
        live = [j for j in range(k) if 0 <= ids[t, j] < n_experts]
        w = {j: float(weights[t, j]) for j in live}
        d = {j: float(dweights[t, j]) for j in live}
        s = sum(w[j] * d[j] for j in live)
        if renorm:
            for j in live:
                out[t, ids[t, j]] += w[j] * (d[j] - s)
            continue
        z = np.asarray(logits[t], np.float64)
        m = z.max()
        p = np.zeros(n_experts) if m == -np.inf else np.exp(z - m) / np.exp(z - m).sum()
        out[t] = -p * s
        for j in live:
            out[t, ids[t, j]] += w[j] * d[j]
    return out


def routed_mlp(x, ids, weights, w1, b1, w2, b2, act):
    x, w1, w2 = (np.asarray(a, np.float64) for a in (x, w1, w2))
    E, d_out, hidden = w2.shape
    out = np.zeros((x.shape[0], d_out))
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < E:
                continue
            z = w1[e] @ x[t] + (0.0 if b1 is None else np.asarray(b1[e], np.float64))
            if act == "relu":
                z = np.maximum(z, 0.0)
            elif act == "gated":
                z = z[:hidden] / (1.0 + np.exp(-z[:hidden])) * z[hidden:]
            y = w2[e] @ z + (0.0 if b2 is None else np.asarray(b2[e], np.float64))
            out[t] += (1.0 if weights is None else float(weights[t, j])) * y
    return out


def _wide(a, d):
    return np.repeat(np.asarray(a, np.float64), d // a.shape[1], axis=1)


def _rows(lo, hi, reverse):
    return range(hi - 1, lo - 1, -1) if reverse else range(lo, hi)


def scan(a, x, offsets, h0=None, reverse=False, mix=False):
    """h [rows, d] (NaN in rows outside every sequence) and the last states."""
    x = np.asarray(x, np.float64)
    d, A = x.shape[1], _wide(a, x.shape[1])
    n = len(offsets) - 1
    h, last = np.full(x.shape, np.nan), np.zeros((n, d))
    for s in range(n):
        state = np.zeros(d) if h0 is None else np.asarray(h0[s], np.float64)
        for r in _rows(offsets[s], offsets[s + 1], reverse):
            state = A[r] * state + ((1.0 - A[r]) * x[r] if mix else x[r])
            h[r] = state
        last[s] = state
    return h, last


def scan_grad(dh, dh_last, a, x, h, h0, offsets, reverse=False, mix=False):
    """da [rows, gates], dx [rows, d] (NaN outside every sequence), dh0."""
    dh, h = np.asarray(dh, np.float64), np.asarray(h, np.float64)
    rows, d = dh.shape
    A = _wide(a, d)
    n, gates = len(offsets) - 1, a.shape[1]
    da, dx, dh0 = np.full((rows, gates), np.nan), np.full((rows, d), np.nan), np.zeros((n, d))
    for s in range(n):
        flow = np.zeros(d) if dh_last is None else np.asarray(dh_last[s], np.float64)
        order = list(_rows(offsets[s], offsets[s + 1], reverse))
        for i in range(len(order) - 1, -1, -1):
            r = order[i]
            before = h[order[i - 1]] if i else (np.zeros(d) if h0 is None else np.asarray(h0[s], np.float64))
            D = dh[r] + flow
            term = D * (before - np.asarray(x[r], np.float64)) if mix else D * before
            da[r] = term.reshape(gates, -1).sum(1)
            dx[r] = (1.0 - A[r]) * D if mix else D
            flow = A[r] * D
        dh0[s] = flow
    return da, dx, dh0


def grad_norm(tensors):
    return float(np.sqrt(sum(np.square(np.asarray(t, np.float64)).sum() for t in tensors)))


def grad_clip(tensors, max_norm):
    norm = grad_norm(tensors)
    f = 1.0 if norm <= max_norm else max_norm / norm
    return norm, [np.asarray(t, np.float64) * f for t in tensors]
