"""The operators next to the owner step (oracle): gradient norm and clipping,
id sort, embedding lookup and gradient, products grouped by expert.

Plain float64 NumPy from the exact stored values; ids outside their range are
masked (zero rows, no contribution, sorted last).
"""
from __future__ import annotations

import numpy as np


def grad_clip_ref(tensors, max_norm: float, eps: float):
    """(norm, coefficient, clipped tensors)."""
    ts = [np.asarray(t, np.float64) for t in tensors]
    norm = float(np.sqrt(sum(float(np.sum(t * t)) for t in ts)))
    if np.isnan(norm):
        coef = norm                       # whatever the limit
    elif np.isinf(max_norm) or norm + eps == 0.0:
        coef = 1.0
    else:
        coef = max_norm / (norm + eps)
        if coef > 1.0:
            coef = 1.0
    return norm, coef, [t * coef for t in ts]


def sort_ids_ref(ids, n_keys: int):
    """(order, starts): positions stably sorted by id, masked ids last."""
    ids = np.asarray(ids, np.int64)
    keys = np.where((ids >= 0) & (ids < n_keys), ids, n_keys)
    order = np.argsort(keys, kind="stable")
    starts = np.array([int(np.sum(keys < k)) for k in range(n_keys + 1)]) if n_keys < 4096 else \
        np.searchsorted(keys[order], np.arange(n_keys + 1), side="left")
    return order.astype(np.int32), starts.astype(np.int32)


def embedding_lookup_ref(weight, ids, scale: float):
    weight, ids = np.asarray(weight, np.float64), np.asarray(ids, np.int64)
    out = np.zeros((ids.size, weight.shape[1]))
    for t, v in enumerate(ids):
        if 0 <= v < weight.shape[0]:
            out[t] = scale * weight[v]
    return out


def embedding_grad_ref(dout, ids, vocab: int, scale: float, grad0=None):
    dout, ids = np.asarray(dout, np.float64), np.asarray(ids, np.int64)
    grad = np.zeros((vocab, dout.shape[1])) if grad0 is None else np.array(grad0, np.float64)
    for t, v in enumerate(ids):
        if 0 <= v < vocab:
            grad[v] += scale * dout[t]
    return grad


def expert_matmul_ref(x, w, starts, input_grad: bool = False):
    """y[t] = W_e x[t] (input_grad: W_e^T x[t]) for t in [starts[e], starts[e + 1]);
    zero rows from starts[-1] on."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    y = np.zeros((x.shape[0], w.shape[2] if input_grad else w.shape[1]))
    for e in range(w.shape[0]):
        lo, hi = int(starts[e]), int(starts[e + 1])
        y[lo:hi] = x[lo:hi] @ (w[e] if input_grad else w[e].T)
    return y


def expert_weight_grad_ref(dy, x, starts, dw0=None):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    n_e = len(starts) - 1
    dw = np.zeros((n_e, dy.shape[1], x.shape[1])) if dw0 is None else np.array(dw0, np.float64)
    for e in range(n_e):
        lo, hi = int(starts[e]), int(starts[e + 1])
        dw[e] += dy[lo:hi].T @ x[lo:hi]
    return dw
