"""fp64 CPU oracle of the operators before and behind the LM head.

TEST INFRASTRUCTURE, as oracle/linear_logp.py: only tests call it, the
product path never does, and it shares no code with it.

Plain definitions in float64 on the exact values of the inputs:

  layer_norm  mean = sum x / H, rstd = 1 / sqrt(sum (x - mean)^2 / H + eps),
              n = (x - mean) rstd, y = n w + b;
              grad_x = rstd (gw - mean(gw) - n mean(gw n)), gw = g w,
              grad_w = sum_t g n, grad_b = sum_t g.
  rms_norm    the same with mean 0 and without the term mean(gw).
  embed       out[t] = scale E[ids[t]], zero rows of ignore_index, NaN rows of
              ids outside [0, V); grad_E[v] = scale sum over ids[t] = v of g[t].
  clip        norm = sqrt(sum x^2), c = max_norm / norm if norm > max_norm.
"""
from __future__ import annotations

import numpy as np

IGNORE_INDEX = -100

__all__ = ["norm_forward", "norm_backward", "embed_forward", "embed_backward", "grad_norm", "clip_factor"]


def norm_forward(x, w, b, eps, center):
    """(y, n, mean [T], rstd [T]); w and b may be None."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(axis=1) if center else np.zeros(x.shape[0])
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    n = d * rstd[:, None]
    y = n if w is None else n * np.asarray(w, dtype=np.float64)
    return (y if b is None else y + np.asarray(b, dtype=np.float64)), n, mean, rstd


def norm_backward(x, w, g, eps, center):
    """(grad_x, grad_w, grad_b) of sum(g * y)."""
    g = np.asarray(g, dtype=np.float64)
    _, n, _, rstd = norm_forward(x, w, None, eps, center)
    gw = g if w is None else g * np.asarray(w, dtype=np.float64)
    grad = gw - n * (gw * n).mean(axis=1, keepdims=True)
    if center:
        grad = grad - gw.mean(axis=1, keepdims=True)
    return rstd[:, None] * grad, (g * n).sum(axis=0), g.sum(axis=0)


def embed_forward(ids, E, scale, ignore_index=IGNORE_INDEX):
    E = np.asarray(E, dtype=np.float64)
    out = np.full((len(ids), E.shape[1]), np.nan)
    for t, i in enumerate(ids):
        if i == ignore_index:
            out[t] = 0.0
        elif 0 <= i < len(E):
            out[t] = scale * E[i]
    return out


def embed_backward(ids, g, V, scale, ignore_index=IGNORE_INDEX):
    g = np.asarray(g, dtype=np.float64)
    grad = np.zeros((V, g.shape[1]))
    for t, i in enumerate(ids):
        if i != ignore_index and 0 <= i < V:
            grad[i] += g[t]
    return scale * grad


def grad_norm(tensors):
    return float(np.sqrt(sum((np.asarray(t, dtype=np.float64) ** 2).sum() for t in tensors)))


def clip_factor(tensors, max_norm):
    norm = grad_norm(tensors)
    return 1.0 if norm <= max_norm else max_norm / norm
