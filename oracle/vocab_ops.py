"""fp64 CPU oracle of the operators on the whole next-token distribution.

TEST INFRASTRUCTURE, as oracle/linear_logp.py: only tests call it, the
product path never does, and it shares no code with it.

Plain definitions in float64 on the exact values of the inputs, z = h W^T:

  top:      logp = z_y - lse, entropy = -sum p log p, the K largest logits
            (ties to the lowest id) and their log p;
            dz_v = g [v = y] - p_v (g + g_entropy (entropy + log p_v)).
  distill:  q = softmax over the kept slots of logits / temperature, p =
            softmax of z / temperature, loss = sum q (log q - log p[ids])
            over slots (an id in two of them keeps two terms);
            dz_v = (g / temperature) (p_v - sum over slots k of v of q_k).
  grad_h = dz W, grad_W = dz^T h.

The pins (tests/test_oracle_vocab_ops_pins.py) are closed forms, brute force
and central differences.
"""
from __future__ import annotations

import numpy as np

from .linear_logp import IGNORE_INDEX, _as_f64

__all__ = ["logits", "top_forward", "top_dz", "teacher", "distill_forward", "distill_dz"]


def logits(h, W, temperature=1.0):
    return _as_f64(h) @ _as_f64(W).T / temperature


def _log_softmax(z):
    m = z.max(axis=1, keepdims=True)
    return z - m - np.log(np.exp(z - m).sum(axis=1, keepdims=True))


def _xlogx_sum(logp):
    p = np.exp(logp)
    return (p * np.where(p > 0, logp, 0.0)).sum(axis=1)


def top_forward(h, W, y, K, ignore_index=IGNORE_INDEX):
    """(logp [T], lse [T], entropy [T], top_logp [T, K], top_ids [T, K])."""
    z = logits(h, W)
    T, V = z.shape
    lp = _log_softmax(z)
    on = np.asarray(y) != ignore_index
    logp = np.where(on, lp[np.arange(T), np.where(on, y, 0)], 0.0)
    lse = np.where(on, (z - lp)[:, 0], 0.0)
    entropy = np.where(on, -_xlogx_sum(lp), 0.0)
    ids = np.full((T, K), -1, dtype=np.int64)
    top = np.full((T, K), -np.inf)
    n = min(K, V)
    order = np.argsort(-z, axis=1, kind="stable")[:, :n]
    ids[:, :n] = order
    top[:, :n] = np.take_along_axis(lp, order, axis=1)
    ids[~on] = -1
    top[~on] = -np.inf
    return logp, lse, entropy, top, ids


def top_dz(h, W, y, g, g_entropy, ignore_index=IGNORE_INDEX):
    """dz [T, V], and the sum of the magnitudes of its terms."""
    lp = _log_softmax(logits(h, W))
    p, ent = np.exp(lp), -_xlogx_sum(lp)[:, None]
    T = len(lp)
    on = (np.asarray(y) != ignore_index)[:, None]
    g, ge = (np.where(on, np.asarray(x, dtype=np.float64)[:, None], 0.0) for x in (g, g_entropy))
    hot = np.zeros_like(p)
    hot[np.arange(T), np.where(on[:, 0], y, 0)] = 1.0
    dz = g * hot - p * (g + ge * (ent + lp))
    size = np.abs(g) * hot + p * (np.abs(g) + np.abs(ge) * (ent + np.abs(lp)))
    return dz, size


def teacher(ids, tlogits, temperature=1.0):
    """(kept [T, K], q [T, K], log q [T, K] with 0 in empty slots)."""
    ids = np.asarray(ids)
    x = np.asarray(tlogits, dtype=np.float64) / temperature
    kept = (ids >= 0) & (x != -np.inf)
    x = np.where(kept, x, -np.inf)
    m = np.where(kept.any(axis=1), x.max(axis=1), 0.0)[:, None]
    e = np.where(kept, np.exp(np.where(kept, x - m, 0.0)), 0.0)
    s = e.sum(axis=1, keepdims=True)
    s = np.where(s > 0, s, 1.0)
    return kept, e / s, np.where(kept, np.where(kept, x - m, 0.0) - np.log(s), 0.0)


def distill_forward(h, W, ids, tlogits, temperature=1.0):
    """(loss [T], lse [T], logp_ids [T, K])."""
    z = logits(h, W, temperature)
    lp = _log_softmax(z)
    kept, q, lq = teacher(ids, tlogits, temperature)
    at = np.where(kept, ids, 0)
    lpk = np.where(kept, np.take_along_axis(lp, at, axis=1), -np.inf)
    loss = np.where(q > 0, q * (lq - np.where(kept, lpk, 0.0)), 0.0).sum(axis=1)
    on = kept.any(axis=1)
    return np.where(on, loss, 0.0), np.where(on, (z - lp)[:, 0], 0.0), lpk


def distill_dz(h, W, ids, tlogits, g, temperature=1.0):
    """dz [T, V], and the sum of the magnitudes of its terms."""
    p = np.exp(_log_softmax(logits(h, W, temperature)))
    kept, q, _ = teacher(ids, tlogits, temperature)
    on = kept.any(axis=1, keepdims=True)
    full = np.zeros_like(p)
    np.add.at(full, (np.arange(len(p))[:, None], np.where(kept, ids, 0)), q)
    c = np.where(on, np.asarray(g, dtype=np.float64)[:, None] / temperature, 0.0)
    return c * (p - full), np.abs(c) * (p + full)
