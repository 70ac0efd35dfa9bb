"""The router's selection, the balance loss and their gradient, and the global
gradient norm with clipping, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The pages give the routing's size only (8 of 384 experts: "Thinking Machines'
Inkling 2 Small Trains a 594B Model in 68 Hours", section "594B weights, 17B
at work"); the formulas are readings:
* scores s: softmax over the experts, or the sigmoid of each logit; a logit of
  -inf closes an expert, a token mask of 0 a token;
* the k open experts of largest logit (with a bias: of largest s + bias) in
  descending order, the lower index first among equals; -1 where none is left;
* gates scale * s, or scale * s / (sum of the selected s);
* loss alpha * E * sum_e f_e P_e with f_e = pairs on e / (N k), P_e = mean over
  the N tokens with an expert of the row's normalised score; f is a constant
  of the gradient;
* norm sqrt(sum of squares of all gradients); clipped = g * min(1, max_norm /
  (norm + 1e-6)); an infinite max_norm bounds nothing, an infinite norm
  included.
"""

import numpy as np

from . import formats as F


def _vals(x):
    """bfloat16 bit patterns (uint16) or floats -> float64 values."""
    x = np.asarray(x)
    return (F.bf16_bits_to_f32(x) if x.dtype == np.uint16 else x).astype(np.float64)


def scores(x, score):
    """Scores [T, E] of float64 logits; rows with no open expert are 0."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-x))
    top = x.max(axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(axis=1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def select(x, k, score="softmax", bias=None, token_mask=None):
    """ids int32 [T, k] of float64 logits x."""
    key = x if bias is None else scores(x, "sigmoid") + np.asarray(bias, np.float64)
    key = np.where(np.isneginf(x), -np.inf, key)
    if token_mask is not None:
        key = np.where(np.asarray(token_mask, bool)[:, None], key, -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    open_ = np.take_along_axis(key, order, axis=1) > -np.inf
    return np.where(open_, order, -1).astype(np.int32)


def _selected(s, ids):
    """Scores of the selected [T, k], 0 in empty slots."""
    return np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)


def _safe(v):
    return np.where(v > 0, v, 1.0)


def gates(x, ids, score="softmax", renorm=True, scale=1.0):
    w = _selected(scores(x, score), ids)
    if renorm:
        w = w / _safe(w.sum(axis=1, keepdims=True))
    return scale * w


def probabilities(x, score):
    s = scores(x, score)
    return s / _safe(s.sum(axis=1, keepdims=True))


def route(logits, k, score="softmax", renorm=True, scale=1.0, bias=None, token_mask=None):
    """Everything moe_route returns: topk_ids, gate, counts [E+1], prob_sum [E]."""
    x = _vals(logits)
    E = x.shape[1]
    ids = select(x, k, score, bias, token_mask)
    live = ids[:, 0] >= 0
    counts = np.zeros(E + 1, np.int64)
    np.add.at(counts, ids[ids >= 0], 1)
    counts[E] = live.sum()
    prob_sum = (probabilities(x, score) * live[:, None]).sum(axis=0)
    return dict(topk_ids=ids, gate=gates(x, ids, score, renorm, scale), counts=counts,
                prob_sum=prob_sum)


def balance_loss(counts, prob_sum, k, alpha):
    counts = np.asarray(counts, np.float64)
    E, n = counts.shape[0] - 1, counts[-1]
    if n == 0:
        return 0.0
    return float(alpha * E * np.sum(counts[:E] / (n * k) * np.asarray(prob_sum, np.float64) / n))


def route_bwd(logits, ids, dgate, score="softmax", renorm=True, scale=1.0, counts=None,
              alpha=0.0, dloss=1.0):
    """(dlogits [T, E] float64, magnitude [T, E]): the gradient by the chain
    rule through the scores, and the same sums with every term positive (what a
    rounding error bound scales with)."""
    x = _vals(logits)
    T, E = x.shape
    k = ids.shape[1]
    s = scores(x, score)
    there = ids >= 0
    rows = np.repeat(np.arange(T), k).reshape(T, k)
    u = np.zeros((T, k)) if dgate is None else np.where(there, np.asarray(dgate, np.float64), 0.0)
    u = u * scale
    w = _selected(s, ids)
    mag = np.abs(u)
    if renorm:
        part = _safe(w.sum(axis=1, keepdims=True))
        mag = (mag + (mag * w).sum(axis=1, keepdims=True) / part) / part
        u = np.where(there, (u - (u * w).sum(axis=1, keepdims=True) / part) / part, 0.0)
    ds, ms = np.zeros((T, E)), np.zeros((T, E))       # gradient of the scores
    np.add.at(ds, (rows[there], ids[there]), u[there])
    np.add.at(ms, (rows[there], ids[there]), mag[there])
    if counts is not None and counts[-1] > 0:
        n = float(counts[-1])
        a = dloss * alpha * E * np.asarray(counts[:E], np.float64) / (k * n * n)
        a = a[None, :] * there[:, :1]
        if score == "softmax":
            ds, ms = ds + a, ms + np.abs(a)
        else:
            total = _safe(s.sum(axis=1, keepdims=True))
            p = s / total
            ds = ds + (a - (a * p).sum(axis=1, keepdims=True)) / total * there[:, :1]
            ms = ms + (np.abs(a) + (np.abs(a) * p).sum(axis=1, keepdims=True)) / total
    if score == "softmax":
        return (s * (ds - (ds * s).sum(axis=1, keepdims=True)),
                s * (ms + (ms * s).sum(axis=1, keepdims=True)))
    z = np.exp(-np.abs(x))
    slope = z / (1 + z) ** 2
    return ds * slope, ms * slope


def sumsq(grads):
    return float(sum(np.sum(_vals(g) ** 2) for g in grads))


def clip(grads, total, max_norm):
    """(norm, clipped copies in float64)."""
    norm = float(np.sqrt(total))
    if np.isnan(norm):
        coef = np.nan
    elif np.isinf(max_norm):                 # no bound, whatever the norm
        coef = 1.0
    else:
        coef = min(1.0, max_norm / (norm + 1e-6))
    return norm, [_vals(g) * coef for g in grads]
