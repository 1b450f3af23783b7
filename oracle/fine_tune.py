"""The operators for fine-tuning a draft on its target, in float64 from exactly
widened inputs: the top logits of a row, the divergence from them with its
gradient, layer norm, and the gradients of the norms.

TEST INFRASTRUCTURE ONLY (see ``oracle/spec_verify.py``).
"""
from __future__ import annotations

import numpy as np


def log_sum_exp(x):
    """Of a vector: -inf of nothing, or of -inf alone."""
    x = np.asarray(x, dtype=np.float64)
    m = np.max(x, initial=-np.inf)
    if not np.isfinite(m):
        return float(m)
    return float(m + np.log(np.sum(np.exp(x - m))))


def top_logits(row, k: int, temperature=1.0):
    """(values [k], tokens [k], log-sum-exp) of one row [V]: the first k of a
    stable descending sort, NaN first."""
    x = np.asarray(row, dtype=np.float64)
    rank = np.where(np.isnan(x), np.inf, x)
    order = np.lexsort((np.arange(x.size), -rank, ~np.isnan(x)))[:k]
    lse = float("nan") if np.isnan(x).any() else log_sum_exp(x / temperature)
    return x[order], order, lse


def distill_row(logits, index, values, lse=None, temperature=1.0, weight=1.0):
    """(loss, gradient [V], details) of one row: the definition written out, a
    token listed twice counting with both its probabilities.  details: the
    probabilities of the list and the rest, the student's rest, and so on."""
    s = np.asarray(logits, dtype=np.float64)
    V = s.size
    # what all logits have in common changes nothing and takes digits
    top = np.max(s, initial=-np.inf)
    s = (s - (top if np.isfinite(top) else 0.0)) / temperature
    entries = [(int(i), float(t)) for i, t in zip(index, values) if 0 <= i < V]
    zero = 0.0, np.zeros(V), None
    if weight == 0.0 or (lse is not None and lse == -np.inf):
        return zero
    if lse is None and all(t == -np.inf for _, t in entries):
        return zero
    t = np.array([t for _, t in entries], dtype=np.float64) / temperature
    at = np.array([i for i, _ in entries], dtype=np.int64)
    p = np.exp(t - (log_sum_exp(t) if lse is None else float(lse)))
    r = 0.0 if lse is None else max(0.0, 1.0 - float(np.sum(p)))
    ls = log_sum_exp(s)
    if np.isnan(np.sum(p)) or (lse is not None and np.isnan(lse)) or np.isnan(s).any() or top == np.inf:
        return float("nan"), np.full(V, np.nan), dict(p=p)
    listed = np.zeros(V, dtype=bool)
    listed[at] = True
    rest = log_sum_exp(s[~listed])
    if rest == -np.inf:
        r = 0.0
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(s == -np.inf, 0.0, np.exp(s - ls))
        R = 0.0 if rest == -np.inf else float(np.exp(rest - ls))
        loss = 0.0
        for i, pj in zip(at, p):
            if pj > 0:
                loss += pj * (np.log(pj) - (s[i] - ls if s[i] != -np.inf else -np.inf))
        if r > 0:
            loss += r * (np.log(r) - (rest - ls))
    # relative to the rest's maximum: where that is far from 0, its log-sum-exp has no bits for the logarithm
    share = np.zeros(V)
    if rest > -np.inf:
        share[~listed] = np.exp(s[~listed] - np.max(s[~listed]))
        share /= np.sum(share)
    g = np.where(listed, q, share * (R - r))
    np.subtract.at(g, at, p)
    return weight * loss, weight / temperature * g, dict(p=p, r=r, q=q, R=R, share=share, listed=listed, s=s, rest=rest)


def layer_norm(x, weight=None, bias=None, residual=None, eps=1e-5):
    """float64 (out [rows, d], h [rows, d])."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    c = h - np.mean(h, axis=-1, keepdims=True)
    y = c / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, h


def norm_backward(center: bool, grad, h, weight=None, grad_residual=None, eps=1e-5):
    """float64 (grad_h [rows, d], grad_weight [d], grad_bias [d])."""
    h, dy = np.asarray(h, dtype=np.float64), np.asarray(grad, dtype=np.float64)
    c = h - np.mean(h, axis=-1, keepdims=True) if center else h
    r = 1.0 / np.sqrt(np.mean(c * c, axis=-1, keepdims=True) + eps)
    n = c * r
    g = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    dh = g - n * np.mean(g * n, axis=-1, keepdims=True)
    if center:
        dh = dh - np.mean(g, axis=-1, keepdims=True)
    dh = r * dh
    if grad_residual is not None:
        dh = dh + np.asarray(grad_residual, dtype=np.float64)
    return dh, np.sum(dy * n, axis=0), np.sum(dy, axis=0)
