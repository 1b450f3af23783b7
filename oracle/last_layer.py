"""The operators between a model's last layer and the verification, in float64
from exactly widened inputs: the root-mean-square norm with the residual's
addition, the matrix product with its epilogue, and penalties, biases and
masks on logits.

TEST INFRASTRUCTURE ONLY (see ``oracle/spec_verify.py``).
"""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
FLT_MIN = 2.0 ** -126


def e4m3_values() -> np.ndarray:
    """The 256 values of e4m3 by bit pattern: sign, 4 exponent bits (bias 7), 3
    of mantissa; 0x7F and 0xFF are NaN, no infinities."""
    v = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        if (b & 0x7F) == 0x7F:
            x = math.nan
        v[b] = -x if b & 0x80 else x
    return v


def rms_norm(x, weight, residual=None, eps=1e-6):
    """float64 (out [rows, d], h [rows, d])."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    return h * np.asarray(weight, dtype=np.float64) / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps), h


def e4m3_scale(y):
    """One scale a row: max |y| / 448, at least FLT_MIN."""
    return np.maximum(np.max(np.abs(y), axis=-1) / E4M3_MAX, FLT_MIN)


_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(v, act: str):
    v = np.asarray(v, dtype=np.float64)
    if act == "none":
        return v
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0))
    z = v if act == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
    if act not in ("silu", "gelu_tanh"):
        raise ValueError(act)
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-z))


def linear(x, weight, bias=None, residual=None, act="none", x_scale=None, weight_scale=None):
    """float64 [M, N]; residual [M, R] is added at column n mod R."""
    y = np.matmul(np.asarray(x, dtype=np.float64), np.asarray(weight, dtype=np.float64).T)
    if x_scale is not None:
        y = y * np.asarray(x_scale, dtype=np.float64)[:, None] * np.asarray(weight_scale, dtype=np.float64)[None, :]
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    y = activate(y, act)
    if residual is not None:
        r = np.asarray(residual, dtype=np.float64)
        y = y + np.tile(r, (1, y.shape[1] // r.shape[1]))
    return y


def adjust_row(logits, prompt, said, repetition=1.0, frequency=0.0, presence=0.0, biases=(), allowed=None):
    """One row [V]: ``prompt`` and ``said`` (output tokens, drafts before the
    row included) are token lists, ``biases`` (token, value) pairs, ``allowed`` a
    boolean [V] or None.  Returns (row, the sum of the magnitudes of what was
    rounded on the way, for error bounds, and which logits were touched)."""
    l = np.array(logits, dtype=np.float64)
    V = l.shape[0]
    cnt = np.zeros(V)
    pr = np.zeros(V, dtype=bool)
    for t in prompt:
        if 0 <= t < V:
            pr[t] = True
    for t in said:
        if 0 <= t < V:
            cnt[t] += 1
    mag = np.zeros(V)
    hit = pr | (cnt > 0)
    with np.errstate(invalid="ignore"):
        l[hit] = np.where(l[hit] > 0, l[hit] / repetition, l[hit] * repetition)
        mag[hit] += np.abs(l[hit])
        out = cnt > 0
        l[out] -= frequency * cnt[out]
        mag[out] += np.abs(frequency * cnt[out]) + np.abs(l[out])
        l[out] -= presence
        mag[out] += np.abs(l[out])
        touched = hit.copy()
        total = {}
        for t, v in biases:
            if 0 <= t < V:
                total.setdefault(int(t), []).append(float(v))
        for t, vs in total.items():
            l[t] += sum(vs)
            mag[t] += sum(abs(v) for v in vs) * (len(vs) - 1) + abs(l[t])
            touched[t] = True
    if allowed is not None:
        l[~allowed] = -np.inf
        mag[~allowed] = 0.0
    return l, mag, touched
