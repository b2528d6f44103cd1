"""fp64 oracle of the residual-block operators: the gated linear recurrence and its gradients, the
RMS norm of the residual stream (also in 8 bits) and its gradients, gradient clipping.

TEST INFRASTRUCTURE ONLY (as the rest of this package).  Each function is the definition of
include/delta_block.h written out with numpy, token by token and row by row; pinned in
tests/test_oracle_block.py.
"""
from __future__ import annotations

import numpy as np

CHUNK = 64
E4M3_MAX = 448.0


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def glr_weight(g, gate):
    """w(g) and dw/dg (0 where w = 0)."""
    g = _f64(g)
    a = np.exp(g)
    if gate == "none":
        return np.ones_like(a), np.zeros_like(a)
    if gate == "complement":
        return -np.expm1(g), -a
    w = np.sqrt(np.maximum(-np.expm1(2 * g), 0.0))
    return w, np.where(w > 0, -a * a / np.where(w > 0, w, 1.0), 0.0)


def glr_fwd(x, g, h0=None, gate="none"):
    """x, g [B, L, H, d]; h0 [B, H, d] or None -> O, h_final, states [B, ceil(L/64), H, d]."""
    x, g = _f64(x), _f64(g)
    B, L = x.shape[:2]
    w, _ = glr_weight(g, gate)
    h = np.zeros(x.shape[:1] + x.shape[2:]) if h0 is None else _f64(h0).copy()
    O = np.empty_like(x)
    states = np.empty((B, -(-L // CHUNK)) + x.shape[2:])
    for t in range(L):
        if t % CHUNK == 0:
            states[:, t // CHUNK] = h
        reset = np.isneginf(g[:, t])
        with np.errstate(invalid="ignore"):
            h = np.where(reset, 0.0, np.exp(g[:, t]) * np.where(reset, 0.0, h)) + w[:, t] * x[:, t]
        O[:, t] = h
    return O, h, states


def glr_bwd(x, g, h0, dO, dh_final=None, gate="none"):
    """Gradients dx, dg, dh0 of <O, dO> + <h_final, dh_final>."""
    x, g, dO = _f64(x), _f64(g), _f64(dO)
    O, _, _ = glr_fwd(x, g, h0, gate)
    w, slope = glr_weight(g, gate)
    start = np.zeros(x.shape[:1] + x.shape[2:]) if h0 is None else _f64(h0)
    flow = np.zeros_like(start) if dh_final is None else _f64(dh_final).copy()
    dx, dg = np.empty_like(x), np.empty_like(x)
    for t in reversed(range(x.shape[1])):
        before = O[:, t - 1] if t else start
        reset, a = np.isneginf(g[:, t]), np.exp(g[:, t])
        lam = dO[:, t] + flow
        dx[:, t] = w[:, t] * lam
        with np.errstate(invalid="ignore"):
            dg[:, t] = np.where(reset, 0.0, lam * (a * before + slope[:, t] * x[:, t]))
            flow = np.where(reset, 0.0, a * lam)
    return dx, dg, flow


def rmsnorm(s, weight, eps):
    s = _f64(s)
    return s / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + eps) * _f64(weight)


def rmsnorm_bwd(dy, s, weight, dsum, eps):
    """dx, dweight for rows [N, width]."""
    dy, s, weight = _f64(dy), _f64(s), _f64(weight)
    r = 1.0 / np.sqrt(np.mean(s * s, axis=-1, keepdims=True) + eps)
    dx = r * weight * dy - s * r ** 3 * np.mean(weight * dy * s, axis=-1, keepdims=True)
    if dsum is not None:
        dx = dx + _f64(dsum)
    return dx, np.sum(dy * s * r, axis=0)


def e4m3(v):
    """v rounded to the nearest OCP e4m3 value (ties to even), saturating at 448."""
    v = _f64(v)
    a = np.minimum(np.abs(v), E4M3_MAX)
    _, e = np.frexp(a)                              # a = m 2^e, m in [0.5, 1)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.sign(v) * np.minimum(np.rint(a / step) * step, E4M3_MAX)


def quantise(y, group):
    """scale [N, groups] and the e4m3 values [N, width] of rows y; group 0: one scale per row."""
    y = _f64(y)
    size = group or y.shape[1]
    scale, q = [], []
    for c in range(0, y.shape[1], size):
        p = y[:, c:c + size]
        m = np.abs(p).max(axis=1)
        zero = m < 2.0 ** -100
        scale.append(np.where(zero, 0.0, m / E4M3_MAX))
        q.append(e4m3(p / np.where(zero, np.inf, m / E4M3_MAX)[:, None]))
    return np.stack(scale, axis=1), np.concatenate(q, axis=1)


def clip(grads, max_norm, eps):
    """norm and the clipped gradients."""
    n = np.sqrt(sum(float(np.sum(_f64(g) ** 2)) for g in grads))
    c = 1.0 if n + eps == 0 else min(1.0, max_norm / (n + eps))
    return n, [_f64(g) * c for g in grads]
