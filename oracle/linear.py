"""fp64 oracle of linear attention with a decay for each head, and of its gradients.

TEST INFRASTRUCTURE ONLY (as the rest of this package).  Each function is the definition of
include/delta_linear.h written out with numpy, token by token; pinned in tests/test_oracle_linear.py.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _gates(g, B, L, H):
    """a = exp(g) as [B, L, H] from [B, L, H], [H] or None."""
    return np.ones((B, L, H)) if g is None else np.broadcast_to(np.exp(_f64(g)), (B, L, H))


def _heads(x, H):
    """The rows that each of H heads reads."""
    return np.repeat(_f64(x), H // x.shape[2], axis=2)


def states(k, v, g=None, S0=None):
    """The state before every token and behind the last, [L + 1][B, H, dk, dv]."""
    v = _f64(v)
    B, L, H, dv = v.shape
    k, a = _heads(k, H), _gates(g, B, L, H)
    S = np.zeros((B, H, k.shape[3], dv)) if S0 is None else _f64(S0)
    out = [S]
    for t in range(L):
        S = a[:, t, :, None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        out.append(S)
    return out


def flows(q, dO, g=None, dS_final=None, scale=1.0):
    """The gradient of the state behind every token, [L][B, H, dk, dv], and of the initial state."""
    dO = _f64(dO)
    B, L, H, dv = dO.shape
    q, a = _heads(q, H), _gates(g, B, L, H)
    G = np.zeros((B, H, q.shape[3], dv)) if dS_final is None else _f64(dS_final)
    out = [None] * L
    for t in reversed(range(L)):
        out[t] = G + scale * q[:, t, :, :, None] * dO[:, t, :, None, :]
        G = a[:, t, :, None, None] * out[t]
    return out, G


def fwd(q, k, v, g=None, S0=None, scale=1.0):
    """O [B, L, H, dv] and the state behind the last token."""
    S = states(k, v, g, S0)
    q = _heads(q, v.shape[2])
    O = np.zeros(v.shape)
    for t in range(v.shape[1]):
        O[:, t] = scale * np.einsum("bhc,bhcd->bhd", q[:, t], S[t + 1])
    return O, S[-1]


def bwd(q, k, v, g, S0, dO, dS_final=None, scale=1.0):
    """dict of dq, dk, dv, dg_log (as g; None without gates) and dS0."""
    B, L, H, dv = v.shape
    Hk = q.shape[2]
    S, (G, dS0) = states(k, v, g, S0), flows(q, dO, g, dS_final, scale)
    a, kh, v, dO = _gates(g, B, L, H), _heads(k, H), _f64(v), _f64(dO)
    dq, dk, dvv, dg = np.zeros(kh.shape), np.zeros(kh.shape), np.zeros(v.shape), np.zeros((B, L, H))
    for t in range(L):
        dq[:, t] = scale * np.einsum("bhcd,bhd->bhc", S[t + 1], dO[:, t])
        dk[:, t] = np.einsum("bhcd,bhd->bhc", G[t], v[:, t])
        dvv[:, t] = np.einsum("bhcd,bhc->bhd", G[t], kh[:, t])
        dg[:, t] = a[:, t] * np.einsum("bhcd,bhcd->bh", G[t], S[t])
    share = lambda x: x.reshape(B, L, Hk, H // Hk, -1).sum(3)
    if g is None:
        dg = None
    elif np.ndim(g) == 1:
        dg = dg.sum((0, 1))
    return {"dq": share(dq), "dk": share(dk), "dv": dvv, "dg_log": dg, "dS0": dS0}
