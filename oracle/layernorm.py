"""fp64 oracle of the residual stream's layer norm and of dropout from a counter-based generator.

TEST INFRASTRUCTURE ONLY (as the rest of this package).  Each function is the definition of
include/delta_layernorm.h written out with numpy; pinned in tests/test_oracle_layernorm.py.
"""
from __future__ import annotations

import numpy as np

MASK = (1 << 32) - 1


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def philox(counter, key):
    """Philox4x32-10 of one counter (four words) and key (two words), in Python integers."""
    c, k = list(counter), list(key)
    for r in range(10):
        if r:
            k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [b >> 32 ^ c[1] ^ k[0], b & MASK, a >> 32 ^ c[3] ^ k[1], a & MASK]
    return c


def factors(rows, width, p, seed, offset):
    """What dropout multiplies each element by, [rows, width]."""
    d = int(np.rint(p * 65536))
    if d == 0:
        return np.ones((rows, width))
    if d == 65536:
        return np.zeros((rows, width))
    blocks = -(-width // 8)
    bits = np.empty((rows, blocks * 8), dtype=np.int64)
    for n in range(rows * blocks):
        w = philox([n & MASK, n >> 32, offset & MASK, offset >> 32], [seed & MASK, seed >> 32])
        bits.reshape(-1, 8)[n] = [v for x in w for v in (x & 0xFFFF, x >> 16)]
    return (bits[:, :width] >= d) * (65536 / (65536 - d))


def layernorm(s, weight, bias, eps):
    """y, and the row's z and 1 / sqrt(var + eps)."""
    s = _f64(s)
    d = s - s.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    return d * r * _f64(weight) + (0.0 if bias is None else _f64(bias)), d * r, r


def layernorm_bwd(dy, s, weight, dsum, eps):
    """ds, dweight, dbias for rows [N, width]."""
    dy, weight = _f64(dy), _f64(weight)
    _, z, r = layernorm(s, weight, None, eps)
    wd = weight * dy
    ds = r * (wd - wd.mean(-1, keepdims=True) - z * (wd * z).mean(-1, keepdims=True))
    return ds + (0.0 if dsum is None else _f64(dsum)), (dy * z).sum(0), dy.sum(0)
