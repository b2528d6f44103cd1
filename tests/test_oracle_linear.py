"""Pins of the linear attention oracle (oracle/linear.py): the quadratic form, closed forms, the delta
rule's oracle where the two agree, and differences for every gradient."""
import numpy as np
import pytest

import oracle
from oracle import linear as Lo


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def case(B=2, L=7, Hk=2, H=4, dk=5, dv=3, gate="token"):
    g = {"token": -np.abs(rnd(4, B, L, H)), "head": -np.abs(rnd(5, H)), "none": None}[gate]
    return rnd(1, B, L, Hk, dk), rnd(2, B, L, Hk, dk), rnd(3, B, L, H, dv), g, rnd(6, B, H, dk, dv)


@pytest.mark.parametrize("gate", ["token", "head", "none"])
def test_quadratic_form(gate):
    q, k, v, g, S0 = case(gate=gate)
    O, S = Lo.fwd(q, k, v, g, S0, scale=0.7)
    B, L, H, _ = v.shape
    c = np.cumsum(np.zeros((B, L, H)) if g is None else np.broadcast_to(g, (B, L, H)), 1)
    for b in range(B):
        for h in range(H):
            Q, K = q[b, :, h // 2], k[b, :, h // 2]
            D = np.tril(np.exp(np.minimum(c[b, :, None, h] - c[b, None, :, h], 0)))
            ref = 0.7 * ((Q @ K.T * D) @ v[b, :, h] + np.exp(c[b, :, h])[:, None] * (Q @ S0[b, h]))
            assert np.allclose(O[b, :, h], ref, rtol=1e-12, atol=1e-12)
            w = np.exp(c[b, -1, h] - c[b, :, h])
            assert np.allclose(S[b, h], np.exp(c[b, -1, h]) * S0[b, h] + (K * w[:, None]).T @ v[b, :, h], rtol=1e-12, atol=1e-12)


def test_running_sums_without_gates():
    q, k, v, _, _ = case(Hk=1, H=1)
    O, S = Lo.fwd(np.ones_like(q), k, v)
    assert np.allclose(S[0, 0], k[0, :, 0].T @ v[0, :, 0])
    assert np.allclose(O[0, :, 0], np.cumsum(k[0, :, 0].sum(1)[:, None] * v[0, :, 0], 0))


def test_reset_and_no_tokens():
    q, k, v, g, S0 = case()
    g[:, 4] = -np.inf
    O, S = Lo.fwd(q, k, v, g, S0)
    O2, S2 = Lo.fwd(q[:, 4:], k[:, 4:], v[:, 4:], g[:, 4:], 100 * S0)
    assert np.array_equal(O[:, 4:], O2) and np.array_equal(S, S2)
    assert np.array_equal(Lo.fwd(q[:, :0], k[:, :0], v[:, :0], g[:, :0], S0)[1], S0)


def test_delta_rule_with_orthonormal_keys():
    """With beta = 1, orthonormal keys and no start state the delta rule erases nothing."""
    L, d = 6, 16
    Q = np.linalg.qr(rnd(9, d, d))[0][:L].astype(np.float32)
    q, k, v = rnd(10, 1, L, 1, d).astype(np.float32), Q[None, :, None], rnd(11, 1, L, 1, 8).astype(np.float32)
    g = -np.abs(rnd(12, 1, L, 1)).astype(np.float32)
    Or, Sr = oracle.fwd(q, k, v, np.ones((1, L, 1), np.float32), g, None)
    O, S = Lo.fwd(q, k, v, g)
    assert np.abs(O - Or).max() < 1e-6 and np.abs(S - Sr).max() < 1e-6   # float32 keys are orthonormal to 1e-7


@pytest.mark.parametrize("gate", ["token", "head", "none"])
def test_gradients_by_differences(gate):
    q, k, v, g, S0 = case(gate=gate)
    dO, dS = rnd(7, *v.shape), rnd(8, *S0.shape)
    got = Lo.bwd(q, k, v, g, S0, dO, dS, scale=0.7)

    def loss(**kw):
        a = dict(q=q, k=k, v=v, g=g, S0=S0)
        a.update(kw)
        O, S = Lo.fwd(a["q"], a["k"], a["v"], a["g"], a["S0"], scale=0.7)
        return (O * dO).sum() + (S * dS).sum()

    h = 1e-5
    for name, key in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg_log"), ("S0", "dS0")):
        x = {"q": q, "k": k, "v": v, "g": g, "S0": S0}[name]
        if x is None:
            assert got[key] is None
            continue
        for i in np.random.default_rng(3).choice(x.size, min(12, x.size), replace=False):
            up, dn = x.copy(), x.copy()
            up.flat[i] += h
            dn.flat[i] -= h
            d = (loss(**{name: up}) - loss(**{name: dn})) / (2 * h)
            assert abs(d - got[key].flat[i]) <= 1e-7 * (1 + abs(d)), (name, i)


def test_one_token_by_hand():
    q, k, v, g, S0 = case(B=1, L=1, Hk=1, H=1)
    dO, dS = rnd(7, *v.shape), rnd(8, *S0.shape)
    r = Lo.bwd(q, k, v, g, S0, dO, dS, scale=2.0)
    a, Q, K, V, o = np.exp(g[0, 0, 0]), q[0, 0, 0], k[0, 0, 0], v[0, 0, 0], dO[0, 0, 0]
    G = dS[0, 0] + 2.0 * np.outer(Q, o)
    S = a * S0[0, 0] + np.outer(K, V)
    for key, ref in (("dq", 2.0 * S @ o), ("dk", G @ V), ("dv", G.T @ K), ("dg_log", a * (G * S0[0, 0]).sum()), ("dS0", a * G)):
        assert np.allclose(r[key].ravel(), np.ravel(ref), rtol=1e-12, atol=1e-12), key
