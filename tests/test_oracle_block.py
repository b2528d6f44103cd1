"""Pins of the residual-block oracle (oracle/block.py) against facts fixed outside it: closed forms,
central differences, torch's own 8-bit rounding on the CPU, invariances."""
import numpy as np
import pytest

from oracle import block as Bk

GATES = ["none", "complement", "norm"]


def rnd(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def gates(seed, *shape):
    return -np.abs(rnd(seed, *shape)) - 0.01


def test_glr_closed_forms():
    # constant gate, unit input: h_t = (1 - a^t) / (1 - a)
    L, a = 130, 0.9
    g = np.full((1, L, 1, 1), np.log(a))
    O, h, st = Bk.glr_fwd(np.ones((1, L, 1, 1)), g)
    t = np.arange(1, L + 1)
    assert np.allclose(O[0, :, 0, 0], (1 - a ** t) / (1 - a), rtol=1e-13)
    assert st.shape[1] == 3 and np.allclose(st[0, :, 0, 0], [0, O[0, 63, 0, 0], O[0, 127, 0, 0]])
    # complement: a running mean with weights summing to 1, so a constant stays
    O, _, _ = Bk.glr_fwd(np.full((1, L, 1, 1), 3.0), g, np.full((1, 1, 1), 3.0), "complement")
    assert np.allclose(O, 3.0, rtol=1e-13)
    # norm: unit-variance input keeps E[h^2] = 1, since a^2 + w^2 = 1
    w, _ = Bk.glr_weight(g, "norm")
    assert np.allclose(w ** 2 + a ** 2, 1.0)
    # g = 0 sums, no weight with the other two
    z = np.zeros((1, 5, 1, 2))
    assert np.allclose(Bk.glr_fwd(np.ones((1, 5, 1, 2)), z)[1], 5.0)
    for gate in GATES[1:]:
        assert np.array_equal(Bk.glr_fwd(np.ones((1, 5, 1, 2)), z, None, gate)[0], np.zeros((1, 5, 1, 2)))


@pytest.mark.parametrize("gate", GATES)
def test_glr_reset_splits_the_sequence(gate):
    x, g, h0 = rnd(1, 2, 90, 2, 3), gates(2, 2, 90, 2, 3), rnd(3, 2, 2, 3)
    g[:, 40] = -np.inf
    O, h, _ = Bk.glr_fwd(x, g, h0, gate)
    O2, h2, _ = Bk.glr_fwd(x[:, 40:], g[:, 40:], None, gate)
    assert np.array_equal(O[:, 40:], O2) and np.array_equal(h, h2)
    x[:, :40] = np.nan     # nothing of the first part is seen after the reset
    O3, _, _ = Bk.glr_fwd(x, g, h0, gate)
    assert np.array_equal(O3[:, 40:], O2) and np.isnan(O3[:, :40]).all()


@pytest.mark.parametrize("gate", GATES)
def test_glr_gradients_against_differences(gate):
    x, g, h0 = rnd(4, 1, 7, 1, 3), gates(5, 1, 7, 1, 3), rnd(6, 1, 1, 3)
    dO, dh = rnd(7, 1, 7, 1, 3), rnd(8, 1, 1, 3)
    loss = lambda: float((Bk.glr_fwd(x, g, h0, gate)[0] * dO).sum() + (Bk.glr_fwd(x, g, h0, gate)[1] * dh).sum())
    grads = Bk.glr_bwd(x, g, h0, dO, dh, gate)
    for arr, grad in zip((x, g, h0), grads):
        for i in np.ndindex(arr.shape):
            keep, e = arr[i], 1e-6
            arr[i] = keep + e
            hi = loss()
            arr[i] = keep - e
            lo = loss()
            arr[i] = keep
            # central difference: error e^2 |f'''| / 6 + 2^-52 |f| / e, below 1e-8 here
            assert abs((hi - lo) / (2 * e) - grad[i]) < 1e-7, (gate, i)


def test_rmsnorm_and_gradients():
    s, w = rnd(9, 4, 12), 1 + 0.1 * rnd(10, 12)
    assert np.allclose(np.mean(Bk.rmsnorm(s, np.ones(12), 0.0) ** 2, axis=1), 1.0)
    assert np.allclose(Bk.rmsnorm(5.0 * s, w, 0.0), Bk.rmsnorm(s, w, 0.0))
    assert np.array_equal(Bk.rmsnorm(np.zeros((1, 12)), w, 1e-6), np.zeros((1, 12)))
    dy, ds, e = rnd(11, 4, 12), rnd(12, 4, 12), 1e-6
    dx, dw = Bk.rmsnorm_bwd(dy, s, w, ds, 1e-3)
    loss = lambda s_, w_: float((Bk.rmsnorm(s_, w_, 1e-3) * dy).sum() + (s_ * ds).sum())
    for i in np.ndindex(s.shape):
        d = np.zeros_like(s)
        d[i] = e
        assert abs((loss(s + d, w) - loss(s - d, w)) / (2 * e) - dx[i]) < 1e-7
    for j in range(12):
        d = np.zeros_like(w)
        d[j] = e
        assert abs((loss(s, w + d) - loss(s, w - d)) / (2 * e) - dw[j]) < 1e-7


def test_e4m3_is_torchs():
    torch = pytest.importorskip("torch")
    v = np.concatenate([rnd(13, 4000) * 100, np.ldexp(rnd(14, 2000), -8), np.array([0.0, 448.0, -448.0, 1.0625, 1.1875])])
    v = np.clip(v.astype(np.float32), -448, 448)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(Bk.e4m3(v), t)
    assert Bk.e4m3(460.0) == 448.0 and Bk.e4m3(-1e9) == -448.0


def test_quantise_groups():
    y = rnd(15, 3, 300)
    y[1] = 0.0
    scale, q = Bk.quantise(y, 128)
    assert scale.shape == (3, 3) and (scale[1] == 0).all() and (q[1] == 0).all()
    assert np.allclose(np.abs(q[0, :128]).max(), 448.0)
    deq = q * np.repeat(scale, [128, 128, 44], axis=1)
    assert (np.abs(deq - y) <= np.abs(y) * 2.0 ** -4 + np.repeat(scale, [128, 128, 44], axis=1) * 2.0 ** -10).all()
    assert Bk.quantise(y, 0)[0].shape == (3, 1)


def test_clip():
    gs = [np.array([3.0, 0.0]), np.array([[4.0]])]
    n, out = Bk.clip(gs, 1.0, 0.0)
    assert n == 5.0 and np.allclose(out[0], [0.6, 0]) and np.allclose(out[1], 0.8)
    n, out = Bk.clip(gs, 10.0, 1e-6)
    assert n == 5.0 and np.array_equal(out[0], gs[0])
    assert Bk.clip([np.zeros(3)], 0.0, 0.0)[0] == 0.0
