"""Pins of the layer norm and dropout oracle (oracle/layernorm.py): the generator's published test vectors,
torch's layer norm in 64 bits, differences for the gradients, and the mask's expectation."""
import numpy as np
import pytest

from oracle import layernorm as Ln


def test_generator_known_answers():
    """The test vectors published with the generator (Random123, philox4x32 with 10 rounds)."""
    for ctr, key, out in (
            ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        assert Ln.philox(ctr, key) == out


def test_factors():
    assert (Ln.factors(3, 5, 0.0, 1, 2) == 1).all() and (Ln.factors(3, 5, 1.0, 1, 2) == 0).all()
    assert (Ln.factors(3, 5, 2.0 ** -18, 1, 2) == 1).all()
    f = Ln.factors(200, 101, 0.25, 7, 9)
    assert set(np.unique(f)) == {0.0, 4 / 3}
    n = f.size
    assert abs((f == 0).mean() - 0.25) < 5 * (0.25 * 0.75 / n) ** 0.5
    assert (f != Ln.factors(200, 101, 0.25, 7, 10)).any() and (f != Ln.factors(200, 101, 0.25, 8, 9)).any()
    # a row's bits do not depend on how many rows there are, nor a channel's on the channels behind it in its vector
    assert np.array_equal(Ln.factors(3, 101, 0.25, 7, 9), f[:3]) and np.array_equal(Ln.factors(200, 104, 0.25, 7, 9)[:, :101], f)


def test_against_torch_in_64_bits():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(1)
    s, w, b, dy = r.standard_normal((6, 37)) + 3, r.standard_normal(37), r.standard_normal(37), r.standard_normal((6, 37))
    t = [torch.tensor(x, requires_grad=True) for x in (s, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (37,), t[1], t[2], eps=1e-3)
    y.backward(torch.tensor(dy))
    assert np.allclose(Ln.layernorm(s, w, b, 1e-3)[0], y.detach().numpy(), rtol=1e-13, atol=1e-13)
    ds, dw, db = Ln.layernorm_bwd(dy, s, w, None, 1e-3)
    for a, x in zip((ds, dw, db), t):
        assert np.allclose(a, x.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(Ln.layernorm_bwd(dy, s, w, dy, 1e-3)[0], ds + dy)


def test_gradients_by_differences():
    r = np.random.default_rng(2)
    s, w, b, dy = r.standard_normal((3, 9)), r.standard_normal(9), r.standard_normal(9), r.standard_normal((3, 9))
    ds, dw, db = Ln.layernorm_bwd(dy, s, w, None, 0.1)
    h = 1e-6
    for x, g, f in ((s, ds, lambda v: Ln.layernorm(v, w, b, 0.1)[0]), (w, dw, lambda v: Ln.layernorm(s, v, b, 0.1)[0]),
                    (b, db, lambda v: Ln.layernorm(s, w, v, 0.1)[0])):
        for i in range(x.size):
            up, dn = x.copy(), x.copy()
            up.flat[i] += h
            dn.flat[i] -= h
            assert abs(((f(up) - f(dn)) * dy).sum() / (2 * h) - g.flat[i]) < 1e-7
