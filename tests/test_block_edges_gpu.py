"""The residual-block operators (include/delta_block.h) at the edges of their contracts: state in place over
many tiles, values whose intermediate products leave float32's range, gates above 1, NaN gates, rows that
workgroups walk over.  Oracle, inputs and bounds as in test_block_gpu.py.
"""
import numpy as np
import pytest

import test_block_gpu as T
from oracle import block as Bk
from parity import say, to_dev
from test_block_gpu import GATES, HALF, U, check, draw, half_step, host, log_gates

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402


@pytest.mark.parametrize("L", [20, 129, 5000])
def test_glr_in_place_equals_out_of_place(L):
    """h_final over h0: only a chain's first tile reads the start state, its last one overwrites it."""
    B, H, d = 2, 3, 48
    say("glr in place", L)
    x, g, h0 = (to_dev(v, "f32") for v in (draw(1, (B, L, H, d)), log_gates(2, (B, L, H, d)), draw(3, (B, H, d))))
    O, h, st = D.fwd_glr(x, g, h0, input_gate="norm", want_states=True)
    for _ in range(3):
        s = h0.clone()
        Oi, hi, sti = D.fwd_glr(x, g, s, input_gate="norm", h_final=s, want_states=True)
        assert hi is s and torch.equal(Oi, O) and torch.equal(s, h) and torch.equal(sti, st)


# ---- norm backward ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [64, 1003, 2048, 16392])
@pytest.mark.parametrize("rms,eps", [(1e14, 1e-6), (1e15, 1e-6), (1e16, 1e-6), (1e-13, 0.0), (1e-16, 0.0)])
def test_rmsnorm_bwd_large_and_tiny_rows(rms, eps, W, dtype):
    """rstd^3 leaves float32's range here, the gradient does not.  Half of the rows have dy along s, where the
    two terms cancel.  Bounds as in test_rmsnorm_bwd: relative to the sum of the terms' magnitudes."""
    N = 6
    say("rmsnorm bwd", rms, eps, W, dtype)
    s, dy = draw(200, (N, W), dtype), draw(201, (N, W), dtype)
    dy[1::2] = s[1::2]
    s = host(to_dev(s * np.float32(rms), dtype)).astype(np.float32)
    w = (1 + 0.2 * draw(202, (W,))).astype(np.float32)
    w[: W // 2] = 1.0
    dx, dw = D.layer_rmsnorm_bwd(to_dev(dy, dtype), to_dev(s, dtype), to_dev(w, "f32"), eps=eps)
    ref, rw = Bk.rmsnorm_bwd(dy, s, w, None, eps)
    S, DY, WT = (np.abs(v.astype(np.float64)) for v in (s, dy, w))
    r = 1 / np.sqrt(np.mean(S * S, axis=1, keepdims=True) + eps)
    mag = r * WT * DY + S * r ** 3 * np.mean(WT * DY * S, axis=1, keepdims=True)
    check("dx", dx, ref, (W / 64 + 24) * U * mag + half_step(ref, dtype))
    check("dweight", dw, rw, (N + W / 64 + 24) * U * np.sum(DY * S * r, axis=0) + 1e-38)


# ---- NaN gates --------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [20, 50, 300])
@pytest.mark.parametrize("gate", GATES)
def test_glr_nan_gate_reaches_everything_it_touches(gate, L, dtype):
    """One log gate is NaN: outputs and gradients are NaN exactly where the formulas' are, and every other
    channel keeps its bits.  Lane and tile routes."""
    B, H, d, t, ch = 1, 2, 16, 13, 5
    say("nan gate", gate, L, dtype)
    x, g, h0, dO, dh = draw(210, (B, L, H, d), dtype), log_gates(211, (B, L, H, d)), draw(212, (B, H, d)), \
        draw(213, (B, L, H, d), dtype), draw(214, (B, H, d))
    bad = g.copy()
    bad[0, t, 1, ch] = np.nan

    def both(gates):
        xd, gd = to_dev(x, dtype), to_dev(gates, "f32")
        O, h, st = D.fwd_glr(xd, gd, to_dev(h0, "f32"), input_gate=gate, want_states=True)
        G = D.bwd_glr(xd, gd, st, to_dev(dO, dtype), to_dev(dh, "f32"), input_gate=gate)
        return {"O": O, "h": h, "states": st, **G}

    got, want = both(bad), both(g)
    O, h, st = Bk.glr_fwd(x, bad, h0, gate)
    dx, dg, dh0 = Bk.glr_bwd(x, bad, h0, dO, dh, gate)
    for n, r in {"O": O, "h": h, "states": st, "dx": dx, "dg_log": dg, "dh0": dh0}.items():
        assert np.array_equal(np.isnan(host(got[n])), np.isnan(r)), n
        a, b = got[n].clone(), want[n].clone()
        a[..., 1, ch], b[..., 1, ch] = 0, 0
        assert torch.equal(a, b), n
    assert torch.isnan(got["dx"][0, t, 1, ch]) == (gate != "none") and torch.isnan(got["dg_log"][0, t, 1, ch])
    s = to_dev(h0, "f32")
    o = D.decode_glr(to_dev(x[:, t:t + 1], dtype), to_dev(bad[:, t:t + 1], "f32"), s, input_gate=gate)
    assert torch.isnan(o).sum() == 1 and torch.isnan(s).sum() == 1 and torch.isnan(s[0, 1, ch])


# ---- norm to 8 bits ---------------------------------------------------------------------------------

@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("W", [60, 256, 1003, 40000])
@pytest.mark.parametrize("rms,weight,eps", [(1e16, 1e25, 1e-6), (1e-18, 1e-22, 0.0), (1e3, 1e37, 1e-6)])
def test_rmsnorm_quant_products_past_float32(rms, weight, eps, W, group):
    """s times the weight leaves float32's range, y does not.  Bounds as in test_rmsnorm_quant."""
    say("quant range", rms, weight, W, group)
    s = rms * draw(240, (5, W)).astype(np.float64)
    s = s.astype(np.float32)
    w = (weight * np.exp2(draw(241, (W,)).clip(-2, 2)).astype(np.float64)).astype(np.float32)
    _, y8, sc = D.layer_rmsnorm_quant(to_dev(s, "f32"), to_dev(w, "f32"), eps=eps, group=group)
    y = Bk.rmsnorm(s, w, eps)
    scale, _ = Bk.quantise(y, group)
    rel = (W / 64 + 18) * U
    check("scale", sc, scale, rel * scale + 1e-38)
    full = np.repeat(host(sc), group or W, axis=1)[:, :W]
    check("y8 * scale", host(y8) * full, y, np.abs(y) * (2.0 ** -4 + 2 * rel) + full * 2.0 ** -10 + 1e-38)


# ---- gates above 1 ----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [20, 33, 64, 65, 128, 129, 400, 3000])
def test_glr_growing_gates_keep_a_zero_state(L, dtype):
    """g = +1 everywhere: a product of many gates is infinite, the state, and the gradient that flows back,
    stay exactly 0."""
    x, g = to_dev(draw(220, (2, L, 1, 48), dtype), dtype), torch.ones((2, L, 1, 48), device="cuda")
    zero = torch.zeros_like(x)
    for gate, xs in (("norm", x), ("none", zero), ("complement", zero)):
        say("growing", L, dtype, gate)
        O, h, st = D.fwd_glr(xs, g, input_gate=gate, want_states=True)
        assert (O == 0).all() and (h == 0).all() and (st == 0).all()
        G = D.bwd_glr(xs, g, st, zero, input_gate=gate)
        assert all((G[n] == 0).all() for n in ("dx", "dg_log", "dh0"))


def growing_bounds(x, g, h0, gate):
    """fwd_bounds of test_block_gpu for gates on both sides of 1.  There w = 1 - a with a > 1.4 carries the
    relative error of a, (2 + 2|g|) u, times a / (a - 1), and one rounding more."""
    x, g = x.astype(np.float64), g.astype(np.float64)
    w, _ = Bk.glr_weight(g, gate)
    fin = np.where(np.isneginf(g), 0.0, g)
    a, u, da = np.exp(g), np.abs(w * x), np.where(np.isneginf(g), 0.0, (2 + 2 * np.abs(fin)) * U)
    dw = np.maximum(12 * U, np.where(fin > 0.35, da * a / np.maximum(a - 1, 0.4) + U, 0.0)) \
        if gate == "complement" else np.full_like(g, 12 * U)
    M = np.abs(h0).astype(np.float64)
    E, Es, Ms = np.zeros_like(M), [np.zeros_like(M)], [M]
    for t in range(x.shape[1]):
        E = a[:, t] * (E + (da[:, t] + 2 * U) * M) + (dw[:, t] + U) * u[:, t]
        M = a[:, t] * M + u[:, t]
        E = E + U * M
        Es.append(E)
        Ms.append(M)
    return 2 * np.stack(Es, 1), np.stack(Ms, 1), dw


def burst(L, B, H, d, at, count, step, channels, resets=()):
    """Slow gates, and in `channels` from token `at` on `count` gates of +step (e^135 and more together), then as
    many that decay by e^-70 together (a product of float32's range, as the header asks).  No inputs before and in
    the burst: the state grows from 1e-30, the gradient that flows back decays from 1 and grows again, so that both
    stay in float32's range though the burst's product does not."""
    g = np.maximum(log_gates(230, (B, L, H, d)), np.float32(-1e-3))
    g[:, at:at + count, :, channels] = step
    g[:, at + count:at + 2 * count, :, channels] = -70.0 / count
    for t in resets:
        g[:, t] = -np.inf
    x, dO = draw(231, (B, L, H, d)), draw(232, (B, L, H, d))
    x[:, :at + 2 * count], dO[:, :at + 2 * count] = 0.0, 0.0
    return x, g, 1e-30 * draw(233, (B, H, d)), dO, draw(234, (B, H, d))


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("L,at,count,step,resets", [
    (290, 10, 100, 1.4, ()), (700, 100, 100, 1.4, ()), (1300, 513, 100, 1.4, (300,)), (300, 1, 5, 28.0, ()),
    (600, 250, 5, 28.0, (249, 400)), (64, 3, 5, 28.0, ()), (32, 3, 5, 28.0, ()), (3000, 1500, 300, 0.45, ()),
])
def test_glr_gates_above_one_as_given(L, at, count, step, resets, gate):
    """A burst of gates above 1 whose product leaves float32's range, and as much decay behind it, computed as
    given: within a group of tokens, a tile, across tiles; in a few channels, the others as ever."""
    say("burst", L, at, count, step, resets, gate)
    B, H, d = 2, 2, 48
    x, g, h0, dO, dh = burst(L, B, H, d, at, count, step, slice(3, 40, 4), resets)
    x[..., 0], dO[..., 0] = draw(235, (B, L, H)), draw(236, (B, L, H))       # a channel with inputs throughout
    xd, gd = to_dev(x, "f32"), to_dev(g, "f32")
    O, h, st = D.fwd_glr(xd, gd, to_dev(h0, "f32"), input_gate=gate, want_states=True)
    Or, hr, sr = Bk.glr_fwd(x, g, h0, gate)
    E, M, dw = growing_bounds(x, g, h0, gate)
    check("O", O, Or, E[:, 1:] + U * (np.abs(Or) + E[:, 1:]) + 1e-38)
    check("h_final", h, hr, E[:, -1] + 1e-38)
    check("states", st, sr, E[:, :-1:64] + 1e-38)
    G = D.bwd_glr(xd, gd, st, to_dev(dO, "f32"), to_dev(dh, "f32"), input_gate=gate)
    dx, dg, dh0 = Bk.glr_bwd(x, g, h0, dO, dh, gate)
    a, (w, sl) = np.exp(g.astype(np.float64)), Bk.glr_weight(g, gate)
    nxt = np.concatenate([g[:, 1:], np.zeros_like(g[:, :1])], 1)
    Eb, Mb, _ = growing_bounds(dO[:, ::-1], nxt[:, ::-1], dh, "none")
    Eb, Mb = Eb[:, :0:-1], Mb[:, :0:-1]
    q = np.abs(sl * x) + a * M[:, :-1]
    fin = np.abs(np.where(np.isneginf(g), 0, g))
    Eq = a * (E[:, :-1] + (4 + 2 * fin) * U * M[:, :-1]) + (24 + 4 * fin) * U * np.abs(sl * x) + 2 * U * q
    check("dx", G["dx"], dx, np.abs(w) * Eb + (dw + 2 * U) * np.abs(w) * Mb + 1e-38)
    check("dg_log", G["dg_log"], dg, Eq * (Mb + Eb) + Eb * q + 2 * U * q * Mb + 1e-38)
    check("dh0", G["dh0"], dh0, a[:, 0] * Eb[:, 0] + (4 + 2 * fin[:, 0]) * U * a[:, 0] * Mb[:, 0] + 1e-38)
    one = D.fwd_glr(xd[1:].contiguous(), gd[1:].contiguous(), to_dev(h0[1:], "f32"), input_gate=gate, want_states=True)
    assert torch.equal(one[0], O[1:]) and torch.equal(one[1], h[1:]) and torch.equal(one[2], st[1:])
    g1 = D.bwd_glr(xd[1:].contiguous(), gd[1:].contiguous(), one[2], to_dev(dO[1:], "f32"), to_dev(dh[1:], "f32"), input_gate=gate)
    assert all(torch.equal(g1[n], G[n][1:]) for n in g1)
    again = D.bwd_glr(xd, gd, st, to_dev(dO, "f32"), to_dev(dh, "f32"), input_gate=gate)
    assert all(torch.equal(again[n], G[n]) for n in again)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("L", [64, 200, 1500])
def test_glr_channels_do_not_see_each_other(L, gate):
    """Resets and gates above 1 in some channels leave every other channel's bits as they were."""
    say("channels", L, gate)
    B, H, d = 2, 1, 48
    x, g, h0, dO, dh = draw(260, (B, L, H, d)), log_gates(261, (B, L, H, d)), draw(262, (B, H, d)), draw(263, (B, L, H, d)), \
        draw(264, (B, H, d))
    other = g.copy()
    other[:, 5:60, :, 3::4] = 2.0
    other[:, 9::7, :, 1::4] = -np.inf

    def both(gates):
        xd, gd = to_dev(x, "f32"), to_dev(gates, "f32")
        O, h, st = D.fwd_glr(xd, gd, to_dev(h0, "f32"), input_gate=gate, want_states=True)
        return {"O": O, "h": h, "states": st, **D.bwd_glr(xd, gd, st, to_dev(dO, "f32"), to_dev(dh, "f32"), input_gate=gate)}

    a, b = both(g), both(other)
    for n in a:
        assert torch.equal(a[n][..., 0::2], b[n][..., 0::2]), n


# ---- rows that workgroups walk over -----------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", [(8195, 300), (65539, 24), (600, 8200), (515, 16392), (4099, 700)])
def test_rmsnorm_walks_over_rows(N, W, dtype):
    """More rows than the launch's workgroups take in one step, the last step ragged."""
    T.test_rmsnorm(N, W, dtype)
    if W != 16392:
        T.test_rmsnorm_quant(N, W, dtype, 0 if dtype == "f32" else 128)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", [(300, 16392), (600, 8200), (1500, 1003), (2051, 300), (32771, 24)])
def test_rmsnorm_bwd_walks_over_rows(N, W, dtype):
    """The same backward, where a workgroup's part of dweight holds several rows (past 16384 channels read back
    for each)."""
    T.test_rmsnorm_bwd(N, W, dtype)


def test_clip_takes_the_gradients_of_the_delta_rule():
    """The dict that bwd returns, as it is, with and without its optional gradients, and those of the mixers
    together."""
    B, L, H, d = 2, 130, 2, 64
    q, k, v = (to_dev(draw(250 + i, (B, L, H, d), "bf16"), "bf16") for i in range(3))
    k = (k.float() / k.float().norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    beta, gl = torch.rand((B, L, H), device="cuda"), -torch.rand((B, L, H), device="cuda")
    for kw in ({"g_log": gl}, {"want_dS0": False}):
        G = D.bwd(q, k, v, beta, dO=v, **kw)
        assert (G["dg_log"] is None) == ("g_log" not in kw)
        ref, outs = Bk.clip([host(t) for t in G.values() if t is not None], 0.5, 1e-6)
        n = D.clip_grads(G, 0.5)
        assert abs(float(n) - ref) <= 2 * U * ref
        for t, r in zip([t for t in G.values() if t is not None], outs):
            check("clipped", t, r, 6 * U * np.abs(r) + 1e-38)
