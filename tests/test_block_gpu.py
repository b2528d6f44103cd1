"""GPU parity of the residual-block operators (include/delta_block.h) with the fp64 oracle in
oracle/block.py.

Tolerances are elementwise and derived from the arithmetic, with u = 2^-24 the float32 half step:
  * gated linear recurrence: a = exp(g) carries a relative error da = (2 + 2|g|) u (an exp2 good to a
    unit in the last place, and the rounding of its argument g log2 e), w at most dw = 12 u (the
    series, or 1 - a with a < 0.71; half of it under the root).  Both are run through the recurrence
    next to M_t = a M_{t-1} + |u_t|, the sum of magnitudes: E_t = a (E_{t-1} + (da + 2u) M_{t-1}) +
    (dw + u) |u_t| + u M_t.  Chunked evaluation re-associates the same products and sums: twice E.
    The backward bound is the same recurrence from the other end, multiplied out.
  * norms: a sum of D squares held in 64 or more partial sums: (D / 64 + 16) u relative.
  * the outputs' own rounding: half a step of their type, eps / 2 relative.
"""
import numpy as np
import pytest

from oracle import block as Bk
from parity import say, to_dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
GATES = ["none", "complement", "norm"]
TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def draw(seed, shape, dtype="f32"):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x


def log_gates(seed, shape, resets=()):
    """Log gates from -9 to -1e-4 (fast and slow channels), -inf at the tokens of `resets`."""
    r = np.random.default_rng(seed)
    g = -np.exp(r.uniform(np.log(1e-4), np.log(9.0), shape)).astype(np.float32)
    for t in resets:
        g[:, t] = -np.inf
    return g


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(name, got, ref, tol):
    got = host(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.size:
        return
    with np.errstate(divide="ignore", invalid="ignore"):
        over = np.nan_to_num(np.abs(got - ref) / tol, nan=np.inf, posinf=np.inf)
    over[(got == ref) | (np.isnan(got) & np.isnan(ref))] = 0.0
    say("  %s: max error / bound %.3f, max |ref| %.3g" % (name, over.max(), np.abs(np.nan_to_num(ref)).max()))
    assert over.max() <= 1.0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def fwd_bounds(x, g, h0, gate):
    """(E, M) after every token, and at the sequence start: [B, L + 1, H, d]."""
    x, g = x.astype(np.float64), g.astype(np.float64)
    w, _ = Bk.glr_weight(g, gate)
    a, u = np.exp(g), np.abs(w * x)
    da = np.where(np.isneginf(g), 0.0, (2 + 2 * np.abs(np.where(np.isneginf(g), 0.0, g))) * U)
    M = np.abs(h0).astype(np.float64) if h0 is not None else np.zeros_like(x[:, 0])
    E = np.zeros_like(M)
    Es, Ms = [E], [M]
    for t in range(x.shape[1]):
        E = a[:, t] * (E + (da[:, t] + 2 * U) * M) + 13 * U * u[:, t]
        M = a[:, t] * M + u[:, t]
        E = E + U * M
        Es.append(E)
        Ms.append(M)
    return 2 * np.stack(Es, 1), np.stack(Ms, 1)


GLR_CASES = [
    # B, L, H, d, dtype, resets
    (1, 1, 1, 16, "f32", ()), (2, 3, 1, 16, "bf16", ()), (1, 15, 3, 48, "f32", (0,)), (2, 16, 2, 16, "bf16", (15,)),
    (1, 17, 5, 48, "bf16", (16,)), (3, 63, 1, 80, "f32", (31, 32)), (1, 64, 2, 128, "bf16", (63,)),
    (2, 65, 3, 16, "f32", (64,)), (1, 127, 1, 256, "bf16", (0, 64)), (2, 128, 1, 112, "bf16", ()),
    (1, 129, 7, 16, "f32", (128,)), (1, 255, 2, 128, "bf16", (254,)), (2, 256, 1, 64, "f32", (255,)),
    (1, 257, 3, 48, "bf16", (256, 128)), (1, 511, 1, 16, "f32", ()), (1, 1025, 1, 32, "bf16", (1024, 512, 3)),
    (3, 1237, 5, 48, "f32", (100, 640)), (2, 4099, 1, 144, "bf16", (4096, 4000)), (1, 9000, 2, 16, "bf16", ()),
    (5, 700, 9, 16, "bf16", (256, 511)),
]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("case", GLR_CASES, ids=lambda c: "x".join(map(str, c[:4])) + c[4])
def test_glr(case, gate):
    B, L, H, d, dtype, resets = case
    say("glr", case, gate)
    x, g, h0 = draw(1, (B, L, H, d), dtype), log_gates(2, (B, L, H, d), resets), draw(3, (B, H, d))
    dO, dh = draw(4, (B, L, H, d), dtype), draw(5, (B, H, d))
    xd, gd, hd = to_dev(x, dtype), to_dev(g, "f32"), to_dev(h0, "f32")
    O, h, st = D.fwd_glr(xd, gd, hd, input_gate=gate, want_states=True)
    G = D.bwd_glr(xd, gd, st, to_dev(dO, dtype), to_dev(dh, "f32"), input_gate=gate)
    torch.cuda.synchronize()
    Or, hr, sr = Bk.glr_fwd(x, g, h0, gate)
    E, M = fwd_bounds(x, g, h0, gate)
    check("O", O, Or, E[:, 1:] + HALF[dtype] * (np.abs(Or) + E[:, 1:]) + 1e-38)
    check("h_final", h, hr, E[:, -1] + 1e-38)
    check("states", st, sr, E[:, :-1:64] + 1e-38)
    dx, dg, dh0 = Bk.glr_bwd(x, g, h0, dO, dh, gate)
    # lambda's bound: the recurrence run from the other end over the gates shifted by one token
    a, (w, sl) = np.exp(g.astype(np.float64)), Bk.glr_weight(g, gate)
    nxt = np.concatenate([g[:, 1:], np.zeros_like(g[:, :1])], 1)
    Eb, Mb = fwd_bounds(dO[:, ::-1], nxt[:, ::-1], dh, "none")
    Eb, Mb = Eb[:, :0:-1], Mb[:, :0:-1]
    q = np.abs(sl * x) + a * M[:, :-1]
    Eq = a * (E[:, :-1] + (2 + 2 * np.abs(np.where(np.isneginf(g), 0, g)) + 2) * U * M[:, :-1]) + 24 * U * np.abs(sl * x) \
        + 2 * U * q
    check("dx", G["dx"], dx, w * Eb + 14 * U * w * Mb + 1e-38)
    check("dg_log", G["dg_log"], dg, Eq * (Mb + Eb) + Eb * q + 2 * U * q * Mb + 1e-38)
    a0 = a[:, 0]
    check("dh0", G["dh0"], dh0, a0 * Eb[:, 0] + (4 + 2 * np.abs(np.where(np.isneginf(g[:, 0]), 0, g[:, 0]))) * U * a0 * Mb[:, 0] + 1e-38)


@pytest.mark.parametrize("gate", GATES)
def test_glr_defaults_and_optional_outputs(gate):
    B, L, H, d = 2, 300, 2, 32
    x, g = draw(11, (B, L, H, d)), log_gates(12, (B, L, H, d))
    xd, gd = to_dev(x, "f32"), to_dev(g, "f32")
    O, h, st = D.fwd_glr(xd, gd, input_gate=gate, want_state=False)
    assert h is None and st is None
    O2, h2, st2 = D.fwd_glr(xd, gd, to_dev(np.zeros((B, H, d)), "f32"), input_gate=gate, want_states=True)
    assert torch.equal(O, O2)
    # the states and the outputs at the same tokens are two evaluations of one value, each within E of it
    E, _ = fwd_bounds(x, g, None, gate)
    check("h_final", h2, host(O2[:, -1]), 2 * E[:, -1] + 1e-38)
    check("states", st2[:, 1:], host(O2[:, 63:L - 1:64]), 2 * E[:, 64:L:64] + 1e-38)
    dO = to_dev(draw(13, (B, L, H, d)), "f32")
    g1 = D.bwd_glr(xd, gd, st2, dO, input_gate=gate, want_dh0=False)
    g2 = D.bwd_glr(xd, gd, st2, dO, to_dev(np.zeros((B, H, d)), "f32"), input_gate=gate)
    assert g1["dh0"] is None and torch.equal(g1["dx"], g2["dx"]) and torch.equal(g1["dg_log"], g2["dg_log"])


def test_glr_in_place_and_split_over_calls():
    """A sequence in two calls, the state carried in place, equals one call within the bound; the same
    call again gives the same bits."""
    B, L, H, d = 2, 1000, 3, 48
    x, g, h0 = draw(14, (B, L, H, d), "bf16"), log_gates(15, (B, L, H, d)), draw(16, (B, H, d))
    xd, gd, st = to_dev(x, "bf16"), to_dev(g, "f32"), to_dev(h0, "f32")
    O, h, _ = D.fwd_glr(xd, gd, st, input_gate="norm")
    again = D.fwd_glr(xd, gd, st, input_gate="norm")
    assert torch.equal(O, again[0]) and torch.equal(h, again[1])
    k = 333
    Oa, ha, _ = D.fwd_glr(xd[:, :k].contiguous(), gd[:, :k].contiguous(), st, input_gate="norm", h_final=st)
    assert ha.data_ptr() == st.data_ptr()
    Ob, hb, _ = D.fwd_glr(xd[:, k:].contiguous(), gd[:, k:].contiguous(), st, input_gate="norm", h_final=st)
    Or, hr, _ = Bk.glr_fwd(x, g, h0, "norm")
    E, _ = fwd_bounds(x, g, h0, "norm")
    check("O", torch.cat([Oa, Ob], 1), Or, E[:, 1:] + HALF["bf16"] * (np.abs(Or) + E[:, 1:]) + 1e-38)
    check("h", hb, hr, E[:, -1] + 1e-38)


def test_glr_empty():
    for B, L, H in ((0, 5, 2), (2, 5, 0), (2, 0, 3)):
        x = torch.empty((B, L, H, 16), device="cuda")
        h0 = torch.randn((B, H, 16), device="cuda")
        O, h, st = D.fwd_glr(x, x, h0, want_states=True)
        assert O.shape == x.shape and torch.equal(h, h0) or B * H == 0
        assert st.shape == (B, -(-L // 64), H, 16)
        G = D.bwd_glr(x, x, st, x, h0)
        torch.cuda.synchronize()
        if L == 0:
            assert torch.equal(G["dh0"], h0)
            assert torch.equal(D.fwd_glr(x, x)[1], torch.zeros_like(h0))


@pytest.mark.parametrize("gate", GATES)
def test_glr_resets_hide_what_is_before_and_behind(gate):
    """NaN and infinities before a reset are not seen after it, in the outputs; nor, in the gradients,
    those after it by what is before it.  Every gate -inf: each token stands alone."""
    B, L, H, d, t = 2, 700, 1, 48, 321
    x, g = draw(17, (B, L, H, d), "bf16"), log_gates(18, (B, L, H, d), (t,))
    dO = draw(19, (B, L, H, d), "bf16")
    bad, badO = x.copy(), dO.copy()
    bad[:, 5], bad[:, 300] = np.nan, np.inf
    badO[:, t + 3] = np.nan
    gd = to_dev(g, "f32")
    O, h, st = D.fwd_glr(to_dev(x, "bf16"), gd, input_gate=gate, want_states=True)
    Ob, hb, stb = D.fwd_glr(to_dev(bad, "bf16"), gd, input_gate=gate, want_states=True)
    assert torch.equal(O[:, t:], Ob[:, t:]) and torch.equal(h, hb) and torch.isnan(Ob[:, 5:t]).all()
    G = D.bwd_glr(to_dev(x, "bf16"), gd, st, to_dev(dO, "bf16"), input_gate=gate)
    Gb = D.bwd_glr(to_dev(x, "bf16"), gd, st, to_dev(badO, "bf16"), input_gate=gate)
    for n in ("dx", "dg_log"):
        assert torch.equal(G[n][:, :t], Gb[n][:, :t]), n
    assert (G["dg_log"][:, t] == 0).all() and torch.equal(G["dh0"], Gb["dh0"])
    alone = torch.full((B, L, H, d), -float("inf"), device="cuda")
    xd = to_dev(bad, "bf16")
    O, h, st = D.fwd_glr(xd, alone, torch.full((B, H, d), float("nan"), device="cuda"), input_gate=gate, want_states=True)
    assert torch.equal(O.view(torch.int16), xd.view(torch.int16)) or torch.equal(torch.nan_to_num(O), torch.nan_to_num(xd))
    G = D.bwd_glr(xd, alone, st, to_dev(dO, "bf16"), torch.full((B, H, d), 2.0, device="cuda"), input_gate=gate)
    assert torch.equal(G["dx"][:, :-1], to_dev(dO, "f32")[:, :-1]) and (G["dg_log"] == 0).all() and (G["dh0"] == 0).all()


def test_glr_open_gates():
    """g = 0: a = 1; sums with weight 1, nothing with the other two, and their slope taken as 0 (norm)
    or -1 (complement)."""
    x = to_dev(draw(20, (1, 200, 1, 16)), "f32")
    g = torch.zeros_like(x)
    O, h, st = D.fwd_glr(x, g, want_states=True)
    # 200 additions of float32 values in some order: 200 u of the sum of magnitudes
    ref, mag = host(x).cumsum(1), np.abs(host(x)).cumsum(1)
    check("O", O, ref, 200 * U * mag)
    h0 = to_dev(draw(21, (1, 1, 16)), "f32")
    for gate in ("complement", "norm"):
        O, h, st = D.fwd_glr(x, g, h0, input_gate=gate, want_states=True)
        assert torch.equal(O, h0[:, None].expand_as(O))
        G = D.bwd_glr(x, g, st, torch.ones_like(x), input_gate=gate)
        assert (G["dx"] == 0).all() and torch.isfinite(G["dg_log"]).all()
        n = torch.arange(200, 0, -1, device="cuda").float().view(1, 200, 1, 1)
        assert torch.equal(G["dh0"], torch.full_like(h0, 200.0))
        want = n * (h0[:, None] - (x if gate == "complement" else 0))
        assert torch.allclose(G["dg_log"], want, rtol=4 * 2.0 ** -23, atol=200 * 4 * 2.0 ** -23)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("B,H,d,dtype", [(1, 1, 16, "bf16"), (3, 5, 48, "f32"), (64, 16, 128, "bf16"), (7, 3, 208, "bf16")])
def test_glr_decode_continues_a_prefill(B, H, d, dtype, gate):
    L, T = 70, 5
    x, g, h0 = draw(22, (B, L + T, H, d), dtype), log_gates(23, (B, L + T, H, d), (L + 2,)), draw(24, (B, H, d))
    xd, gd = to_dev(x, dtype), to_dev(g, "f32")
    O, h, _ = D.fwd_glr(xd[:, :L].contiguous(), gd[:, :L].contiguous(), to_dev(h0, "f32"), input_gate=gate)
    outs = [O]
    for t in range(L, L + T):
        outs.append(D.decode_glr(xd[:, t:t + 1].contiguous(), gd[:, t:t + 1].contiguous(), h, input_gate=gate))
    torch.cuda.synchronize()
    Or, hr, _ = Bk.glr_fwd(x, g, h0, gate)
    E, _ = fwd_bounds(x, g, h0, gate)
    check("O", torch.cat(outs, 1), Or, E[:, 1:] + HALF[dtype] * (np.abs(Or) + E[:, 1:]) + 1e-38)
    check("h", h, hr, E[:, -1] + 1e-38)


def test_glr_offsets_past_32_bits():
    """2.3e9 elements: the last sequence's results equal a call on it alone, bit for bit."""
    B, L, H, d = 17, 65536, 16, 128
    x = torch.empty((B, L, H, d), dtype=torch.bfloat16, device="cuda").normal_()
    g = torch.empty((B, L, H, d), device="cuda").uniform_(-0.5, -0.001)
    O, h, st = D.fwd_glr(x, g, want_states=True)
    O1, h1, st1 = D.fwd_glr(x[-1:], g[-1:], want_states=True)
    assert torch.equal(O[-1:], O1) and torch.equal(h[-1:], h1) and torch.equal(st[-1:], st1)
    del O, O1
    G = D.bwd_glr(x, g, st, x)
    G1 = D.bwd_glr(x[-1:], g[-1:], st1, x[-1:])
    for n in ("dx", "dg_log", "dh0"):
        assert torch.equal(G[n][-1:], G1[n]), n


# ---- norm of the residual stream -------------------------------------------------------------------

ROWS = [(1, 1), (1, 16), (3, 7), (5, 63), (2, 64), (17, 100), (4, 128), (64, 129), (9, 512), (1, 1000), (33, 1003), (6, 2048),
        (257, 300), (3, 4096), (2, 4104), (5, 8192), (1, 8200), (2, 16384), (1, 16392), (2, 20001), (1, 40000), (3000, 24)]


def half_step(v, dtype):
    """Half a step of dtype at v (its subnormals' at least)."""
    return HALF[dtype] * np.abs(v) + 1e-38


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_rmsnorm(N, W, dtype):
    say("rmsnorm", N, W, dtype)
    x, r = draw(31, (N, W), dtype), 2 * draw(32, (N, W), dtype)
    w = (1 + 0.2 * draw(33, (W,))).astype(np.float32)
    x[0] = 0.0
    r[0] = 0.0                                           # a row of zeros
    xd, rd, wd = to_dev(x, dtype), to_dev(r, dtype), to_dev(w, "f32")
    s, y = D.layer_rmsnorm(xd, wd, rd, eps=1e-5)
    assert torch.equal(s, xd + rd)                       # one float32 sum, rounded once
    ref = Bk.rmsnorm(host(s), w, 1e-5)
    rel = (W / 64 + 16) * U
    check("y", y, ref, rel * np.abs(ref) + half_step(ref, dtype) * (1 + rel))
    s0, y0 = D.layer_rmsnorm(s, wd, eps=1e-5)            # no residual: x itself, the same bits
    assert s0 is s and torch.equal(y0, y)
    r2 = rd.clone()
    s2, y2 = D.layer_rmsnorm(xd, wd, r2, eps=1e-5, sum=r2)
    assert s2 is r2 and torch.equal(s2, s) and torch.equal(y2, y)
    x2 = xd.clone()
    s3, y3 = D.layer_rmsnorm(x2, wd, rd, eps=1e-5, sum=x2)
    assert torch.equal(s3, s) and torch.equal(y3, y)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_rmsnorm_quant(N, W, dtype, group):
    say("rmsnorm quant", N, W, dtype, group)
    x, r = draw(41, (N, W), dtype), 2 * draw(42, (N, W), dtype)
    w = (1 + 0.2 * draw(43, (W,))).astype(np.float32)
    x[0], r[0] = 0.0, 0.0
    s, y8, sc = D.layer_rmsnorm_quant(to_dev(x, dtype), to_dev(w, "f32"), to_dev(r, dtype), eps=1e-5, group=group)
    assert torch.equal(s, to_dev(x, dtype) + to_dev(r, dtype))
    y = Bk.rmsnorm(host(s), w, 1e-5)
    scale, q = Bk.quantise(y, group)
    rel = (W / 64 + 18) * U
    check("scale", sc, scale, rel * scale + 1e-38)
    size = group or W
    full = np.repeat(host(sc), size, axis=1)[:, :W]
    got = host(y8) * full
    # e4m3: half a step is 2^-4 of the value, or 2^-10 (half its smallest step) below 2^-6
    check("y8 * scale", got, y, np.abs(y) * (2.0 ** -4 + 2 * rel) + full * 2.0 ** -10 + 1e-38)
    assert (sc[0] == 0).all() and (y8[0].float() == 0).all()
    # where float32 leaves no doubt about the rounding the value is the oracle's
    lo, hi = Bk.e4m3(y / np.where(full > 0, full, 1) * (1 - 4 * rel)), Bk.e4m3(y / np.where(full > 0, full, 1) * (1 + 4 * rel))
    sure = lo == hi
    assert sure.mean() > 0.9 and np.array_equal(host(y8)[sure], lo[sure])
    s0, y80, sc0 = D.layer_rmsnorm_quant(s, to_dev(w, "f32"), eps=1e-5, group=group)
    assert s0 is s and torch.equal(y80.view(torch.uint8), y8.view(torch.uint8)) and torch.equal(sc0, sc)


def test_rmsnorm_quant_extremes():
    W = 384
    x = np.ones((5, W), dtype=np.float32)
    w = np.ones(W, dtype=np.float32)
    w[128:256] = 0.0                                     # a group of zeros
    w[256:] = 1e-36                                      # below what counts
    x[1, 3], x[2, 300] = np.nan, np.inf
    x[3, 5] = 1e19                                       # squares to 1e38: still finite
    xd, wd = to_dev(x, "f32"), to_dev(w, "f32")
    _, y8, sc = D.layer_rmsnorm_quant(xd, wd, group=128)
    v, sc = host(y8), host(sc)
    assert (sc[0, 1:] == 0).all() and (v[0, 128:] == 0).all() and (v[0, :128] == 448).all()
    assert np.isnan(sc[1]).all() or np.isnan(v[1, :128] * sc[1, 0]).all()
    assert not np.isfinite(v[2] * np.repeat(sc[2], 128))[256:].any()   # infinity / infinity
    assert v[3, 5] == 448 and abs(sc[3, 0] - np.sqrt(W) / 448) < 1e-5
    assert np.isfinite(v[4]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_rmsnorm_bwd(N, W, dtype):
    say("rmsnorm bwd", N, W, dtype)
    s, dy, ds = 2 * draw(51, (N, W), dtype), draw(52, (N, W), dtype), draw(53, (N, W), dtype)
    w = (1 + 0.2 * draw(54, (W,))).astype(np.float32)
    eps = 1e-4
    dev = [to_dev(dy, dtype), to_dev(s, dtype), to_dev(w, "f32"), to_dev(ds, dtype)]
    dx, dw = D.layer_rmsnorm_bwd(*dev, eps=eps)
    ref, rw = Bk.rmsnorm_bwd(dy, s, w, ds, eps)
    S, DY, WT = (np.abs(v.astype(np.float64)) for v in (s, dy, w))
    r = 1 / np.sqrt(np.mean(S * S, axis=1, keepdims=True) + eps)
    mag = np.abs(ds) + r * WT * DY + S * r ** 3 * np.mean(WT * DY * S, axis=1, keepdims=True)
    rel = (W / 64 + 24) * U
    check("dx", dx, ref, rel * mag + half_step(ref, dtype))
    # dweight: a sum over N rows in float32, in any order
    check("dweight", dw, rw, (N + W / 64 + 24) * U * np.sum(DY * S * r, axis=0) + 1e-38)
    dx2, dw2 = D.layer_rmsnorm_bwd(*dev, eps=eps)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    dx3, dw3 = D.layer_rmsnorm_bwd(*dev, eps=eps, want_dweight=False)
    assert dw3 is None and torch.equal(dx, dx3)
    dx4, _ = D.layer_rmsnorm_bwd(*dev[:3], eps=eps)      # no residual gradient
    check("dx without dsum", dx4, ref - ds, rel * mag + half_step(ref - ds, dtype))


def test_rmsnorm_no_rows():
    x, w = torch.empty((0, 32), device="cuda"), torch.ones(32, device="cuda")
    assert D.layer_rmsnorm(x, w)[1].shape == (0, 32)
    dx, dw = D.layer_rmsnorm_bwd(x, x, w)
    assert dx.shape == (0, 32) and torch.equal(dw, torch.zeros_like(w))


# ---- gradient norm and clipping --------------------------------------------------------------------

@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f32", "bf16")])
@pytest.mark.parametrize("sizes", [[1], [0, 5], [7, 0, 1023, 65], [16384, 16385, 3], [5000] * 300, [1 << 22, 17, 999999]],
                         ids=lambda s: "%dx%d" % (len(s), max(s)))
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(sizes, dtypes, max_norm):
    say("clip", len(sizes), dtypes, max_norm)
    dts = [dtypes[i % len(dtypes)] for i in range(len(sizes))]
    gs = [0.1 * draw(60 + i % 7, (n,), dt) for i, (n, dt) in enumerate(zip(sizes, dts))]
    gs = [to_dev(g, dt) for g, dt in zip(gs, dts)]
    ref, outs = Bk.clip([host(g) for g in gs], max_norm, 1e-6)
    n0 = D.grad_norm(gs)
    out = [torch.full_like(g, 7.0) for g in gs]
    keep = [g.clone() for g in gs]
    n1 = D.clip_grads(gs, max_norm, out=out)
    assert torch.equal(n0, n1) and abs(float(n1) - ref) <= 2 * U * ref
    for i, (g, o, r) in enumerate(zip(gs, out, outs)):
        assert torch.equal(g, keep[i])
        if g.numel():
            check("out %d" % i, o, r, 5 * U * np.abs(r) + half_step(r, dts[i])) if i < 4 else None
            if max_norm > 1e8:
                assert torch.equal(o, g)
    n2 = D.clip_grads({str(i): g for i, g in enumerate(gs)}, max_norm)      # in place, from a dict
    assert torch.equal(n1, n2) and all(torch.equal(g, o) for g, o in zip(gs, out))


def test_clip_unaligned_views():
    """Gradients that are slices of one flat buffer: aligned to their element only."""
    for dt in ("f32", "bf16"):
        flat, o = to_dev(draw(70, (100003,), dt), dt), to_dev(draw(71, (100003,), dt), dt)
        cuts = [1, 2, 5, 9, 40000, 40001, 99998]
        gs, outs = [flat[a:b] for a, b in zip(cuts, cuts[1:])], [o[a + 1:b + 1] for a, b in zip(cuts, cuts[1:])]
        before = o.clone()
        ref, rs = Bk.clip([host(g) for g in gs], 1.0, 1e-6)
        n = D.clip_grads(gs, 1.0, out=outs)
        assert abs(float(n) - ref) <= 2 * U * ref
        for i, (a, r) in enumerate(zip(outs, rs)):
            check("out %d" % i, a, r, 5 * U * np.abs(r) + half_step(r, dt))
        assert torch.equal(o[:2], before[:2]) and torch.equal(o[99999:], before[99999:])   # nothing past the ends
        D.clip_grads(gs, 1.0)
        assert all(torch.equal(g, a) for g, a in zip(gs, outs))


def test_clip_extreme_values():
    big = torch.full((1000,), 1e30, device="cuda")       # squares past float32
    n = D.grad_norm([big])
    assert abs(float(n) - 1e30 * np.sqrt(1000)) <= 1e24 * 4
    for bad in (float("nan"), float("inf")):
        g = [torch.ones(10, device="cuda"), torch.tensor([1.0, bad], device="cuda")]
        n = D.clip_grads(g, 1.0)
        assert not torch.isfinite(n) and (torch.isnan(g[0]).all() if bad != bad else (g[0] == 0).all())
    z = [torch.zeros(5, device="cuda")]
    assert float(D.clip_grads(z, 0.0, eps=0.0)) == 0.0 and (z[0] == 0).all()
    g = [torch.ones(4, device="cuda")]
    D.clip_grads(g, 0.0)
    assert (g[0] == 0).all()
    with pytest.raises(D.DeltaError):
        D.clip_grads([g[0], g[0]], 1.0)                   # listed twice
    with pytest.raises(ValueError):
        D.clip_grads(g, 1.0, out=[torch.ones(5, device="cuda")])


# ---- graphs, streams, refusals ---------------------------------------------------------------------

def calls():
    """One call of each operator over preallocated outputs: {name: (call, outputs)}."""
    B, L, H, d = 2, 1500, 3, 48
    x, g, h0 = to_dev(draw(80, (B, L, H, d)), "bf16"), to_dev(log_gates(81, (B, L, H, d), (700,)), "f32"), to_dev(draw(82, (B, H, d)), "f32")
    dO = to_dev(draw(83, (B, L, H, d)), "bf16")
    O, hf, st = torch.empty_like(x), torch.empty_like(h0), torch.empty((B, 24, H, d), device="cuda")
    st0 = D.fwd_glr(x, g, h0, input_gate="norm", want_states=True)[2]
    G = {"dx": torch.empty_like(g), "dg_log": torch.empty_like(g), "dh0": torch.empty_like(h0)}
    w1 = torch.empty(max(1, D.glr_workspace_bytes(B, L, H, d)), dtype=torch.uint8, device="cuda")
    w2 = torch.empty(max(1, D.bwd_glr_workspace_bytes(B, L, H, d)), dtype=torch.uint8, device="cuda")
    N, W = 700, 1000
    s, r, w = to_dev(draw(84, (N, W)), "bf16"), to_dev(draw(85, (N, W)), "bf16"), to_dev(1 + 0.1 * draw(86, (W,)), "f32")
    so, y, y8, sc = torch.empty_like(s), torch.empty_like(s), torch.empty((N, W), dtype=torch.float8_e4m3fn, device="cuda"), \
        torch.empty((N, 8), device="cuda")
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    w3 = torch.empty(D.rmsnorm_bwd_workspace_bytes(N, W), dtype=torch.uint8, device="cuda")
    gs = [to_dev(draw(87, (n,)), "f32") for n in (5, 70000, 999)]
    out, norm = [torch.empty_like(t) for t in gs], torch.empty((), device="cuda")
    w4 = torch.empty(4096, dtype=torch.uint8, device="cuda")
    return {
        "fwd_glr": (lambda **k: D.fwd_glr(x, g, h0, input_gate="norm", O=O, h_final=hf, states=st, workspace=w1, **k), [O, hf, st]),
        "bwd_glr": (lambda **k: D.bwd_glr(x, g, st0, dO, h0, input_gate="norm", grads=G, workspace=w2, **k), list(G.values())),
        "rmsnorm": (lambda **k: D.layer_rmsnorm(s, w, r, sum=so, y=y, **k), [so, y]),
        "rmsnorm_quant": (lambda **k: D.layer_rmsnorm_quant(s, w, r, sum=so, y8=y8, scale=sc, **k), [so, y8, sc]),
        "rmsnorm_bwd": (lambda **k: D.layer_rmsnorm_bwd(s, r, w, s, dx=dx, dweight=dw, workspace=w3, **k), [dx, dw]),
        "clip": (lambda **k: D.clip_grads(gs, 1.0, out=out, norm=norm, workspace=w4, **k), [norm] + out),
    }


NAMES = ["fwd_glr", "bwd_glr", "rmsnorm", "rmsnorm_quant", "rmsnorm_bwd", "clip"]


def same_bits(a, b):
    as_int = {1: torch.uint8, 2: torch.int16, 4: torch.int32}
    return torch.equal(a.view(as_int[a.element_size()]), b.view(as_int[a.element_size()]))


@pytest.mark.parametrize("name", NAMES)
def test_graph_replays(name):
    call, outs = calls()[name]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs:
            t.view(torch.uint8).zero_() if t.dim() else t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(outs, want))
        call()                                           # the program's own eager work between replays
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """Given as a torch stream, as a raw handle, or made current: the work follows that stream."""
    call, outs = calls()[name]
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    for form in (s, s.cuda_stream, None):
        for t in outs:
            t.view(torch.uint8).zero_() if t.dim() else t.zero_()
        torch.cuda.synchronize()
        if form is None:
            with torch.cuda.stream(s):
                call()
        else:
            call(stream=form)
        s.synchronize()
        assert all(same_bits(a, b) for a, b in zip(outs, want))


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace, do not see each other."""
    B, L, H, d = 1, 20000, 4, 64
    xs = [to_dev(draw(90 + i, (B, L, H, d)), "bf16") for i in range(2)]
    gs = [to_dev(log_gates(92 + i, (B, L, H, d)), "f32") for i in range(2)]
    want = [D.fwd_glr(x, g, input_gate="norm", want_states=True) for x, g in zip(xs, gs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            got[i].append(D.fwd_glr(xs[i], gs[i], input_gate="norm", want_states=True, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_workspace_contents_are_ignored():
    B, L, H, d = 2, 3000, 2, 64
    x, g, dO = to_dev(draw(95, (B, L, H, d)), "bf16"), to_dev(log_gates(96, (B, L, H, d)), "f32"), to_dev(draw(97, (B, L, H, d)), "bf16")
    want = D.fwd_glr(x, g, want_states=True)
    wb = D.bwd_glr(x, g, want[2], dO)
    for fill in (0, 0xff, 0x7f):
        w = torch.full((max(1, D.glr_workspace_bytes(B, L, H, d)),), fill, dtype=torch.uint8, device="cuda")
        assert all(torch.equal(a, b) for a, b in zip(D.fwd_glr(x, g, want_states=True, workspace=w), want))
        w = torch.full((max(1, D.bwd_glr_workspace_bytes(B, L, H, d)),), fill, dtype=torch.uint8, device="cuda")
        got = D.bwd_glr(x, g, want[2], dO, workspace=w)
        assert all(torch.equal(got[n], wb[n]) for n in wb)


def test_binding_refusals():
    x, g, h = torch.zeros(2, 8, 2, 16, device="cuda"), torch.zeros(2, 8, 2, 16, device="cuda"), torch.zeros(2, 2, 16, device="cuda")
    w = torch.ones(16, device="cuda")
    bad = [
        (ValueError, lambda: D.fwd_glr(x, g[:, :7])), (ValueError, lambda: D.fwd_glr(x, g, h[:1])),
        (TypeError, lambda: D.fwd_glr(x, g.bfloat16())), (TypeError, lambda: D.fwd_glr(x.half(), g)),
        (ValueError, lambda: D.fwd_glr(x.transpose(1, 2), g)), (ValueError, lambda: D.fwd_glr(x, g, input_gate="tanh")),
        (ValueError, lambda: D.fwd_glr(x, g, O=torch.empty(2, 8, 2, 32, device="cuda"))), (ValueError, lambda: D.fwd_glr(x[0], g[0])),
        (ValueError, lambda: D.bwd_glr(x, g, h, x)), (ValueError, lambda: D.decode_glr(x, g, h)),
        (ValueError, lambda: D.fwd_glr(x, g.cpu())), (D.DeltaError, lambda: D.fwd_glr(x[..., :8].contiguous(), g[..., :8].contiguous())),
        (ValueError, lambda: D.layer_rmsnorm(x, w[:8])), (ValueError, lambda: D.layer_rmsnorm(x, w, x[:1])),
        (D.DeltaError, lambda: D.layer_rmsnorm(x, w, eps=-1.0)), (D.DeltaError, lambda: D.layer_rmsnorm(x, w, y=x)),
        (ValueError, lambda: D.layer_rmsnorm_quant(x, w, group=64)), (TypeError, lambda: D.layer_rmsnorm_bwd(x, x.bfloat16(), w)),
        (ValueError, lambda: D.layer_rmsnorm_quant(x, w, scale=torch.empty(2, 8, 2, 2, device="cuda"))),
        (ValueError, lambda: D.fwd_glr(x, None)), (ValueError, lambda: D.bwd_glr(x, g, None, x)), (ValueError, lambda: D.bwd_glr(x, None, h, x)),
        (ValueError, lambda: D.layer_rmsnorm(x, None)), (ValueError, lambda: D.decode_glr(x[:, :1].contiguous(), g[:, :1].contiguous(), None)),
        (ValueError, lambda: D.grad_norm([x.transpose(1, 2)])), (TypeError, lambda: D.grad_norm([x.long()])),
    ]
    for i, (err, f) in enumerate(bad):
        with pytest.raises(err):
            say("refusal", i)
            f()
    torch.cuda.synchronize()


def test_validate_switch(monkeypatch):
    monkeypatch.setenv("DELTA_VALIDATE", "1")
    x, g = torch.zeros(1, 3000, 1, 16, device="cuda"), torch.zeros(1, 3000, 1, 16, device="cuda")
    g[0, 5] = -float("inf")
    O, h, st = D.fwd_glr(x, g, want_states=True)         # -inf is a reset, not an error
    for v in (float("nan"), float("inf")):
        g[0, 2999, 0, 15] = v
        for f in (lambda: D.fwd_glr(x, g), lambda: D.bwd_glr(x, g, st, x),
                  lambda: D.decode_glr(x[:, :1], g[:, 2999:].contiguous(), h)):
            with pytest.raises(D.DeltaError) as e:
                f()
            assert e.value.code == -8


# ---- together ---------------------------------------------------------------------------------------

def test_a_training_step_of_a_block():
    """A pre-norm residual block with the recurrence as its mixer (norm -> projections -> recurrence ->
    projection -> next norm), forward, backward and clipping, against autograd in 64 bits on the CPU.
    Tolerance: the chain is 10 stages whose longest sum has 128 terms; each adds at most (128 + 32) u of
    the magnitudes it handles, and the block's gain on them is below 8: 10 * 160 * 8 * u = 8e-4 of the
    2-norm."""
    B, L, H, d = 2, 200, 2, 64
    W = H * d
    r = lambda s, *shape: torch.from_numpy(draw(s, shape))
    P = {"x": r(101, B, L, W), "res": r(102, B, L, W), "w1": 1 + 0.1 * r(103, W), "w2": 1 + 0.1 * r(104, W),
         "Wx": r(105, W, W) / W ** 0.5, "Wg": r(106, W, W) / W ** 0.5, "Wo": r(107, W, W) / W ** 0.5, "h0": r(108, B, H, d)}
    dy, ds2 = r(109, B, L, W), r(110, B, L, W)
    base = torch.from_numpy(log_gates(111, (W,)))        # per-channel decay, sharpened by the gate's projection

    def f64():
        p = {k: v.double().requires_grad_() for k, v in P.items()}
        norm = lambda s, w: s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-6) * w
        s1 = p["x"] + p["res"]
        y1 = norm(s1, p["w1"])
        u, z = y1 @ p["Wx"], y1 @ p["Wg"]
        g = base.double() * torch.sigmoid(z)
        a, wt = torch.exp(g), torch.sqrt(-torch.expm1(2 * g))
        h, hs = p["h0"].view(B, W), []
        for t in range(L):
            h = a[:, t] * h + wt[:, t] * u[:, t]
            hs.append(h)
        s2 = torch.stack(hs, 1) @ p["Wo"] + s1
        y2 = norm(s2, p["w2"])
        ((y2 * dy.double()).sum() + (s2 * ds2.double()).sum()).backward()
        gr = {k: v.grad for k, v in p.items()}
        gr["res"] = None                                 # the same tensor's values as x's
        return y2.detach(), {k: v for k, v in gr.items() if v is not None}

    q = {k: v.cuda() for k, v in P.items()}
    s1, y1 = D.layer_rmsnorm(q["x"], q["w1"], q["res"])
    y1f = y1.view(-1, W)
    u, z = (y1f @ q["Wx"]).view(B, L, H, d), (y1f @ q["Wg"]).view(B, L, H, d)
    sg, bs = torch.sigmoid(z), base.cuda().view(H, d)
    g = (bs * sg).contiguous()
    O, _, st = D.fwd_glr(u, g, q["h0"], input_gate="norm", want_states=True)
    s2, y2 = D.layer_rmsnorm((O.view(-1, W) @ q["Wo"]).view(B, L, W), q["w2"], s1)
    dd = dy.cuda()
    dm, dw2 = D.layer_rmsnorm_bwd(dd, s2, q["w2"], ds2.cuda())
    dmf = dm.view(-1, W)
    dO = (dmf @ q["Wo"].t().contiguous()).view(B, L, H, d)
    G = D.bwd_glr(u, g, st, dO, input_gate="norm")
    du, dz = G["dx"].view(-1, W), (G["dg_log"] * bs * sg * (1 - sg)).view(-1, W)
    dy1 = du @ q["Wx"].t().contiguous() + dz @ q["Wg"].t().contiguous()
    dx, dw1 = D.layer_rmsnorm_bwd(dy1.view(B, L, W), s1, q["w1"], dm)
    grads = {"x": dx, "w1": dw1, "w2": dw2, "Wx": y1f.t().contiguous() @ du, "Wg": y1f.t().contiguous() @ dz,
             "Wo": O.view(-1, W).t().contiguous() @ dmf, "h0": G["dh0"]}
    y64, ref = f64()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())
    say("  y2", rel(y2, y64))
    assert rel(y2, y64) < 8e-4
    for k, v in ref.items():
        say("  grad", k, rel(grads[k].view(v.shape), v))
        assert rel(grads[k].view(v.shape), v) < 8e-4, k
    n = D.clip_grads(grads, 1.0)
    n64 = torch.sqrt(sum((v ** 2).sum() for v in ref.values()))
    assert abs(float(n) / float(n64) - 1) < 8e-4
    assert abs(float(D.grad_norm(grads)) - 1.0) < 1e-5 and rel(grads["Wx"] * n, ref["Wx"]) < 8e-4


def test_a_serving_step_of_a_block():
    """Prefill, then tokens one at a time: norm to 8 bits, a projection of what the 8 bits stand for,
    the recurrence's step; the same steps over the whole sequence give the same state within the bound of
    the recurrence (its inputs are the same bits either way)."""
    B, L, T, H, d = 3, 40, 4, 2, 64
    W = H * d
    x, w = to_dev(draw(120, (B, L + T, W), "bf16"), "bf16"), to_dev(1 + 0.1 * draw(121, (W,)), "f32")
    g = to_dev(log_gates(122, (B, L + T, H, d)), "f32")

    def feed(x):
        _, y8, sc = D.layer_rmsnorm_quant(x, w, group=128)
        return (y8.float() * sc).to(torch.bfloat16).view(B, -1, H, d)

    u = feed(x)
    O, h, _ = D.fwd_glr(u[:, :L].contiguous(), g[:, :L].contiguous(), input_gate="complement")
    for t in range(L, L + T):
        ut = feed(x[:, t:t + 1].contiguous())
        assert torch.equal(ut, u[:, t:t + 1])
        o = D.decode_glr(ut, g[:, t:t + 1].contiguous(), h, input_gate="complement")
    _, hr, _ = Bk.glr_fwd(host(u), host(g), None, "complement")
    E, _ = fwd_bounds(host(u), host(g), None, "complement")
    check("h", h, hr, E[:, -1] + 1e-38)
    check("o", o[:, 0], hr, E[:, -1] + HALF["bf16"] * (np.abs(hr) + E[:, -1]) + 1e-38)


def test_rmsnorm_quant_small_products():
    """s and the weight both small, rstd large: s w is near the smallest floats, y is not."""
    W = 256
    s = 1e-17 * draw(130, (3, W))
    w = (1e-21 * (1 + 0.2 * draw(131, (W,)))).astype(np.float32)
    _, y8, sc = D.layer_rmsnorm_quant(to_dev(s, "f32"), to_dev(w, "f32"), eps=0.0, group=128)
    y = Bk.rmsnorm(s, w, 0.0)
    full = np.repeat(host(sc), 128, axis=1)
    # the products keep 2^-149 / 1e-38 of their value or better: 2^-23 or so; the rest as above
    check("y8 * scale", host(y8) * full, y, np.abs(y) * (2.0 ** -4 + 1e-4) + full * 2.0 ** -9)


@pytest.mark.parametrize("n,empty", [(95, 1), (96, 0), (96, 3), (97, 0), (192, 2), (193, 0)])
def test_clip_around_a_full_table(n, empty):
    """A launch describes 96 tensors: sets that fill one or two exactly, with empty tensors behind them."""
    gs = [to_dev(draw(140 + i % 5, (3 + i % 7,)), "f32") for i in range(n)] + [torch.empty(0, device="cuda")] * empty
    ref, outs = Bk.clip([host(g) for g in gs], 1.0, 1e-6)
    got = D.clip_grads(gs, 1.0, out=[torch.empty_like(g) for g in gs[:n]] + gs[n:])
    assert abs(float(got) - ref) <= 2 * U * ref
    norm = D.clip_grads(gs, 1.0)
    assert torch.equal(norm, got)
    for i in range(n):
        check("out %d" % i, gs[i], outs[i], 6 * U * np.abs(outs[i]) + 1e-38) if i % 48 in (0, 47) else None
        assert torch.allclose(gs[i].double().cpu(), torch.from_numpy(outs[i]), rtol=1e-6, atol=0)
    assert float(D.clip_grads([torch.empty(0, device="cuda")] * 2, 1.0)) == 0.0


def test_glr_batch_does_not_matter():
    """A sequence's results are the same bits whatever batch it is in."""
    for L in (7, 32, 33, 128, 129, 3000):
        x, g = to_dev(draw(150, (5, L, 3, 32), "bf16"), "bf16"), to_dev(log_gates(151, (5, L, 3, 32)), "f32")
        O, h, st = D.fwd_glr(x, g, input_gate="norm", want_states=True)
        G = D.bwd_glr(x, g, st, x, h, input_gate="norm")
        for b in (0, 4):
            O1, h1, st1 = D.fwd_glr(x[b:b + 1], g[b:b + 1], input_gate="norm", want_states=True)
            G1 = D.bwd_glr(x[b:b + 1], g[b:b + 1], st1, x[b:b + 1], h1, input_gate="norm")
            assert torch.equal(O[b:b + 1], O1) and torch.equal(h[b:b + 1], h1) and torch.equal(st[b:b + 1], st1)
            assert all(torch.equal(G[n][b:b + 1], G1[n]) for n in G)


def test_calls_from_several_threads():
    """Calls at once from several host threads, each on its own stream and without a given workspace."""
    import threading
    B, L, H, d = 2, 5000, 2, 64
    x, g = to_dev(draw(160, (B, L, H, d), "bf16"), "bf16"), to_dev(log_gates(161, (B, L, H, d)), "f32")
    want = D.fwd_glr(x, g, input_gate="complement", want_states=True)
    n0 = D.grad_norm([g.clamp_min(-9.0)])
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(6):
            r = D.fwd_glr(x, g, input_gate="complement", want_states=True, stream=s)
            with torch.cuda.stream(s):
                n = D.grad_norm([g.clamp_min(-9.0)])
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(r, want)) or not torch.equal(n, n0):
                bad.append(1)

    ts = [threading.Thread(target=work) for _ in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_clip_outputs_by_name():
    """Outputs of a dict are found by name whatever its order; a gradient that is None has none."""
    gs = {k: to_dev(draw(150 + i, (64,), "f32"), "f32") for i, k in enumerate("wvu")}
    gs["none"] = None
    out = {k: None if gs[k] is None else torch.zeros_like(gs[k]) for k in ("none", "u", "v", "w")}
    ref, outs = Bk.clip([host(gs[k]) for k in "wvu"], 1.0, 1e-6)
    n = D.clip_grads(gs, 1.0, out=out)
    assert abs(float(n) - ref) <= 2 * U * ref
    for k, r in zip("wvu", outs):
        check(k, out[k], r, 6 * U * np.abs(r))
    mine = [torch.zeros_like(g) for g in (gs["w"], gs["u"])]
    D.clip_grads([gs["w"], None, gs["u"]], 1e9, out=[mine[0], torch.zeros(64, device="cuda"), mine[1]])
    assert torch.equal(mine[0], gs["w"]) and torch.equal(mine[1], gs["u"])


@pytest.mark.parametrize("N,W", [(4103, 1003), (2051, 2048), (1030, 2056), (1029, 4096), (2050, 4104)])
def test_rmsnorm_more_rows_than_workgroups(N, W):
    """Rows of several wavefronts, more than one launch has workgroups for: these walk over them."""
    test_rmsnorm(N, W, "bf16")
    for group in (0, 128):
        test_rmsnorm_quant(N, W, "bf16", group)
    test_rmsnorm_bwd(N, W, "bf16")
