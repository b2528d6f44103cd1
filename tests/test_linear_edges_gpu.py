"""Linear attention where its inputs leave the ordinary: gates above 1 next to resets and over several segments, and
sequences whose tokens differ by orders of magnitude.

Tolerances are those of test_linear_gpu.py (u = 2^-24, M the same recurrence on magnitudes), elementwise.  A decay e^x
carries (2 + |x|) u, so along a path over n chunks whose log gates add up to at most X in magnitude in each, the
decays carry n (4 + X) u: c = dk + dv + 64 + n (4 + X) + 100.
"""
import numpy as np
import pytest

from oracle import linear as Lo
from parity import say, to_dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
CHUNK = {"bf16": 64, "f32": 32}


def draw(seed, shape, dtype="f32"):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(name, got, ref, tol):
    got = host(got)
    with np.errstate(divide="ignore", invalid="ignore"):
        over = np.nan_to_num(np.abs(got - ref) / tol, nan=np.inf, posinf=np.inf)
    over[got == ref] = 0.0
    say("  %s: max error / bound %.3f" % (name, over.max()))
    assert over.max() <= 1.0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


class Problem:
    """Inputs by hand, the oracle's results, and the bounds above."""

    def __init__(self, dtype, q, k, v, g, S0=None, dO=None, dS=None, scale=1.0):
        self.dtype, self.x, self.dO, self.dS, self.scale = dtype, dict(q=q, k=k, v=v, g=g, S0=S0), dO, dS, scale
        self.dev = [to_dev(self.x[n], dtype if n in "qkv" else "f32") for n in ("q", "k", "v", "g", "S0")]
        self.x["g"] = np.where(np.exp(g.astype(np.float32)) == 0, -np.inf, g)    # by the header a reset is an exact 0
        L, C = q.shape[1], CHUNK[dtype]
        finite = np.where(np.isfinite(g), np.abs(g), 0.0)
        X = max(finite[:, i:i + C].sum(1).max() for i in range(0, L, C))
        self.c = q.shape[3] + v.shape[3] + 64 + -(-L // C) * (4 + X) + 100
        self.once = HALF["bf16"] if dtype == "bf16" else 0.0
        self.abs = {n: a if a is None or n == "g" else np.abs(a) for n, a in self.x.items()}

    def rounded(self, M, ref):
        return (self.once + self.c * U) * M + HALF[self.dtype] * (np.abs(ref) + (self.once + self.c * U) * M) + 1e-36

    def check_fwd(self):
        O, S = D.fwd_lin(*self.dev, scale=self.scale)
        torch.cuda.synchronize()
        Or, Sr = Lo.fwd(**self.x, scale=self.scale)
        Om, Sm = Lo.fwd(**self.abs, scale=self.scale)
        check("S_final", S, Sr, self.c * U * Sm + 1e-36)
        check("O", O, Or, self.rounded(Om, Or))
        return O, S

    def check_bwd(self):
        """dq, dk, dv and dS0, as test_linear_gpu.py bounds them."""
        mag = lambda x: None if x is None else np.abs(x)
        ref = Lo.bwd(*self.x.values(), self.dO, self.dS, self.scale)
        M = Lo.bwd(*self.abs.values(), mag(self.dO), mag(self.dS), self.scale)
        G = D.bwd_lin(*self.dev, to_dev(self.dO, self.dtype), to_dev(self.dS, "f32"), scale=self.scale)
        torch.cuda.synchronize()
        for n in ("dq", "dk", "dv"):
            check(n, G[n], ref[n], self.rounded(M[n], ref[n]))
        check("dS0", G["dS0"], ref["dS0"], self.c * U * M["dS0"] + 1e-36)
        return G, ref, M


def above_one(seed, B, L, H, span, top):
    """Gates up to e^(top / span), most of them above 1, with a reset at least every `span` tokens: their product
    over any stretch between two resets, and over any chunk, is below e^top."""
    r = np.random.default_rng(seed)
    g = (r.uniform(-0.2, 1.0, (B, L, H)) * top / span).astype(np.float32)
    t = int(r.integers(0, span))
    while t < L:
        g[:, t] = -np.inf if r.random() < 0.5 else -104.5      # exp(-104.5) is 0 in float32 too
        t += int(r.integers(span // 3, span))
    return g


# ---- resets among gates above 1 -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H", [(1, 1), (3, 100)])
def test_a_reset_stays_one_behind_gates_above_1(dtype, B, H):
    """The first gate is a reset and nothing is written behind it: every output is 0, however large the gates behind
    the reset are (a chunk's product is in float32's range), in segments and without."""
    C = CHUNK[dtype]
    L, d = 6 * C, 16
    g = np.full((B, L, H), 80.0 / C, np.float32)
    g[:, 0] = -np.inf
    z, r = np.zeros((B, L, H, d), np.float32), draw(1, (B, L, H, d), dtype)
    O, S = D.fwd_lin(*(to_dev(x, dtype) for x in (r, z, r)), to_dev(g, "f32"), torch.ones(B, H, d, d, device="cuda"))
    assert not O.any() and not S.any()
    # mirrored: the last gate a reset, and only the state behind it has a gradient
    g = np.full((B, L, H), 80.0 / C, np.float32)
    g[:, -1] = -np.inf
    G = D.bwd_lin(*(to_dev(x, dtype) for x in (z, r, r)), to_dev(g, "f32"), None, to_dev(z, dtype), torch.ones(B, H, d, d, device="cuda"))
    # (not dg_log: the states themselves grow by e^80 in each of six chunks, past float32, and their products with 0 are NaN)
    assert not G["dS0"].any() and not G["dk"][:, :-1].any() and not G["dv"][:, :-1].any()


@pytest.mark.parametrize("B,L,Hk,H,dk,dv,dtype", [
    (1, 64, 1, 1, 16, 16, "bf16"), (2, 200, 1, 2, 32, 48, "f32"), (1, 700, 1, 2, 64, 64, "bf16"), (1, 450, 2, 2, 128, 144, "f32"),
    (2, 333, 1, 1, 32, 160, "bf16"), (3, 130, 30, 90, 16, 32, "bf16"), (1, 500, 3, 3, 64, 32, "f32")])
def test_gates_above_1_between_resets(B, L, Hk, H, dk, dv, dtype):
    r = lambda seed, *shape, t=dtype: draw(seed, shape, t)
    p = Problem(dtype, r(1, B, L, Hk, dk), r(2, B, L, Hk, dk), r(3, B, L, H, dv), above_one(4, B, L, H, 60, 50.0),
                r(5, B, H, dk, dv, t="f32"), r(6, B, L, H, dv), r(7, B, H, dk, dv, t="f32"), dk ** -0.5)
    say("above 1", B, L, Hk, H, dk, dv, dtype)
    p.check_fwd()
    G, _, _ = p.check_bwd()
    check_gates("dg_log", G["dg_log"], p.x, p.dO, p.dS, p.scale, p.c)
    hard = p.x["g"] == -np.inf
    assert hard.any() and not host(G["dg_log"])[hard].any()


# ---- gates above 1 over several segments -----------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_above_1_before_anything_is_written(dtype):
    """A chunk's product is in float32's range (e^38), a segment's (e^153) is not, but there is nothing for it to
    multiply: the state is 0 until the last tokens, and its gradient behind the first."""
    B, L, H, d = 1, 4096, 16, 16
    g = np.full((B, L, H), 0.6, np.float32)
    late, early = np.arange(L)[:, None, None] >= L - 60, np.arange(L)[:, None, None] < 60
    r = lambda seed: draw(seed, (B, L, H, d), dtype)
    p = Problem(dtype, r(1), (r(2) * late).astype(np.float32), r(3), g, None, (r(4) * early).astype(np.float32))
    say("before anything is written", dtype)
    p.check_fwd()
    G, _, _ = p.check_bwd()
    assert not G["dg_log"].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_small_state_grows_past_a_segments_range(dtype):
    """A start state of 1e-30 and gates of e^130 in all within a segment (e^42 at most in a chunk), and back again for
    the gradient of the state behind the last token: the results are float32 numbers, the segment's product is none."""
    B, L, H, d = 1, 4096, 16, 16
    t = np.arange(L)[None, :, None]
    r = lambda seed, *s: draw(seed, s, dtype)
    grow = np.broadcast_to(((t >= 20) & (t < 220)) * np.float32(0.65), (B, L, H)).astype(np.float32)
    x = [r(s, B, L, H, d) for s in (1, 2, 3)]
    still = (x[1] * (t[..., None] >= 220)).astype(np.float32)
    p = Problem(dtype, x[0], still, x[2], grow, np.float32(1e-30) * draw(5, (B, H, d, d)))
    say("a small state", dtype)
    p.check_fwd()
    late = grow[:, ::-1].copy()                                   # the same in the last segment, met by the gradient first
    end = (x[1] * (t[..., None] >= L - 20)).astype(np.float32)    # (the states would outgrow float32)
    p = Problem(dtype, x[0], end, x[2], late, None, (r(6, B, L, H, d) * (t[..., None] < L - 220)).astype(np.float32),
                np.float32(1e-30) * draw(7, (B, H, d, d)))
    p.check_bwd()


# ---- gradients of the gates where tokens differ by orders of magnitude ------------------------------

def crossing(x, dO, dS, scale):
    """Per token, what the gate's gradient is a sum of, in magnitudes: a_t <|S_{t-1}|, |G_t|> of the recurrences on
    magnitudes (every pair of a write before t and a read from t on, with its decays)."""
    a = Lo._gates(x["g"], *dO.shape[:3])
    S, (G, _) = Lo.states(x["k"], x["v"], x["g"], x["S0"]), Lo.flows(x["q"], dO, x["g"], dS, scale)
    return np.stack([a[:, t] * (S[t] * G[t]).sum((2, 3)) for t in range(dO.shape[1])], 1)


def check_gates(name, got, x, dO, dS, scale, c):
    """dg_log elementwise: the two states of every product are each within c u of their magnitudes, as S_final and dS0
    are, and the product's sums add 64 terms in a lane and 64 more over lanes, tokens and blocks at most: an error of
    (2 c + 128) u times what crosses this very token.  1e-30 for what falls out of float32."""
    ref = Lo.bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], dO, dS, scale)["dg_log"]
    mag = {n: a if a is None or n == "g" else np.abs(a) for n, a in x.items()}
    tol = (2 * c + 128) * U * crossing(mag, np.abs(dO), None if dS is None else np.abs(dS), scale) + 1e-30
    if ref.ndim == 1:  # the sum over tokens in 64 bits, rounded once
        tol = tol.sum((0, 1)) + U * np.abs(ref)
    check(name, got, ref, tol)


def steps(kind, L):
    """How much larger the tokens of v and dO are."""
    s, t = np.ones(L, np.float32), np.arange(L)
    if kind == "early":
        s[t < 40] = 1e3
    elif kind == "twice":
        s[(t % 211 > 20) & (t % 211 < 33)] = 1e4
    elif kind == "late":
        s[t >= L - 40] = 1e3
    return s[None, :, None, None]


@pytest.mark.parametrize("B,L,Hk,H,dk,dv,dtype,kind,rate", [
    (33, 300, 2, 2, 16, 32, "bf16", "early", 0.3), (33, 300, 2, 2, 32, 16, "f32", "early", 0.3), (33, 700, 1, 2, 16, 16, "f32", "twice", 0.1),
    (33, 900, 2, 2, 128, 128, "bf16", "twice", 0.1), (33, 300, 2, 2, 128, 128, "f32", "late", 0.3), (70, 400, 1, 1, 64, 80, "bf16", "late", 0.02),
    (1, 3000, 2, 2, 64, 64, "bf16", "early", 0.3), (1, 2000, 1, 2, 32, 96, "f32", "twice", 0.1), (40, 500, 1, 2, 32, 240, "bf16", "twice", 0.1),
    (40, 300, 2, 2, 128, 144, "f32", "early", 0.3), (2, 130, 1, 1, 64, 48, "bf16", "twice", 1.0), (1, 64, 1, 1, 16, 16, "bf16", "late", 0.5),
    (1, 33, 1, 1, 16, 16, "f32", "early", 0.5), (2, 1, 1, 1, 32, 16, "bf16", "even", 0.5), (3, 65, 1, 3, 128, 32, "bf16", "even", 0.05)])
@pytest.mark.parametrize("gate", ["token", "head"])
def test_gradients_of_gates_next_to_much_larger_tokens(B, L, Hk, H, dk, dv, dtype, kind, rate, gate):
    """Each token's gradient is as good as what crosses that token, whatever the sequence holds elsewhere (the state
    forgets it), with a launch of one segment and of several; the oracle on the first and last sequence."""
    r = lambda seed, *shape, t=dtype: draw(seed, shape, t)
    big = steps(kind, L)
    to = lambda x: draw_as(x * big, dtype)
    g = -np.random.default_rng(5).uniform(0.5, 1.5, (B, L, H) if gate == "token" else H).astype(np.float32) * np.float32(rate)
    x = dict(q=r(1, B, L, Hk, dk), k=r(2, B, L, Hk, dk), v=to(r(3, B, L, H, dv)), g=g, S0=r(6, B, H, dk, dv, t="f32"))
    dO, dS, scale = to(r(4, B, L, H, dv)), r(7, B, H, dk, dv, t="f32"), dk ** -0.5
    dev = [to_dev(x[n], dtype if n in "qkv" else "f32") for n in ("q", "k", "v", "g", "S0")]
    say("gates", B, L, Hk, H, dk, dv, dtype, kind, gate)
    C = CHUNK[dtype]
    c = dk + dv + 64 + -(-L // C) * (4 + 1.5 * rate * C) + 100
    one = lambda b: {n: a if n == "g" and gate == "head" else a[b:b + 1] for n, a in x.items()}
    if gate == "token":
        G = D.bwd_lin(*dev, to_dev(dO, dtype), to_dev(dS, "f32"), scale=scale)
        for b in {0, B - 1}:
            check_gates("dg_log", G["dg_log"][b:b + 1], one(b), dO[b:b + 1], dS[b:b + 1], scale, c)
        return
    # a fixed decay's gradient takes all sequences: with nothing else than the first and the last one's dO and dS
    dO[1:-1], dS[1:-1] = 0, 0
    G = D.bwd_lin(*dev, to_dev(dO, dtype), to_dev(dS, "f32"), scale=scale)
    pick = [0, B - 1] if B > 1 else [0]
    two = {n: a if n == "g" else a[pick] for n, a in x.items()}
    check_gates("dg_log", G["dg_log"], two, dO[pick], dS[pick], scale, c)


def draw_as(x, dtype):
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x.astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_workspace_for_sequences_up_to_the_longest(dtype):
    B, Hk, H, dk, dv = 3, 2, 6, 64, 80
    code = D.BF16 if dtype == "bf16" else D.F32
    ws = torch.empty(max(D.lin_workspace_bytes(B, 1500, Hk, H, dk, dv, code), D.bwd_lin_workspace_bytes(B, 1500, Hk, H, dk, dv, code, 1)),
                     dtype=torch.uint8, device="cuda")
    for L in (1500, 223, 260, 40, 700, 1):
        r = lambda seed, *s: to_dev(draw(seed, s, dtype), dtype)
        q, k, v, dO = r(1, B, L, Hk, dk), r(2, B, L, Hk, dk), r(3, B, L, H, dv), r(4, B, L, H, dv)
        g = to_dev(-np.abs(draw(5, (B, L, H))), "f32")
        ws.fill_(255)
        for a, b in zip(D.fwd_lin(q, k, v, g), D.fwd_lin(q, k, v, g, workspace=ws)):
            assert torch.equal(a, b)
        for a, b in zip(D.bwd_lin(q, k, v, g, None, dO).values(), D.bwd_lin(q, k, v, g, None, dO, workspace=ws).values()):
            assert torch.equal(a, b)


# ---- bf16 outputs: their own rounding and one operand's --------------------------------------------

@pytest.mark.parametrize("gate", ["none", "head", "token"])
@pytest.mark.parametrize("B,L,Hk,H,dk,dv", [(4, 171, 8, 16, 32, 48), (2, 1500, 2, 2, 32, 64), (1, 1200, 1, 1, 128, 160), (40, 300, 2, 2, 64, 64),
                                            (1, 1000, 2, 2, 128, 128)])
def test_bf16_outputs_carry_one_operands_rounding(gate, B, L, Hk, H, dk, dv):
    """Each output is a sum of products one operand of which is rounded to bf16 (the state, or a pair's weight), and is
    rounded itself.  With rho the 2-norm of the outputs' own rounding and operands whose roundings are as large and
    independent, that is sqrt(2) rho; a second operand's would make it sqrt(3).  Bound 1.5.  The oracle on the first and
    last sequence."""
    r = lambda seed, *shape, t="bf16": draw(seed, shape, t)
    g = None if gate == "none" else -np.random.default_rng(5).uniform(0.0, 0.01, (B, L, H) if gate == "token" else H).astype(np.float32)
    x = dict(q=r(1, B, L, Hk, dk), k=r(2, B, L, Hk, dk), v=r(3, B, L, H, dv), g=g, S0=r(6, B, H, dk, dv, t="f32"))
    dO, dS, scale = r(4, B, L, H, dv), r(7, B, H, dk, dv, t="f32"), dk ** -0.5
    dev = [to_dev(x[n], "bf16" if n in "qkv" else "f32") for n in ("q", "k", "v", "g", "S0")]
    say("roundings", gate, B, L, Hk, H, dk, dv)
    got = {"O": D.fwd_lin(*dev, scale=scale)[0]}
    for want in (True, False):
        G = D.bwd_lin(*dev, to_dev(dO, "bf16"), to_dev(dS, "f32"), scale=scale, want_dg_log=want)
        got.update({"%s%d" % (n, want): G[n] for n in ("dq", "dk", "dv")})
    pick = sorted({0, B - 1})
    one = {n: a if a is None or a.ndim == 1 else a[pick] for n, a in x.items()}
    ref = Lo.bwd(*one.values(), dO[pick], dS[pick], scale)
    ref["O"] = Lo.fwd(**one, scale=scale)[0]
    for n, t in got.items():
        want = ref[n.rstrip("01")]
        own = torch.from_numpy(want).to(torch.bfloat16).double().numpy() - want
        ratio = np.linalg.norm(host(t[pick]) - want) / np.linalg.norm(own)
        say("  %s: %.3f of its own rounding" % (n, ratio))
        assert ratio <= 1.5, (n, ratio)
