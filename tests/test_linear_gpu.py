"""GPU parity of linear attention (include/delta_linear.h) with the fp64 oracle in oracle/linear.py.

Tolerances are elementwise and derived from the arithmetic, with u = 2^-24 the float32 half step.  Every
output is a sum of products whose magnitudes add up to M, the same recurrence run on |q|, |k|, |v|, |S0|,
|dO|, |dS_final|:
  * float32 sums of n terms in any order: n u M.  Along a product's path there are at most dk + dv
    (contractions), 64 (tokens of a chunk), 4 per chunk (a state's decay, its addition, the combination
    over segments); a decay e^-x carries (2 + x) u, and where x > 87 its product counts for nothing: 100 u
    with the few roundings of factors.  c = dk + dv + 64 + 4 chunks + 100.
  * bf16 inputs: an output's share of the state, and of the chunk, goes through one operand rounded to
    bf16, half a step 2^-8 of M.  States, gates' gradients and float32 inputs do not.
  * the outputs' own rounding: half a step of their type.
  * a gate's gradient is the inner product of a state and its gradient, carried through a segment as sums
    of what each token adds (e, f): c u times all of those magnitudes added up.
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


def draw(seed, shape, dtype="f32"):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x


def gates(seed, B, L, H, kind, resets=()):
    """Log gates from -9 to -1e-3 (each head of a strength of its own), -inf at the tokens of `resets`."""
    if kind == "none":
        return None
    r = np.random.default_rng(seed)
    if kind == "head":
        return -np.exp(r.uniform(np.log(1e-3), np.log(2.0), H)).astype(np.float32)
    g = -np.exp(r.uniform(np.log(1e-3), np.log(0.5), (1, 1, H)) + r.uniform(-1, 3, (B, L, H))).astype(np.float32)
    for t in resets:
        g[:, t] = -np.inf
    return g


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


def check(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    if not got.size:
        return
    with np.errstate(divide="ignore", invalid="ignore"):
        over = np.nan_to_num(np.abs(got - ref) / tol, nan=np.inf, posinf=np.inf)
    over[got == ref] = 0.0
    norm = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
    say("  %s: max error / bound %.3f, 2-norm %.2e" % (name, over.max(), norm))
    assert over.max() <= 1.0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


class Case:
    def __init__(self, B, L, Hk, H, dk, dv, dtype, kind, resets=(), S0=True, dS=True, seed=0):
        self.dtype, self.L, self.scale = dtype, L, dk ** -0.5
        self.np = dict(q=draw(seed + 1, (B, L, Hk, dk), dtype), k=draw(seed + 2, (B, L, Hk, dk), dtype),
                       v=draw(seed + 3, (B, L, H, dv), dtype), g=gates(seed + 4, B, L, H, kind, resets),
                       S0=draw(seed + 5, (B, H, dk, dv)) if S0 else None)
        self.dO, self.dS = draw(seed + 6, (B, L, H, dv), dtype), draw(seed + 7, (B, H, dk, dv)) if dS else None
        self.dev = [to_dev(self.np[n], dtype) for n in "qkv"] + [None if self.np[n] is None else to_dev(self.np[n], "f32") for n in ("g", "S0")]
        self.devO, self.devS = to_dev(self.dO, dtype), None if self.dS is None else to_dev(self.dS, "f32")
        self.c = dk + dv + 64 + 4 * (L // 32 + 1) + 100
        self.abs = {n: None if x is None else x if n == "g" else np.abs(x) for n, x in self.np.items()}
        self.once = HALF["bf16"] if dtype == "bf16" else 0.0  # an operand's rounding

    def bound(self, M, ref):
        return (self.once + self.c * U) * M + HALF[self.dtype] * (np.abs(ref) + (self.once + self.c * U) * M) + 1e-36

    def check_fwd(self, O, S):
        Or, Sr = Lo.fwd(**self.np, scale=self.scale)
        Om, Sm = Lo.fwd(**self.abs, scale=self.scale)
        check("O", O, Or, self.bound(Om, Or))
        check("S_final", S, Sr, self.c * U * Sm + 1e-36)

    def check_bwd(self, G):
        a = self.abs
        ref = Lo.bwd(*self.np.values(), self.dO, self.dS, self.scale)
        mag = Lo.bwd(*a.values(), np.abs(self.dO), None if self.dS is None else np.abs(self.dS), self.scale)
        for n in ("dq", "dk", "dv"):
            check(n, G[n], ref[n], self.bound(mag[n], ref[n]))
        check("dS0", G["dS0"], ref["dS0"], self.c * U * mag["dS0"] + 1e-36)
        if a["g"] is None:
            assert G["dg_log"] is None
            return
        B, L, H, dv = a["v"].shape
        share = H // a["q"].shape[2]
        e = (np.repeat(mag["dq"] * a["q"], share, 2)).sum((1, 3)) / share + (np.repeat(mag["dk"] * a["k"], share, 2)).sum((1, 3)) / share
        ends = 0.0
        if self.L:
            S, (F, F0) = Lo.states(a["k"], a["v"], a["g"], a["S0"]), Lo.flows(a["q"], np.abs(self.dO), a["g"], self.dS if self.dS is None else np.abs(self.dS), self.scale)
            ends = max((s * f).sum((2, 3)).max() for s, f in zip(S, [F0] + F))
        if share > 1:
            e = e.sum(1, keepdims=True) * share                       # all heads': more than any one's
        tol = self.c * U * (np.broadcast_to(e, (B, H)) + ends)
        if a["g"].ndim == 1:
            check("dg_log", G["dg_log"], ref["dg_log"], L * tol.sum(0) + 1e-36)
        else:
            check("dg_log", G["dg_log"], ref["dg_log"], np.broadcast_to(tol[:, None], (B, L, H)) + 1e-36)
        # the bound above counts every rounding at its worst; as random ones they are this far off in the 2-norm
        # (a sum over all tokens, or of one token, cancels what a norm over many does not)
        if a["g"].ndim == 3 and L > 8:
            d = host(G["dg_log"]) - ref["dg_log"]
            assert np.linalg.norm(d) <= 2e-5 * np.linalg.norm(ref["dg_log"])


CASES = [
    # B, L, Hk, H, dk, dv, dtype, gates, resets, S0, dS_final
    (1, 1, 1, 1, 16, 16, "f32", "token", (), True, True), (1, 1, 1, 1, 16, 16, "bf16", "head", (), True, True),
    (2, 2, 1, 3, 32, 32, "bf16", "token", (1,), True, False), (1, 31, 2, 2, 64, 48, "f32", "token", (0,), False, True),
    (1, 32, 1, 2, 128, 16, "f32", "token", (31,), True, True), (1, 33, 1, 1, 32, 112, "f32", "none", (), False, False),
    (2, 63, 1, 2, 64, 48, "bf16", "token", (62, 5), True, True), (1, 64, 2, 2, 128, 128, "bf16", "token", (0, 63), True, True),
    (1, 65, 1, 1, 16, 256, "bf16", "token", (64,), True, True), (1, 65, 1, 2, 16, 256, "f32", "head", (), True, True),
    (2, 129, 1, 3, 128, 144, "bf16", "head", (), True, True), (3, 127, 1, 1, 64, 128, "f32", "token", (64, 96, 95), True, True),
    (1, 300, 2, 2, 32, 96, "bf16", "token", (128, 129, 299), True, True), (1, 300, 3, 6, 128, 240, "f32", "token", (32,), True, False),
    (1, 1000, 1, 1, 128, 256, "bf16", "head", (), True, True), (1, 1000, 1, 2, 128, 128, "bf16", "none", (), True, True),
    (3, 1237, 2, 6, 64, 80, "f32", "token", (100, 640, 1236), True, True), (2, 777, 4, 8, 128, 128, "bf16", "token", (), True, True),
    (16, 200, 16, 16, 32, 32, "bf16", "token", (70,), True, True), (1, 4099, 1, 1, 64, 64, "bf16", "token", (4096, 17), True, True),
]


def name(c):
    return "x".join(map(str, c[:6])) + c[6] + c[7]


@pytest.mark.parametrize("case", CASES, ids=name)
def test_lin(case):
    say("lin", case)
    c = Case(*case)
    O, S = D.fwd_lin(*c.dev, scale=c.scale)
    torch.cuda.synchronize()
    c.check_fwd(O, S)
    G = D.bwd_lin(*c.dev, c.devO, c.devS, scale=c.scale)
    torch.cuda.synchronize()
    c.check_bwd(G)
    # the same call again: the same bits, whatever the workspace holds
    code = D.BF16 if c.dtype == "bf16" else D.F32
    kind = {"none": 0, "token": 1, "head": 2}[case[7]]
    need = max(D.lin_workspace_bytes(*case[:6], code), D.bwd_lin_workspace_bytes(*case[:6], code, kind), 16)
    ws = torch.full((need // 4,), float("nan"), device="cuda")
    O2, S2 = D.fwd_lin(*c.dev, scale=c.scale, workspace=ws)
    assert torch.equal(O, O2) and torch.equal(S, S2)
    ws.fill_(float("nan"))
    G2 = D.bwd_lin(*c.dev, c.devO, c.devS, scale=c.scale, workspace=ws)
    for n, t in G.items():
        assert (t is None and G2[n] is None) or torch.equal(t, G2[n]), n


@pytest.mark.parametrize("case", [
    (5, 450, 8, 16, 128, 128, "bf16", "token", (70, 200, 449), True, True), (6, 200, 8, 16, 64, 80, "f32", "head", (), True, True),
    (5, 170, 16, 16, 128, 128, "f32", "token", (33,), False, True), (6, 300, 16, 16, 32, 144, "bf16", "token", (64,), True, False),
    (260, 130, 1, 1, 16, 32, "bf16", "none", (), True, True), (33, 200, 2, 8, 32, 64, "bf16", "head", (), True, True)], ids=name)
def test_many_heads_in_one_segment(case):
    """Chunk after chunk in one launch, where heads alone fill the card."""
    test_lin(case)


def test_the_full_shape():
    """The 2 x 8K-token, 16-head shape with heads that share q and k; the oracle on two value heads of one
    sequence, one from either end."""
    B, L, Hk, H, dk, dv = 2, 8192, 8, 16, 128, 128
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    q, k, v, dO = (r(B, L, n, 128).to(torch.bfloat16) for n in (Hk, Hk, H, H))
    g = -torch.nn.functional.softplus(r(B, L, H) + torch.linspace(2, -4, H, device="cuda"))
    g[1, 3000] = -float("inf")
    S0, dS = r(B, H, dk, dv), r(B, H, dk, dv)
    O, S = D.fwd_lin(q, k, v, g, S0, scale=dk ** -0.5)
    G = D.bwd_lin(q, k, v, g, S0, dO, dS, scale=dk ** -0.5)
    say("full shape")
    for b, h in ((1, 0), (0, 14)):  # the even head of a pair; the pair's dq and dk take both
        one = lambda x, i, n=1: host(x[b:b + 1, ..., i:i + n, :] if x.dim() == 4 else x[b:b + 1, ..., i:i + n])
        args = (one(q, h // 2), one(k, h // 2), host(v[b:b + 1, :, h:h + 2]), host(g[b:b + 1, :, h:h + 2]), host(S0[b:b + 1, h:h + 2]))
        Or, Sr = Lo.fwd(*args, scale=dk ** -0.5)
        ref = Lo.bwd(*args, host(dO[b:b + 1, :, h:h + 2]), host(dS[b:b + 1, h:h + 2]), scale=dk ** -0.5)
        got = {"O": (O[b:b + 1, :, h:h + 2], Or), "S": (S[b:b + 1, h:h + 2], Sr), "dq": (G["dq"][b:b + 1, :, h // 2:h // 2 + 1], ref["dq"]),
               "dk": (G["dk"][b:b + 1, :, h // 2:h // 2 + 1], ref["dk"]), "dv": (G["dv"][b:b + 1, :, h:h + 2], ref["dv"]),
               "dg_log": (G["dg_log"][b:b + 1, :, h:h + 2], ref["dg_log"]), "dS0": (G["dS0"][b:b + 1, h:h + 2], ref["dS0"])}
        for n, (x, want) in got.items():
            e = np.linalg.norm(host(x) - want) / np.linalg.norm(want)
            say("  head %d %s: 2-norm %.2e" % (h, n, e))
            # bf16: an operand's and the output's rounding, each at most 2^-8 and at random about 2^-9.2; float32:
            # as in check_bwd
            assert e <= (2 * 2.0 ** -8 if x.dtype == torch.bfloat16 else 2e-5), n


def test_optional_arguments():
    c = Case(2, 200, 1, 2, 32, 48, "f32", "token", S0=False, dS=False)
    q, k, v, g, _ = c.dev
    zero = torch.zeros(2, 2, 32, 48, device="cuda")
    O, S = D.fwd_lin(q, k, v, g)
    O2, none = D.fwd_lin(q, k, v, g, zero, want_state=False)
    assert none is None and torch.equal(O, O2) and torch.equal(S, D.fwd_lin(q, k, v, g, zero)[1])
    G, G2 = D.bwd_lin(q, k, v, g, None, c.devO), D.bwd_lin(q, k, v, g, zero, c.devO, zero)
    for n in G:
        assert torch.equal(G[n], G2[n]), n
    G3 = D.bwd_lin(q, k, v, g, zero, c.devO, want_dg_log=False, want_dS0=False)
    assert G3["dg_log"] is None and G3["dS0"] is None
    G4 = D.bwd_lin(q, k, v, g, torch.randn_like(zero), c.devO, want_dS0=False)
    assert G4["dS0"] is None and torch.isfinite(G4["dg_log"]).all()
    for n in ("dq", "dk", "dv"):
        assert torch.allclose(G[n], G3[n], rtol=1e-5, atol=1e-5), n
    # without gates: as with gates of 0
    O0, S0 = D.fwd_lin(q, k, v, torch.zeros_like(g))
    O1, S1 = D.fwd_lin(q, k, v)
    assert torch.equal(O0, O1) and torch.equal(S0, S1)
    outs = {n: torch.empty_like(G[n]) for n in ("dq", "dS0", "dg_log")}
    G5 = D.bwd_lin(q, k, v, g, None, c.devO, grads=outs)
    for n, t in outs.items():
        assert G5[n] is t and torch.equal(t, G[n])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_fixed_decays_are_gates_that_do_not_change(dtype):
    c = Case(2, 333, 2, 4, 64, 64, dtype, "head")
    q, k, v, g, S0 = c.dev
    full = g.expand(2, 333, 4).contiguous()
    O, S = D.fwd_lin(q, k, v, g, S0)
    O2, S2 = D.fwd_lin(q, k, v, full, S0)
    assert torch.equal(O, O2) and torch.equal(S, S2)
    G, G2 = D.bwd_lin(q, k, v, g, S0, c.devO, c.devS), D.bwd_lin(q, k, v, full, S0, c.devO, c.devS)
    for n in ("dq", "dk", "dv", "dS0"):
        assert torch.equal(G[n], G2[n]), n
    # the sum over tokens, held in 64 bits here, from values rounded to float32 there
    want = G2["dg_log"].double().sum((0, 1))
    assert ((G["dg_log"].double() - want).abs() <= U * (G2["dg_log"].double().abs().sum((0, 1)) + want.abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_heads_are_repeated_heads(dtype):
    c = Case(1, 500, 2, 6, 64, 80, dtype, "token")
    q, k, v, g, S0 = c.dev
    q3, k3 = (x.repeat_interleave(3, 2) for x in (q, k))
    O, S = D.fwd_lin(q, k, v, g, S0)
    O2, S2 = D.fwd_lin(q3, k3, v, g, S0)
    assert torch.equal(O, O2) and torch.equal(S, S2)
    G, G2 = D.bwd_lin(q, k, v, g, S0, c.devO, c.devS), D.bwd_lin(q3, k3, v, g, S0, c.devO, c.devS)
    for n in ("dv", "dg_log", "dS0"):
        assert torch.equal(G[n], G2[n]), n
    for n in ("dq", "dk"):
        parts = G2[n].double().view(1, 500, 2, 3, 64)
        want = parts.sum(3)
        # three parts each rounded there, their sum here
        assert ((G[n].double() - want).abs() <= HALF[dtype] * (parts.abs().sum(3) + want.abs()) * 1.01 + 4 * U * parts.abs().sum(3)).all(), n


def test_shared_heads_of_more_rows_than_the_sum_has_threads():
    """In float32 dq and dk of a shared head are the sums of what each value head's own call gives, bit for bit."""
    B, L, Hk, H, dk, dv = 1, 70001, 4, 8, 128, 16
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    q, k, v, dO, g = r(B, L, Hk, dk), r(B, L, Hk, dk) / 16, r(B, L, H, dv), r(B, L, H, dv), -torch.rand((B, L, H), generator=gen, device="cuda")
    shared = D.bwd_lin(q, k, v, g, None, dO)
    each = D.bwd_lin(q.repeat_interleave(2, 2), k.repeat_interleave(2, 2), v, g, None, dO)
    for n in ("dq", "dk"):
        assert torch.equal(shared[n], each[n][:, :, 0::2] + each[n][:, :, 1::2]), n
    assert torch.equal(shared["dv"], each["dv"]) and torch.equal(shared["dg_log"], each["dg_log"])


def test_in_place_and_split_over_calls():
    c = Case(2, 1000, 1, 3, 64, 48, "bf16", "token")
    q, k, v, g, S0 = c.dev
    st = S0.clone()
    cut = lambda x, a, b: x[:, a:b].contiguous()
    outs = []
    for a, b in ((0, 333), (333, 334), (334, 1000)):
        O, S = D.fwd_lin(cut(q, a, b), cut(k, a, b), cut(v, a, b), cut(g, a, b), st, scale=c.scale, S_final=st)
        assert S is st
        outs.append(O)
    c.check_fwd(torch.cat(outs, 1), st)


def test_empty():
    for B, L, H in ((0, 5, 2), (2, 0, 3)):
        x, s = torch.empty((B, L, H, 16), device="cuda"), torch.randn((B, H, 16, 16), device="cuda")
        g = torch.empty((B, L, H), device="cuda")
        O, S = D.fwd_lin(x, x, x, g, s)
        assert O.shape == x.shape and torch.equal(S, s)
        G = D.bwd_lin(x, x, x, g, s, x, s)
        assert G["dq"].shape == x.shape and torch.equal(G["dS0"], s)
        fixed = D.bwd_lin(x, x, x, torch.full((H,), -0.1, device="cuda"), s, x, s)
        assert (fixed["dg_log"] == 0).all()
        if L == 0:
            assert (D.fwd_lin(x, x, x)[1] == 0).all() and torch.equal(D.fwd_lin(x, x, x, g, s, S_final=s)[1], s)
    x = torch.empty((2, 5, 1, 16), device="cuda")
    v = torch.empty((2, 5, 0, 16), device="cuda")
    assert D.fwd_lin(x, x, v)[0].shape == v.shape


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets(dtype):
    """Every gate -inf: each token stands alone, and no gate has a gradient; a reset in a sequence hides
    what is before it, whatever its size."""
    c = Case(2, 150, 1, 2, 32, 32, dtype, "token", resets=range(150))
    q, k, v, g, S0 = c.dev
    O, S = D.fwd_lin(*c.dev)
    w = (q.double() * k.double()).sum(-1, keepdim=True)
    tol = HALF[dtype] * 2.02 * (w * v.double()).abs() + 40 * U * (q.double() * k.double()).abs().sum(-1, keepdim=True) * v.double().abs()
    assert ((O.double() - w * v.double()).abs() <= tol).all()
    want = k[:, -1].double().unsqueeze(-1) * v[:, -1].double().unsqueeze(-2)
    assert ((S.double() - want).abs() <= 4 * U * want.abs()).all()
    G = D.bwd_lin(*c.dev, c.devO, c.devS)
    assert (G["dg_log"] == 0).all() and (G["dS0"] == 0).all()
    t = 77
    g2 = to_dev(gates(9, 2, 150, 2, "token", (t,)), "f32")
    far = v.clone()
    far[:, :t] *= 1e4
    O1, S1 = D.fwd_lin(q, k, v, g2, S0)
    O2, S2 = D.fwd_lin(q, k, far, g2, 1e6 * S0)
    assert torch.equal(O1[:, t:], O2[:, t:]) and torch.equal(S1, S2)
    G1 = D.bwd_lin(q, k, v, g2, S0, c.devO, c.devS)
    far = c.devO.clone()
    far[:, t:] *= 1e4
    G2 = D.bwd_lin(q, k, v, g2, S0, far, c.devS)
    for n in ("dq", "dk", "dv", "dg_log"):
        assert torch.equal(G1[n][:, :t], G2[n][:, :t]), n
    assert (G1["dg_log"][:, t] == 0).all() and torch.equal(G1["dS0"], G2["dS0"])


def test_strong_gates_underflow_and_open_gates_add_up():
    x = to_dev(draw(41, (1, 400, 1, 16)), "f32")
    O, S = D.fwd_lin(x, x, x, torch.full((1, 400, 1), -86.0, device="cuda"))
    assert torch.isfinite(O).all() and torch.isfinite(S).all()
    G = D.bwd_lin(x, x, x, torch.full((1, 400, 1), -1e30, device="cuda"), None, x)
    assert all(torch.isfinite(t).all() for t in G.values())
    one = torch.ones_like(x)
    O, S = D.fwd_lin(one, one, one)
    assert torch.equal(S, torch.full_like(S, 400.0)) and torch.equal(O[0, :, 0, 0], 16 * torch.arange(1, 401, device="cuda").float())
    # gates above 1, as given: 2^(100/64) over a chunk
    g = torch.full((1, 100, 1), float(np.log(2.0) / 64), device="cuda")
    y = x[:, :100].contiguous()
    O, S = D.fwd_lin(y, y, y, g)
    Or, Sr = Lo.fwd(host(y), host(y), host(y), host(g))
    Om, Sm = Lo.fwd(np.abs(host(y)), np.abs(host(y)), np.abs(host(y)), host(g))
    check("O", O, Or, 400 * U * Om)
    check("S", S, Sr, 400 * U * Sm)


def test_non_finite_values_stay_in_their_sequence_and_head():
    c = Case(2, 300, 2, 4, 32, 32, "bf16", "token")
    q, k, v, g, S0 = c.dev
    O, S = D.fwd_lin(*c.dev)
    G = D.bwd_lin(*c.dev, c.devO, c.devS)
    for bad in (float("nan"), float("inf")):
        v2 = v.clone()
        v2[1, 130, 2, 5] = bad                            # chunk 2, value head 2
        O2, S2 = D.fwd_lin(q, k, v2, g, S0)
        G2 = D.bwd_lin(q, k, v2, g, S0, c.devO, c.devS)
        assert torch.equal(O2[0], O[0]) and torch.equal(S2[0], S[0])
        for h in (0, 1, 3):
            assert torch.equal(O2[1, :, h], O[1, :, h]) and torch.equal(G2["dv"][1, :, h], G["dv"][1, :, h])
        assert torch.equal(O2[1, :128, 2], O[1, :128, 2]) and not torch.isfinite(O2[1, 130:, 2, 5]).any()
        assert torch.equal(G2["dq"][0], G["dq"][0]) and torch.equal(G2["dk"][1, :, 0], G["dk"][1, :, 0])
        assert torch.equal(G2["dq"][1, :128], G["dq"][1, :128])
    g2 = g.clone()
    g2[0, 70, 1] = float("nan")
    O2, _ = D.fwd_lin(q, k, v, g2, S0)
    assert torch.isnan(O2[0, 70:, 1]).all() and torch.equal(O2[1], O[1]) and torch.equal(O2[0, :64, 1], O[0, :64, 1])


@pytest.mark.parametrize("B,Hk,H,dk,dv,dtype,kind", [
    (1, 1, 1, 16, 16, "bf16", "token"), (3, 1, 5, 64, 48, "f32", "head"), (64, 16, 16, 128, 128, "bf16", "token"),
    (7, 3, 3, 32, 208, "bf16", "none"), (2, 2, 8, 128, 256, "f32", "token")])
def test_decode_continues_a_prefill(B, Hk, H, dk, dv, dtype, kind):
    L, T = 70, 5
    c = Case(B, L + T, Hk, H, dk, dv, dtype, kind, resets=(L + 2,) if kind == "token" else ())
    q, k, v, g, S0 = c.dev
    cut = lambda x, a, b: x if x is None or x.dim() == 1 else x[:, a:b].contiguous()
    O, S = D.fwd_lin(*(cut(x, 0, L) for x in (q, k, v, g)), S0, scale=c.scale)
    outs = [O]
    for t in range(L, L + T):
        outs.append(D.decode_lin(*(cut(x, t, t + 1) for x in (q, k, v, g)), S, scale=c.scale))
    torch.cuda.synchronize()
    c.check_fwd(torch.cat(outs, 1), S)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hk,H,dk,dv", [
    (1, 1, 1, 128, 16), (2101, 1, 3, 16, 16), (1031, 5, 5, 16, 48), (6, 2, 2, 16, 256), (131, 3, 9, 32, 112), (515, 4, 4, 32, 32),
    (41, 1, 7, 128, 112), (31, 5, 5, 64, 80), (3, 3, 3, 128, 240), (257, 2, 8, 64, 64), (9, 1, 1, 64, 144)])
def test_decode_widths(B, Hk, H, dk, dv, dtype):
    """States that share a workgroup, slabs with a narrower last one, and what lies behind the tensors left as it was.
    Bounds: a state's element has three roundings and expf's (4 u); o a sum of dk products, each of which carries its
    state's error, and its own rounding."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")
    q, k, v = r(B, 1, Hk, dk).to(t), r(B, 1, Hk, dk).to(t), r(B, 1, H, dv).to(t)
    g = -torch.rand((B, 1, H), generator=gen, device="cuda")
    n, m, pad = B * H * dk * dv, B * H * dv, 64
    flat, out = torch.full((n + pad,), 7.0, device="cuda"), torch.full((m + pad,), 7.0, device="cuda", dtype=t)
    S0 = r(B, H, dk, dv)
    S = flat[:n].view(B, H, dk, dv).copy_(S0)
    O = D.decode_lin(q, k, v, g, S, scale=0.5, O=out[:m].view(B, 1, H, dv))
    assert bool((flat[n:] == 7).all()) and bool((out[m:] == 7).all())
    u, rep = 2.0 ** -24, H // Hk
    Q, K = (x.double().repeat_interleave(rep, 2)[:, 0] for x in (q, k))
    decayed, taken = g.double().exp()[:, 0, :, None, None] * S0.double(), K[..., None] * v.double()[:, 0, :, None, :]
    ref, mag = decayed + taken, decayed.abs() + taken.abs()
    assert bool(((S.double() - ref).abs() <= 6 * u * mag).all())
    o = 0.5 * (Q[..., None] * ref).sum(2)
    tol = 0.5 * (dk + 8) * u * (Q.abs()[..., None] * mag).sum(2)
    half = torch.finfo(t).eps / 2
    assert bool(((O.double()[:, 0] - o).abs() <= tol * (1 + half) + half * o.abs()).all())


def test_offsets_past_32_bits():
    """2.3e9 elements of each tensor: the last sequence against a call on it alone (which is split into
    segments, where the whole batch is not), and the states of both."""
    B, L, H, d = 17, 65536, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((B, L, H, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    g = torch.empty((B, L, H), device="cuda").uniform_(-0.5, -0.001, generator=gen)
    near = lambda a, b, tol: float((a.double() - b.double()).norm() / b.double().norm()) <= tol
    O, S = D.fwd_lin(x, x, x, g)
    O1, S1 = D.fwd_lin(x[-1:], x[-1:], x[-1:], g[-1:])
    # two evaluations of one value: the operands' roundings are other ones, the output's the same or the next
    assert near(O[-1:], O1, 2.0 ** -7) and near(S[-1:], S1, 1e-5)
    del O, O1
    G = D.bwd_lin(x, x, x, g, None, x)
    G1 = D.bwd_lin(x[-1:], x[-1:], x[-1:], g[-1:], None, x[-1:])
    for n in ("dq", "dk", "dv"):
        assert near(G[n][-1:], G1[n], 2.0 ** -7), n
    assert near(G["dg_log"][-1:], G1["dg_log"], 4e-5) and near(G["dS0"][-1:], G1["dS0"], 1e-5)


# ---- graphs, streams, refusals ----------------------------------------------------------------------

def calls(c):
    return {"fwd": lambda **kw: D.fwd_lin(*c.dev, scale=c.scale, **kw),
            "bwd": lambda **kw: list(D.bwd_lin(*c.dev, c.devO, c.devS, scale=c.scale, **kw).values())}


@pytest.mark.parametrize("kind", ["fwd", "bwd", "decode"])
def test_graph_replays(kind):
    """Replays with the program's own eager work and synchronisations between them, on inputs that change;
    an eager autograd graph over the same leaves lives meanwhile."""
    c = Case(2, 700, 1, 2, 64, 64, "bf16", "token")
    leaf = c.dev[2].clone().requires_grad_()
    alive = (leaf * 2).sum()
    if kind == "decode":
        one = [x[:, :1].contiguous() for x in c.dev[:4]]
        S, start = c.dev[4].clone(), c.dev[4]
        f = lambda: [D.decode_lin(*one, S), S]
    else:
        f = lambda: calls(c)[kind]()
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = f()
    for i in range(3):
        v = c.dev[2]
        v.copy_(to_dev(draw(60 + i, tuple(v.shape), "bf16"), "bf16"))
        if kind == "decode":
            one[2].copy_(v[:, :1])
            S.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        if kind == "decode":
            S.copy_(start)
        for a, b in zip(got, f()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
    alive.backward()
    assert torch.equal(leaf.grad, torch.full_like(leaf, 2.0))


def test_on_another_stream_and_two_at_once():
    cs = [Case(1, 2000, 1, 2, 64, 64, "bf16", "token", seed=s) for s in (0, 50)]
    ref = [(calls(c)["fwd"](), calls(c)["bwd"]()) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = [(calls(c)["fwd"](stream=s), calls(c)["bwd"](stream=s)) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        for (rf, rb), (gf, gb) in zip(ref, got):
            for a, b in zip(list(rf) + rb, list(gf) + gb):
                assert torch.equal(a, b)
    with torch.cuda.stream(streams[0]):
        again = calls(cs[0])["bwd"]()
    streams[0].synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, ref[0][1]))


def test_captured_calls_of_one_workspace():
    """Two graphs whose calls share a workspace, replayed one after the other, in either order."""
    cs = [Case(1, 1500, 2, 2, 64, 64, "bf16", "token", seed=s) for s in (0, 50)]
    ref = [[t.clone() for t in calls(c)["bwd"]()] for c in cs]
    ws = torch.empty(D.bwd_lin_workspace_bytes(1, 1500, 2, 2, 64, 64), dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for c in cs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(calls(c)["bwd"](workspace=ws))
    for order in ((0, 1), (1, 0), (0, 0), (1, 1)):
        for o in outs:
            for t in o:
                t.zero_()
        ws.fill_(255)                                      # NaN wherever it is read before it is written
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(order):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], ref[i]))


def test_calls_from_several_threads():
    import threading
    cs = [Case(1, 900, 1, 1, 32, 64, "bf16", "token", seed=s) for s in (0, 50, 100, 150)]
    ref = [calls(c)["bwd"]() for c in cs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(5):
            got = calls(cs[i])["bwd"](stream=s)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, ref[i])):
                bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_binding_refusals():
    q, v, s = torch.zeros(1, 4, 2, 32, device="cuda"), torch.zeros(1, 4, 4, 16, device="cuda"), torch.zeros(1, 4, 32, 16, device="cuda")
    g = torch.zeros(1, 4, 4, device="cuda")
    one = lambda x: x[:, :1].contiguous()
    for i, (err, f) in enumerate([
            (ValueError, lambda: D.fwd_lin(q[0], q[0], v)), (ValueError, lambda: D.fwd_lin(q, q, v[0])),
            (TypeError, lambda: D.fwd_lin(q.half(), q.half(), v.half())), (TypeError, lambda: D.fwd_lin(q, q.bfloat16(), v)),
            (ValueError, lambda: D.fwd_lin(q, q[:, :3], v)), (ValueError, lambda: D.fwd_lin(q, q, v[:, :, :3].contiguous())),
            (ValueError, lambda: D.fwd_lin(q, q, v[:, :, :0].contiguous().expand(1, 4, 0, 16), g)),
            (ValueError, lambda: D.fwd_lin(q, q, v, g[:, :, :2].contiguous())), (ValueError, lambda: D.fwd_lin(q, q, v, g[:, 0])),
            (ValueError, lambda: D.fwd_lin(q, q, v, torch.zeros(2, device="cuda"))), (TypeError, lambda: D.fwd_lin(q, q, v, g.double())),
            (ValueError, lambda: D.fwd_lin(q, q, v, g, s[:, :2])), (ValueError, lambda: D.fwd_lin(q, q, v, g.cpu())),
            (ValueError, lambda: D.fwd_lin(q.transpose(1, 2), q.transpose(1, 2), v)),
            (ValueError, lambda: D.fwd_lin(q, q, v, g, O=torch.empty_like(q))),
            (D.DeltaError, lambda: D.fwd_lin(q, q, v, g, s, O=v)),
            (ValueError, lambda: D.fwd_lin(q, q, v, g, workspace=torch.empty(10))),
            (ValueError, lambda: D.bwd_lin(q, q, v, g, s, q)), (ValueError, lambda: D.bwd_lin(q, q, v, g, s, v, grads={"dO": v})),
            (ValueError, lambda: D.bwd_lin(q, q, v, None, s, v, grads={"dg_log": g})),
            (D.DeltaError, lambda: D.bwd_lin(q, q, v, g, s, v, grads={"dv": v})),
            (D.DeltaError, lambda: D.bwd_lin(q, q, v, g, s, v, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
            (ValueError, lambda: D.decode_lin(q, q, v, g, s)), (ValueError, lambda: D.decode_lin(one(q), one(q), one(v), one(g), s[:, :, :16].contiguous())),
            (D.DeltaError, lambda: D.fwd_lin(torch.zeros(1, 4, 1, 48, device="cuda"), torch.zeros(1, 4, 1, 48, device="cuda"), v)),
            (D.DeltaError, lambda: D.fwd_lin(q, q, torch.zeros(1, 4, 4, 24, device="cuda")))]):
        with pytest.raises(err):
            say("refusal", i)
            f()
    torch.cuda.synchronize()


def test_validate_switch(monkeypatch):
    monkeypatch.setenv("DELTA_VALIDATE", "1")
    x, s = torch.zeros(1, 3000, 1, 16, device="cuda"), torch.zeros(1, 1, 16, 16, device="cuda")
    g = torch.zeros(1, 3000, 1, device="cuda")
    g[0, 5] = -float("inf")
    D.fwd_lin(x, x, x, g)                                 # -inf is a reset, not an error
    for v in (float("nan"), float("inf")):
        g[0, 2999, 0] = v
        one = x[:, :1].contiguous()
        for f in (lambda: D.fwd_lin(x, x, x, g), lambda: D.bwd_lin(x, x, x, g, s, x), lambda: D.fwd_lin(x, x, x, torch.full((1,), v, device="cuda")),
                  lambda: D.decode_lin(one, one, one, g[:, 2999:].contiguous(), s)):
            with pytest.raises(D.DeltaError) as e:
                f()
            assert e.value.code == -8
