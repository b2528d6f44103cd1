"""GPU parity of the layer norm and of dropout (include/delta_layernorm.h) with the fp64 oracle in
oracle/layernorm.py.

Tolerances are elementwise and derived from the arithmetic, with u = 2^-24 the float32 half step:
  * a sum of D values held in 64 or more partial sums: (D / 64 + 16) u of its magnitudes.
  * a deviation s - mean carries u of itself and that much of the row's mean deviation (what rounding left
    of the mean itself is taken out again), so z = (s - mean) / sqrt(var + eps) is good to
    rel (|z| + 1), rel = (D / 64 + 24) u; products with it inherit that.
  * the outputs' own rounding: half a step of their type, eps / 2 relative.
"""
import numpy as np
import pytest

from oracle import layernorm as Ln
from parity import say, to_dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def draw(seed, shape, dtype="f32"):
    x = np.random.default_rng(seed).standard_normal(shape).astype(np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x


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
    say("  %s: max error / bound %.3f" % (name, over.max()))
    assert over.max() <= 1.0, (name, float(over.max()), np.unravel_index(over.argmax(), over.shape))


def half(v, dtype):
    return HALF[dtype] * np.abs(v) + 1e-38


ROWS = [(1, 1), (1, 16), (3, 7), (5, 63), (2, 64), (17, 100), (4, 128), (64, 129), (9, 512), (1, 1000), (33, 1003), (6, 2048),
        (257, 300), (3, 4096), (2, 4104), (5, 8192), (1, 8200), (2, 16384), (1, 16392), (2, 20001), (3000, 24)]


# ---- dropout ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_dropout(N, W, dtype):
    say("dropout", N, W, dtype)
    p, seed, offset = 0.3, (1 << 63) + 12345, (7 << 32) + N
    x, r = draw(1, (N, W), dtype), draw(2, (N, W), dtype)
    f = Ln.factors(N, W, p, seed, offset)
    xd, rd = to_dev(x, dtype), to_dev(r, dtype)
    kw = dict(p=p, seed=seed, offset=offset)
    y = D.layer_dropout(xd, **kw)
    # one float32 product by a factor that is itself rounded, then the output's rounding
    check("y", y, f * x, 2 * U * np.abs(f * x) + half(f * x, dtype))
    assert ((host(y) == 0) == (f * x == 0)).all()
    s = D.layer_dropout(xd, rd, **kw)
    check("y + residual", s, f * x + r, 4 * U * (np.abs(f * x) + np.abs(r)) + half(f * x + r, dtype))
    a, b = xd.clone(), rd.clone()
    assert D.layer_dropout(a, **kw, y=a) is a and torch.equal(a, y)
    assert D.layer_dropout(xd, b, **kw, y=b) is b and torch.equal(b, s)
    a = xd.clone()
    assert torch.equal(D.layer_dropout(a, rd, **kw, y=a), s)
    step = torch.tensor(offset, dtype=torch.int64, device="cuda")
    assert torch.equal(D.layer_dropout(xd, rd, p=p, seed=seed, offset=step), s)


def test_dropout_extremes():
    x = torch.ones(100, 1003, device="cuda")
    assert torch.equal(D.layer_dropout(x, p=0.0, seed=1), x) and (D.layer_dropout(x, p=1.0, seed=1) == 0).all()
    assert torch.equal(D.layer_dropout(x, p=2.0 ** -18, seed=1), x)
    assert torch.equal(D.layer_dropout(x, x, p=1.0, seed=1), x)
    bad = torch.full_like(x, float("nan"))
    y = D.layer_dropout(bad, p=0.5, seed=3)
    assert torch.equal(y == 0, D.layer_dropout(x, p=0.5, seed=3) == 0) and torch.isnan(y[y != 0]).all()
    # the largest p below 1, the kept ones at 65536 times their value
    y = D.layer_dropout(torch.ones(512, 2048, device="cuda"), p=1 - 2.0 ** -16, seed=5)
    assert set(y.unique().tolist()) <= {0.0, 65536.0} and 0 < int((y != 0).sum()) < 64
    for p in (0.1, 0.25, 0.9):
        y = D.layer_dropout(torch.ones(1024, 2048, device="cuda"), p=p, seed=9)
        share = round(p * 65536) / 65536
        assert abs(float((y == 0).double().mean()) - share) < 5 * (share * (1 - share) / y.numel()) ** 0.5
        assert abs(float(y.double().mean()) - 1) < 5 * (share / (1 - share) / y.numel()) ** 0.5


def test_dropout_masks_differ_between_calls_and_not_between_batches():
    x = torch.ones(64, 200, device="cuda")
    keep = lambda x, **kw: D.layer_dropout(x, p=0.5, **kw) != 0
    a = keep(x, seed=1)
    for kw in (dict(seed=2), dict(seed=1, offset=1), dict(seed=1 + (1 << 32)), dict(seed=1, offset=1 << 32)):
        agree = float((keep(x, **kw) == a).double().mean())
        assert abs(agree - 0.5) < 5 * 0.5 / a.numel() ** 0.5, kw
    assert torch.equal(keep(x[:7].contiguous(), seed=1), a[:7])
    assert torch.equal(keep(x.view(8, 8, 200), seed=1).view(64, 200), a)
    assert torch.equal(keep(x.bfloat16(), seed=1), a)
    # a row's vectors end with it: 1003 channels use the first of 1008's bits
    wide = torch.ones(5, 1008, device="cuda")
    assert torch.equal(keep(wide, seed=4)[:, :1003], keep(wide[:, :1003].contiguous(), seed=4))


def test_dropout_past_32_bits():
    """4.3e9 elements: rows past the 2^32nd element against the oracle's bits."""
    N, W = (1 << 22) + 3, 1027
    x = torch.ones(N, W, dtype=torch.bfloat16, device="cuda")
    y = D.layer_dropout(x, p=0.5, seed=11, y=x)
    blocks = -(-W // 8)
    for row in (0, N // 2, N - 1):
        bits = []
        for n in range(row * blocks, (row + 1) * blocks):
            for w in Ln.philox([n & Ln.MASK, n >> 32, 0, 0], [11, 0]):
                bits += [w & 0xFFFF, w >> 16]
        assert np.array_equal(host(y[row]), 2.0 * (np.array(bits[:W]) >= 32768)), row


# ---- layer norm ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_layernorm(N, W, dtype, p):
    say("layernorm", N, W, dtype, p)
    x, r = draw(31, (N, W), dtype), 2 * draw(32, (N, W), dtype)
    w, b = (1 + 0.2 * draw(33, (W,))).astype(np.float32), draw(34, (W,))
    x[0], r[0] = 0.0, 0.0                                # a row of zeros
    xd, rd, wd, bd = to_dev(x, dtype), to_dev(r, dtype), to_dev(w, "f32"), to_dev(b, "f32")
    kw = dict(p=p, seed=5, offset=3)
    s, y = D.layer_layernorm(xd, wd, bd, rd, eps=1e-5, **kw)
    assert torch.equal(s, D.layer_dropout(xd, rd, **kw))
    ref, z, _ = Ln.layernorm(host(s), w, b, 1e-5)
    rel = (W / 64 + 24) * U
    bound = rel * np.abs(w) * (np.abs(z) + 1) + 2 * U * np.abs(b)
    check("y", y, ref, bound + half(np.abs(ref) + bound, dtype))
    s0, y0 = D.layer_layernorm(s, wd, bd, eps=1e-5)      # no residual, nothing dropped: x itself, the same bits
    assert s0 is s and torch.equal(y0, y)
    s1, y1 = D.layer_layernorm(xd, wd, eps=1e-5, **kw)   # no residual, no bias
    assert torch.equal(s1, D.layer_dropout(xd, **kw)) and (s1 is xd) == (p == 0)
    ref, z, _ = Ln.layernorm(host(s1), w, None, 1e-5)
    bound = rel * np.abs(w) * (np.abs(z) + 1)
    check("y without residual", y1, ref, bound + half(np.abs(ref) + bound, dtype))
    for i in range(2):
        t = [xd.clone(), rd.clone()]
        s2, y2 = D.layer_layernorm(t[0], wd, bd, t[1], eps=1e-5, **kw, sum=t[i])
        assert s2 is t[i] and torch.equal(s2, s) and torch.equal(y2, y)


@pytest.mark.parametrize("W", [100, 2048, 8192, 20001])
def test_rows_far_from_zero(W):
    """A mean of 1e5 times the spread: the variance is that of the rounded values, not of a difference of
    large sums."""
    s = (1e5 + draw(41, (7, W))).astype(np.float32)
    w, dy = (1 + 0.2 * draw(42, (W,))).astype(np.float32), draw(43, (7, W))
    sd, wd, dyd = to_dev(s, "f32"), to_dev(w, "f32"), to_dev(dy, "f32")
    _, y = D.layer_layernorm(sd, wd, eps=1e-5)
    ref, z, _ = Ln.layernorm(s, w, None, 1e-5)
    # the first mean is off by at most (W / 64 + 16) u of 1e5; deviations from it are exact (Sterbenz), its own
    # deviation's square is taken out again at (off)^2 u
    off = (W / 64 + 16) * U * 1e5
    rel = (W / 64 + 24) * U * (1 + off) ** 2
    check("y", y, ref, rel * np.abs(w) * (np.abs(z) + 1) + half(ref, "f32"))
    G = D.layer_layernorm_bwd(dyd, sd, wd, eps=1e-5)
    ds, dw, db = Ln.layernorm_bwd(dy, s, w, None, 1e-5)
    mag = np.abs(w * dy) + np.mean(np.abs(w * dy), 1, keepdims=True) + (np.abs(z) + 1) * np.mean(np.abs(w * dy) * (np.abs(z) + 1), 1, keepdims=True)
    check("ds", G["dresidual"], ds, 4 * rel * mag * Ln.layernorm(s, w, None, 1e-5)[2])


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", ROWS)
def test_layernorm_bwd(N, W, dtype, p):
    say("layernorm bwd", N, W, dtype, p)
    s, dy, ds = 2 * draw(51, (N, W), dtype) + np.float32(0.5), draw(52, (N, W), dtype), draw(53, (N, W), dtype)
    w = (1 + 0.2 * draw(54, (W,))).astype(np.float32)
    eps, kw = 1e-2, dict(p=p, seed=77, offset=1)
    dev = [to_dev(dy, dtype), to_dev(s, dtype), to_dev(w, "f32"), to_dev(ds, dtype)]
    s = host(dev[1])                                     # 2 x + 0.5 rounded
    G = D.layer_layernorm_bwd(*dev, eps=eps, **kw)
    ref, rw, rb = Ln.layernorm_bwd(dy, s, w, ds, eps)
    _, z, r = Ln.layernorm(s, w, None, eps)
    wd, zz = np.abs(w * dy), np.abs(z) + 1
    mag = np.abs(ds) + r * (wd + wd.mean(1, keepdims=True) + zz * (wd * zz).mean(1, keepdims=True))
    rel = (W / 64 + 32) * U
    check("dresidual", G["dresidual"], ref, rel * mag + half(ref, dtype) + half(rel * mag, dtype))
    f = Ln.factors(N, W, p, 77, 1)
    check("dx", G["dx"], f * ref, f * (rel + 2 * U) * mag + half(f * ref, dtype) + half(f * rel * mag, dtype))
    # sums over N rows in float32, in any order
    check("dweight", G["dweight"], rw, (N + W / 64 + 32) * U * np.sum(np.abs(dy) * zz, axis=0) + 1e-38)
    check("dbias", G["dbias"], rb, N * U * np.sum(np.abs(dy), axis=0) + 1e-38)
    assert (G["dx"] is G["dresidual"]) == (p == 0)
    G2 = D.layer_layernorm_bwd(*dev, eps=eps, **kw)
    assert all(torch.equal(G[n], G2[n]) for n in G)
    for a, b in ((False, True), (True, False), (False, False)):
        G3 = D.layer_layernorm_bwd(*dev, eps=eps, **kw, want_dweight=a, want_dbias=b)
        assert torch.equal(G3["dx"], G["dx"])
        for n, want in (("dweight", a), ("dbias", b)):
            assert torch.equal(G3[n], G[n]) if want else G3[n] is None
    G4 = D.layer_layernorm_bwd(*dev[:3], eps=eps, **kw)  # no residual gradient
    check("dresidual without dsum", G4["dresidual"], ref - ds, rel * mag + half(ref - ds, dtype) + half(rel * mag, dtype))


@pytest.mark.parametrize("N,W", [(70000, 40), (9001, 1003), (5000, 2048), (1500, 4100), (1100, 9000), (700, 17000)])
def test_more_rows_than_workgroups(N, W):
    """Workgroups that walk over rows: every row as in a call on a few rows."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    x, res, w, b = r(N, W), r(N, W), 1 + 0.1 * r(W).float(), r(W).float()
    s, y = D.layer_layernorm(x, w, b, res)
    G = D.layer_layernorm_bwd(x, s, w, res)
    for a in (0, N // 2 + 1, N - 5):
        cut = lambda t: t[a:a + 5].contiguous()
        s1, y1 = D.layer_layernorm(cut(x), w, b, cut(res))
        assert torch.equal(s1, cut(s)) and torch.equal(y1, cut(y))
        assert torch.equal(D.layer_layernorm_bwd(cut(x), s1, w, cut(res))["dx"], cut(G["dx"]))
    z = (s.double() - s.double().mean(1, keepdim=True)) / torch.sqrt(s.double().var(1, keepdim=True, correction=0) + 1e-5)
    for n, ref, mag in (("dweight", (x.double() * z).sum(0), (x.double().abs() * (z.abs() + 1)).sum(0)),
                        ("dbias", x.double().sum(0), x.double().abs().sum(0))):
        # a column's sum over its rows in at most N / 256 + 600 steps one after another
        assert ((G[n].double() - ref).abs() <= (N / 256 + 600 + W / 64 + 32) * U * mag).all(), n


@pytest.mark.parametrize("N,W", [(200001, 40), (25001, 1000), (13001, 2048), (2001, 4096), (4200, 16392)])
def test_more_rows_than_forward_workgroups(N, W):
    """The forward pass has more workgroups before they walk; with dropout, whose mask goes by the row."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    x, res, w, b = r(N, W), r(N, W), 1 + 0.1 * r(W).float(), r(W).float()
    s, y = D.layer_layernorm(x, w, b, res, p=0.25, seed=9)
    assert torch.equal(s, D.layer_dropout(x, res, p=0.25, seed=9))
    assert torch.equal(y, D.layer_layernorm(s, w, b)[1])
    for a in (0, N // 2 + 1, N - 5):
        assert torch.equal(D.layer_layernorm(s[a:a + 5].contiguous(), w, b)[1], y[a:a + 5])


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,W", [(1, 1024), (4103, 1024), (1031, 2048), (517, 4096), (259, 8192)])
def test_backward_rows_at_any_element(N, W, dtype, p):
    """Rows of whole vectors that start on 16 bytes are loaded a step ahead, others are not: both against float64, with
    rows behind the tensors left as they were."""
    say("layernorm bwd, rows at an odd element", N, W, dtype, p)
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = torch.bfloat16 if dtype == "bf16" else torch.float32
    flat = [torch.randn((N + 2) * W + 1, generator=gen, device="cuda").to(t) for _ in range(3)]
    w = 1 + 0.1 * torch.randn(W, generator=gen, device="cuda")
    for off in (0, 1):
        s, dy, ds = (f[off:off + N * W].view(N, W) for f in flat)
        outs = [torch.full(((N + 2) * W + 1,), 7.0, dtype=t, device="cuda") for _ in range(2)]
        names = ("dresidual", "dx") if p else ("dresidual",)
        G = D.layer_layernorm_bwd(dy, s, w, ds, eps=1e-2, p=p, seed=5,
                                  grads={n: o[off:off + N * W].view(N, W) for n, o in zip(names, outs)})
        for o in outs[:len(names)]:
            assert bool((o[:off] == 7).all()) and bool((o[off + N * W:] == 7).all())
        S, Y = s.double(), dy.double()
        rstd = 1 / torch.sqrt(S.var(1, keepdim=True, correction=0) + 1e-2)
        z, wd = (S - S.mean(1, keepdim=True)) * rstd, w.double() * Y
        ref = ds.double() + rstd * (wd - wd.mean(1, keepdim=True) - z * (wd * z).mean(1, keepdim=True))
        # as in test_layernorm_bwd, the dropped channels' reference through the same mask
        zz = z.abs() + 1
        mag = ds.double().abs() + rstd * (wd.abs() + wd.abs().mean(1, keepdim=True) + zz * (wd.abs() * zz).mean(1, keepdim=True))
        rel = (W / 64 + 32) * U
        check("dresidual", G["dresidual"], ref.cpu().numpy(), (rel * mag * (1 + HALF[dtype]) + HALF[dtype] * ref.abs() + 1e-38).cpu().numpy())
        if p:
            f = D.layer_dropout(torch.ones(N, W, device="cuda"), p=p, seed=5).double()
            check("dx", G["dx"], (f * ref).cpu().numpy(),
                  (f * ((rel + 2 * U) * mag * (1 + HALF[dtype]) + (HALF[dtype] + U) * ref.abs()) + 1e-38).cpu().numpy())
        check("dweight", G["dweight"], (Y * z).sum(0).cpu().numpy(), ((N + W / 64 + 32) * U * (Y.abs() * zz).sum(0) + 1e-38).cpu().numpy())
        check("dbias", G["dbias"], Y.sum(0).cpu().numpy(), (N * U * Y.abs().sum(0) + 1e-38).cpu().numpy())


def test_special_rows():
    W = 300
    x = np.ones((6, W), dtype=np.float32)
    x[1, 3], x[2, 299], x[3] = np.nan, np.inf, 7.25
    x[4] = draw(61, (W,)) * 1e17                         # squares to 1e34 each
    x[5] = draw(62, (W,)) * 1e-17
    w, b = torch.ones(W, device="cuda"), torch.full((W,), 0.5, device="cuda")
    xd = to_dev(x, "f32")
    _, y = D.layer_layernorm(xd, w, b, eps=1e-5)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert (y[0] == 0.5).all() and (y[3] == 0.5).all()   # constant rows: the bias
    ref = Ln.layernorm(x[4:5], np.ones(W), np.full(W, 0.5), 1e-5)[0]
    check("large", y[4:5], ref, (W / 64 + 24) * U * (np.abs(ref) + 1.5) + half(ref, "f32"))
    assert torch.allclose(y[5], b, atol=1e-12)
    G = D.layer_layernorm_bwd(torch.ones_like(xd), xd, w, eps=1e-5)
    assert torch.isnan(G["dx"][1]).all() and torch.isfinite(G["dx"][[0, 3, 4, 5]]).all()


def test_no_rows():
    x, w = torch.empty((0, 32), device="cuda"), torch.ones(32, device="cuda")
    assert D.layer_layernorm(x, w, w, x, p=0.1)[1].shape == (0, 32)
    assert D.layer_dropout(x, p=0.5, seed=1).shape == (0, 32)
    G = D.layer_layernorm_bwd(x, x, w)
    assert G["dx"].shape == (0, 32) and (G["dweight"] == 0).all() and (G["dbias"] == 0).all()


# ---- graphs, streams, refusals ------------------------------------------------------------------------

def test_graph_replays_draw_anew():
    """A captured step that advances its own offset: every replay has the mask of its number, forward and
    backward the same one; an eager autograd graph over a leaf of the call lives meanwhile."""
    N, W = 300, 520
    x, res, dy = (to_dev(draw(70 + i, (N, W)), "f32") for i in range(3))
    leaf = torch.ones(W, device="cuda", requires_grad=True)
    alive = (leaf * 3).sum()
    w, step = leaf.detach(), torch.zeros((), dtype=torch.int64, device="cuda")
    eager = lambda n: (D.layer_layernorm(x, w, None, res, p=0.25, seed=6, offset=n),
                       D.layer_layernorm_bwd(dy, D.layer_layernorm(x, w, None, res, p=0.25, seed=6, offset=n)[0], w, p=0.25, seed=6, offset=n))
    eager(0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s, y = D.layer_layernorm(x, w, None, res, p=0.25, seed=6, offset=step)
        G = D.layer_layernorm_bwd(dy, s, w, p=0.25, seed=6, offset=step)
        d = D.layer_dropout(dy, p=0.25, seed=6, offset=step)
        step.add_(1)
    for n in range(4):
        graph.replay()
        torch.cuda.synchronize()
        (s2, y2), G2 = eager(n)
        assert torch.equal(s, s2) and torch.equal(y, y2) and torch.equal(d, D.layer_dropout(dy, p=0.25, seed=6, offset=n))
        for k in G:
            assert torch.equal(G[k], G2[k]), (n, k)
    alive.backward()
    assert torch.equal(leaf.grad, torch.full_like(leaf, 3.0))


def test_streams_and_threads():
    import threading
    N, W = 2000, 1003
    w = torch.ones(W, device="cuda")
    ins = [to_dev(draw(80 + i, (N, W), "bf16"), "bf16") for i in range(4)]
    run = lambda i, **kw: (*D.layer_layernorm(ins[i], w, w, ins[i], p=0.1, seed=i, **kw),
                           *D.layer_layernorm_bwd(ins[i], ins[i], w, p=0.1, seed=i, **kw).values())
    ref = [run(i) for i in range(4)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        for _ in range(5):
            got = run(i, stream=st)
            st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, ref[i])):
                bad.append(i)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not bad


def test_workspace_contents_are_ignored():
    x, w = to_dev(draw(90, (500, 300)), "f32"), torch.ones(300, device="cuda")
    G = D.layer_layernorm_bwd(x, x, w)
    ws = torch.full((D.layernorm_bwd_workspace_bytes(500, 300, D.F32) // 4,), float("nan"), device="cuda")
    G2 = D.layer_layernorm_bwd(x, x, w, workspace=ws)
    assert all(torch.equal(G[n], G2[n]) for n in G)


def test_binding_refusals():
    x, w, t = torch.zeros(4, 32, device="cuda"), torch.ones(32, device="cuda"), torch.zeros((), dtype=torch.int64, device="cuda")
    for i, (err, f) in enumerate([
            (ValueError, lambda: D.layer_dropout(x, p=1.5, seed=1)), (ValueError, lambda: D.layer_dropout(x, p=float("nan"), seed=1)),
            (ValueError, lambda: D.layer_dropout(x, p=0.1, seed=-1)), (ValueError, lambda: D.layer_dropout(x, p=0.1, seed=1, offset=1 << 64)),
            (TypeError, lambda: D.layer_dropout(x, p=0.1, seed=1, offset=t.int())), (ValueError, lambda: D.layer_dropout(x, p=0.1, seed=1, offset=t.cpu())),
            (ValueError, lambda: D.layer_dropout(x, p=0.1, seed=1, offset=t.view(1))), (TypeError, lambda: D.layer_dropout(x.half(), p=0.1, seed=1)),
            (ValueError, lambda: D.layer_dropout(x, x[:3], p=0.1, seed=1)), (ValueError, lambda: D.layer_dropout(x.t(), p=0.1, seed=1)),
            (TypeError, lambda: D.layer_dropout(x, x.bfloat16(), p=0.1, seed=1)),
            (ValueError, lambda: D.layer_layernorm(x, w[:31])), (TypeError, lambda: D.layer_layernorm(x, w.bfloat16())),
            (ValueError, lambda: D.layer_layernorm(x, w, w[:3])), (D.DeltaError, lambda: D.layer_layernorm(x, w, eps=-1.0)),
            (D.DeltaError, lambda: D.layer_layernorm(x, w, y=x)), (ValueError, lambda: D.layer_layernorm(x, w, p=2.0)),
            (ValueError, lambda: D.layer_layernorm_bwd(x[:2], x, w)), (D.DeltaError, lambda: D.layer_layernorm_bwd(x, x, w, grads={"dx": x})),
            (ValueError, lambda: D.layer_layernorm_bwd(x, x, w, grads={"dz": x})),
            (ValueError, lambda: D.layer_layernorm_bwd(x, x, w, grads={"dx": torch.empty_like(x), "dresidual": torch.empty_like(x)})),
            (D.DeltaError, lambda: D.layer_layernorm_bwd(x, x, w, workspace=torch.empty(8, device="cuda"))),
            (ValueError, lambda: D.layer_layernorm(torch.empty(3, 0, device="cuda"), torch.empty(0, device="cuda")))]):
        with pytest.raises(err):
            say("refusal", i)
            f()
    torch.cuda.synchronize()
