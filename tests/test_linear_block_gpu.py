"""Linear attention, the layer norm and dropout together, as a stack uses them: a block's training step
against autograd in 64 bits, and its serving steps against the whole sequence."""
import numpy as np
import pytest

from oracle import layernorm as Ln
from oracle import linear as Lo
from parity import say, to_dev

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import chunkwise_delta_rule_chunked_amd as D  # noqa: E402

U = 2.0 ** -24


def draw(seed, *shape):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32))


@pytest.mark.parametrize("gate", ["token", "head"])
def test_a_training_step_of_a_block(gate):
    """Norm (with the branch before it dropped and added) -> projections -> linear attention with gates from a
    projection or fixed decays to learn -> projection -> dropout, residual and the next norm; forward, backward
    and clipping.  Tolerance: the chain is 10 stages whose longest sum has 128 terms; each adds at most (128 + 64)
    u of the magnitudes it handles, and the block's gain on them is below 8: 10 * 192 * 8 * u = 9e-4 of the
    2-norm."""
    B, L, Hk, H, dk, dv, p = 2, 200, 1, 2, 32, 64, 0.2
    W = H * dv
    P = {"x": draw(1, B, L, W), "res": draw(2, B, L, W), "w1": 1 + 0.1 * draw(3, W), "b1": 0.1 * draw(4, W), "w2": 1 + 0.1 * draw(5, W),
         "b2": 0.1 * draw(6, W), "Wq": draw(7, W, Hk * dk) / W ** 0.5, "Wk": draw(8, W, Hk * dk) / W ** 0.5, "Wv": draw(9, W, W) / W ** 0.5,
         "Wo": draw(10, W, W) / W ** 0.5, "Wg": draw(11, W, H) / W ** 0.5, "fixed": -draw(12, H).abs(), "S0": draw(13, B, H, dk, dv)}
    dy, ds2 = draw(14, B, L, W), draw(15, B, L, W)
    drop = [dict(p=p, seed=99, offset=i) for i in range(2)]
    f = [torch.from_numpy(Ln.factors(B * L, W, p, 99, i)).view(B, L, W) for i in range(2)]

    def f64():
        t = {k: v.double().requires_grad_() for k, v in P.items()}
        norm = lambda s, w, b: (s - s.mean(-1, keepdim=True)) / torch.sqrt(s.var(-1, keepdim=True, correction=0) + 1e-5) * w + b
        s1 = t["x"] * f[0] + t["res"]
        y1 = norm(s1, t["w1"], t["b1"])
        q, k, v = (y1 @ t["Wq"]).view(B, L, Hk, dk), (y1 @ t["Wk"]).view(B, L, Hk, dk), (y1 @ t["Wv"]).view(B, L, H, dv)
        g = -torch.nn.functional.softplus(y1 @ t["Wg"]) if gate == "token" else t["fixed"].expand(B, L, H)
        S, out = t["S0"], []
        for i in range(L):
            S = torch.exp(g[:, i])[..., None, None] * S + k[:, i].repeat_interleave(H, 1)[..., None] * v[:, i, :, None]
            out.append(dk ** -0.5 * (q[:, i].repeat_interleave(H, 1)[..., None] * S).sum(2))
        s2 = (torch.stack(out, 1).view(B, L, W) @ t["Wo"]) * f[1] + s1
        y2 = norm(s2, t["w2"], t["b2"])
        ((y2 * dy.double()).sum() + (s2 * ds2.double()).sum()).backward()
        return y2.detach(), {k: v.grad for k, v in t.items() if v.grad is not None}

    q = {k: v.cuda() for k, v in P.items()}
    T = lambda m: m.t().contiguous()
    s1, y1 = D.layer_layernorm(q["x"], q["w1"], q["b1"], q["res"], **drop[0])
    yf = y1.view(-1, W)
    Q, K, V = (yf @ q["Wq"]).view(B, L, Hk, dk), (yf @ q["Wk"]).view(B, L, Hk, dk), (yf @ q["Wv"]).view(B, L, H, dv)
    z = yf @ q["Wg"]
    g = -torch.nn.functional.softplus(z).view(B, L, H) if gate == "token" else q["fixed"]
    O, _ = D.fwd_lin(Q, K, V, g, q["S0"], scale=dk ** -0.5, want_state=False)
    s2, y2 = D.layer_layernorm((O.view(-1, W) @ q["Wo"]).view(B, L, W), q["w2"], q["b2"], s1, **drop[1])
    n2 = D.layer_layernorm_bwd(dy.cuda(), s2, q["w2"], ds2.cuda(), **drop[1])
    dm = n2["dx"].view(-1, W)
    G = D.bwd_lin(Q, K, V, g, q["S0"], (dm @ T(q["Wo"])).view(B, L, H, dv), scale=dk ** -0.5)
    dQ, dK, dV = G["dq"].view(-1, Hk * dk), G["dk"].view(-1, Hk * dk), G["dv"].view(-1, W)
    dy1 = dQ @ T(q["Wq"]) + dK @ T(q["Wk"]) + dV @ T(q["Wv"])
    grads = {"Wq": T(yf) @ dQ, "Wk": T(yf) @ dK, "Wv": T(yf) @ dV, "Wo": T(O.view(-1, W)) @ dm, "S0": G["dS0"]}
    if gate == "token":
        dz = -G["dg_log"].view(-1, H) * torch.sigmoid(z)
        dy1 = dy1 + dz @ T(q["Wg"])
        grads["Wg"] = T(yf) @ dz
    else:
        grads["fixed"] = G["dg_log"]
    n1 = D.layer_layernorm_bwd(dy1.view(B, L, W), s1, q["w1"], n2["dresidual"], **drop[0])
    grads.update(x=n1["dx"], res=n1["dresidual"], w1=n1["dweight"], b1=n1["dbias"], w2=n2["dweight"], b2=n2["dbias"])
    y64, ref = f64()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())
    say("  y2", rel(y2, y64))
    assert rel(y2, y64) < 9e-4 and grads.keys() == ref.keys()
    for k, v in ref.items():
        say("  grad", k, rel(grads[k].view(v.shape), v))
        assert rel(grads[k].view(v.shape), v) < 9e-4, k
    n = D.clip_grads(grads, 1.0)
    n64 = torch.sqrt(sum((v ** 2).sum() for v in ref.values()))
    assert abs(float(n) / float(n64) - 1) < 9e-4


def test_serving_steps_of_a_block():
    """A prefill, then tokens one at a time through norm and mixer from a captured step, the state carried in
    place: as the oracle over the whole sequence.  Tolerance as in test_linear_gpu.py: the norm's rows are the
    same bits either way, an output's operands and the output itself are rounded to bf16, its float32 sums have
    c = 32 + 64 + 64 + 16 + 100 steps."""
    B, L, T, H, d = 3, 70, 6, 2, 32
    W = H * 64
    x, w, b = to_dev(draw(21, B, L + T, W).numpy(), "bf16"), to_dev((1 + 0.1 * draw(22, W)).numpy(), "f32"), to_dev(draw(23, W).numpy(), "f32")
    res = to_dev(draw(24, B, L + T, W).numpy(), "bf16")
    g = to_dev(-draw(25, B, L + T, H).abs().numpy(), "f32")

    def feed(x, r):
        s, y = D.layer_layernorm(x, w, b, r)
        y = y.view(*y.shape[:2], H, 64)
        return y[..., :32].contiguous(), y[..., 32:].contiguous(), y.contiguous()   # q, k and v of each head

    q, k, v = feed(x, res)
    cut = lambda t, i, j: t[:, i:j].contiguous()
    O, S = D.fwd_lin(cut(q, 0, L), cut(k, 0, L), cut(v, 0, L), cut(g, 0, L))
    xt, rt, gt = cut(x, L, L + 1), cut(res, L, L + 1), cut(g, L, L + 1)
    keep = S.clone()
    D.decode_lin(*feed(xt, rt), gt, S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = D.decode_lin(*feed(xt, rt), gt, S)
    S.copy_(keep)
    outs = [O]
    for t in range(L, L + T):
        xt.copy_(x[:, t:t + 1]), rt.copy_(res[:, t:t + 1]), gt.copy_(g[:, t:t + 1])
        graph.replay()
        outs.append(o.clone())
    torch.cuda.synchronize()
    host = lambda t: t.float().cpu().numpy().astype(np.float64)
    args = (host(q), host(k), host(v), host(g))
    Or, Sr = Lo.fwd(*args)
    Om, Sm = Lo.fwd(*(np.abs(a) for a in args[:3]), args[3])
    c = 276 * U
    assert (np.abs(host(torch.cat(outs, 1)) - Or) <= (2.0 ** -8 + c) * Om * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(Or) + 1e-36).all()
    assert (np.abs(host(S) - Sr) <= c * Sm + 1e-36).all()
