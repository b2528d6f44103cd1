"""Cases of linear attention with a decay for each head, of the residual stream's layer norm and of dropout.

`run` computes an operator either in its plain form (elementary torch operations) or, where `own` is
true, through the package.  See `listed` for what each case stands for.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64
EPS = 1e-5
RESET = -150.0      # a log gate whose exp is 0 in float32 and whose sums stay finite
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pkg():
    import chunkwise_delta_rule_chunked_amd as delta
    return delta


# ---- cases -----------------------------------------------------------------------------------------

def listed():
    return [
        # prefill of one 64K-token sequence, 16 heads, a gate for each token and head, state in and out
        dict(name="lin_fwd_b1_l64k", op="lin_fwd", B=1, L=65536, Hk=16, H=16, dk=128, dv=128, dtype="bf16", gate="token"),
        # ragged float32 with a fixed decay for each head: odd batch and length, heads that share q and k
        dict(name="lin_fwd_odd_f32", op="lin_fwd", B=3, L=1237, Hk=2, H=6, dk=64, dv=80, dtype="f32", gate="head"),
        # training at the repository's 2 x 8K-token, 16-head shape, gradients of the gates too
        dict(name="lin_bwd_b2_l8k", op="lin_bwd", B=2, L=8192, Hk=16, H=16, dk=128, dv=128, dtype="bf16", gate="token"),
        # gradients over many short ragged sequences, two value heads to a query and key head
        dict(name="lin_bwd_b8_l777", op="lin_bwd", B=8, L=777, Hk=4, H=8, dk=128, dv=128, dtype="bf16", gate="token"),
        # one token for each of 64 sequences (the repository's decode batch)
        dict(name="lin_decode_b64", op="lin_decode", B=64, Hk=16, H=16, dk=128, dv=128, dtype="bf16", gate="token"),
        # one token for one sequence, where latency is all there is
        dict(name="lin_decode_b1_f32", op="lin_decode", B=1, Hk=4, H=8, dk=64, dv=128, dtype="f32", gate="head"),
        # the norm before a layer's projections while training, dropout on the branch: 2 x 8K tokens, 16 heads of 128
        dict(name="ln_fwd_16k_2048", op="ln_fwd", rows=16384, width=2048, dtype="bf16", p=0.1, bias=True),
        # a decode batch's rows in a width whose rows do not start on 16 bytes, nothing dropped
        dict(name="ln_fwd_64_1003", op="ln_fwd", rows=64, width=1003, dtype="bf16", p=0.0, bias=False),
        dict(name="ln_bwd_16k_2048", op="ln_bwd", rows=16384, width=2048, dtype="bf16", p=0.1, bias=True),
        dict(name="ln_bwd_odd_f32", op="ln_bwd", rows=3711, width=1003, dtype="f32", p=0.0, bias=True),
        # the branch dropped and added to the residual stream without a norm; and alone, an odd float32 width
        dict(name="dropout_16k_2048", op="dropout", rows=16384, width=2048, dtype="bf16", p=0.1, residual=True),
        dict(name="dropout_1237_1003", op="dropout", rows=1237, width=1003, dtype="f32", p=0.5, residual=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_bwd", "lin_bwd", "lin_decode", "ln_fwd", "ln_bwd", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op.startswith("lin"):
        c = dict(op=op, dtype=dtype, gate=rng.choice(["token", "token", "head", "none"]))
        while True:
            c["Hk"] = rng.randint(1, 32)
            c["H"] = c["Hk"] * rng.choice([1, 1, 2, 4])
            c["dk"], c["dv"] = rng.choice([16, 32, 64, 128]), 16 * rng.randint(1, 16)
            if op == "lin_decode":
                c["B"] = _log(rng, 1, 512)
                if c["B"] * c["H"] * c["dk"] * c["dv"] <= 1 << 25:
                    return c
                continue
            c["B"], c["L"] = _log(rng, 1, 16), _log(rng, 1, 65536 if op == "lin_fwd" else 16384)
            if c["B"] * c["L"] * c["H"] * (c["dk"] + c["dv"]) <= (1 << 26 if op == "lin_bwd" or dtype == "f32" else 1 << 28):
                return c
    while True:
        width = _log(rng, 16, 16384)
        if rng.random() < 0.75 and width > 64:
            width = width // 16 * 16
        rows = _log(rng, 1, 65536)
        if rows * width <= (1 << 25 if dtype == "bf16" else 1 << 24):
            break
    c = dict(op=op, rows=rows, width=width, dtype=dtype, p=rng.choice([0.05, 0.1, 0.5, round(rng.random(), 3)]))
    if op == "dropout":
        c["residual"] = rng.random() < 0.5
    else:
        c["bias"] = rng.random() < 0.7
        if rng.random() < 0.4:
            c["p"] = 0.0
    return c


# ---- inputs ----------------------------------------------------------------------------------------

def _gates(gen, case, L):
    """Log gates: for each token and head from strong to weak over the heads, with a hard reset (-inf)
    where a packed document starts; or a fixed decay for each head, from fast to slow."""
    B, H = case["B"], case["H"]
    if case["gate"] == "none":
        return None
    if case["gate"] == "head":
        return -torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)
    g = torch.randn((B, L, H), generator=gen, device="cuda") + torch.linspace(2.0, -4.0, H, device="cuda")
    g = -torch.nn.functional.softplus(g)
    for b in range(B):
        at = torch.randint(0, max(L, 1), (L // 1500,), generator=gen, device="cuda").tolist()
        g[b, at] = -math.inf
    return g


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    rnd = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    st = dict(case)
    if op.startswith("lin"):
        B, L, Hk, H, dk, dv = case["B"], case.get("L", 1), case["Hk"], case["H"], case["dk"], case["dv"]
        st["q"], st["k"], st["v"] = rnd(B, L, Hk, dk).to(dt), rnd(B, L, Hk, dk).to(dt), rnd(B, L, H, dv).to(dt)
        st["g"] = _gates(gen, case, L)
        st["S0"] = rnd(B, H, dk, dv)
        st["scale"] = dk ** -0.5
        if op == "lin_bwd":
            st["dO"], st["dS"] = rnd(B, L, H, dv).to(dt), 0.1 * rnd(B, H, dk, dv)
        return st
    N, D = case["rows"], case["width"]
    st["seed"], st["offset"] = int(torch.randint(0, 1 << 62, (), generator=gen, device="cuda")), seed % 1000
    if op == "dropout":
        st["x"] = rnd(N, D).to(dt)
        st["r"] = rnd(N, D).to(dt) if case["residual"] else None
        return st
    st["w"] = 1.0 + 0.1 * rnd(D)
    st["b"] = 0.1 * rnd(D) if case["bias"] else None
    if op == "ln_fwd":
        st["x"], st["r"] = rnd(N, D).to(dt), (1.5 * rnd(N, D) + 0.2).to(dt)
    else:
        st["s"] = (1.5 * rnd(N, D) + 0.2).to(dt)
        st["dy"], st["ds"] = rnd(N, D).to(dt), rnd(N, D).to(dt)
    return st


# ---- plain forms -----------------------------------------------------------------------------------

def _decays(g, B, L, H, N):
    """Running sums of the log gates within each chunk in 64 bits: [B, H, N, CHUNK]."""
    if g is None:
        return torch.zeros((B, H, N, CHUNK), dtype=torch.float64, device="cuda")
    g = g.double().clamp_min(RESET).expand(B, L, H).transpose(1, 2)
    return torch.cat([g, g.new_zeros(B, H, N * CHUNK - L)], 2).view(B, H, N, CHUNK).cumsum(-1)


def _chunked(x, H, N):
    """[B, L, heads, d] in float32 as [B, H, N, CHUNK, d], heads repeated, padded with zeros."""
    B, L, h, d = x.shape
    x = x.float().repeat_interleave(H // h, 2).transpose(1, 2)
    return torch.cat([x, x.new_zeros(B, H, N * CHUNK - L, d)], 2).view(B, H, N, CHUNK, d)


def _flat(x, L):
    """Back to [B, L, H, d]."""
    B, H, _, _, d = x.shape
    return x.reshape(B, H, -1, d)[:, :, :L].transpose(1, 2)


def _starts(a, u, S):
    """States before each chunk and after the last: S_0 = S, S_{n+1} = a_n S_n + u_n, by doubling along dim 2."""
    a = torch.cat([torch.ones_like(a[:, :, :1]), a], 2)[..., None, None].expand(-1, -1, -1, *u.shape[3:])
    a, u, s = a.clone(), torch.cat([S[:, :, None], u], 2), 1
    while s < u.shape[2]:
        u[:, :, s:] += a[:, :, s:] * u[:, :, :-s]
        a[:, :, s:] = a[:, :, s:] * a[:, :, :-s]
        s *= 2
    return u


def _lin_parts(st):
    B, L, H = st["q"].shape[0], st["q"].shape[1], st["H"]
    N = -(-L // CHUNK)
    q, k, v = (_chunked(st[n], H, N) for n in "qkv")
    gc = _decays(st["g"], B, L, H, N)
    last = gc[..., -1:]
    causal = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device="cuda").tril()
    between = torch.exp((gc[..., :, None] - gc[..., None, :]).masked_fill(~causal, -math.inf)).float()
    begin, end, whole = torch.exp(gc).float()[..., None], torch.exp(last - gc).float()[..., None], torch.exp(last[..., 0]).float()
    S = _starts(whole, (k * end).mT.contiguous() @ v, st["S0"])
    return L, q, k, v, between, begin, end, whole, S


def _lin_fwd(st):
    L, q, k, v, between, begin, _, _, S = _lin_parts(st)
    O = begin * (q @ S[:, :, :-1]) + ((q @ k.mT.contiguous()) * between) @ v
    return {"O": _flat(st["scale"] * O, L).to(st["v"].dtype), "S": S[:, :, -1].clone()}


def _shared(x, Hk):
    """Sum over the heads that share one."""
    B, L, H, d = x.shape
    return x.reshape(B, L, Hk, H // Hk, d).sum(3)


def _back_sum(x):
    return x.flip(-1).cumsum(-1).flip(-1)


def _lin_bwd(st):
    L, q, k, v, between, begin, end, whole, S = _lin_parts(st)
    N, Hk, dt, scale = q.shape[2], st["Hk"], st["q"].dtype, st["scale"]
    dO = scale * _chunked(st["dO"], st["H"], N)
    S = S[:, :, :-1]
    G = _starts(whole.flip(2), ((q * begin).mT.contiguous() @ dO).flip(2), st["dS"])
    dS0, G = G[:, :, -1].clone(), G[:, :, :-1].flip(2)      # G: gradient of the state after each chunk
    A, P = (q @ k.mT.contiguous()), (dO @ v.mT.contiguous()) * between
    inter_q, inter_v = begin * (dO @ S.mT.contiguous()), end * (k @ G)
    out = {"dq": _shared(_flat(inter_q + P @ k, L), Hk).to(dt),
           "dk": _shared(_flat(end * (v @ G.mT.contiguous()) + P.mT.contiguous() @ q, L), Hk).to(dt),
           "dv": _flat(inter_v + (A * between).mT.contiguous() @ dO, L).to(dt), "dS0": dS0}
    if st["g"] is not None:
        # d log g_t: pairs of tokens before and from t on, with the states at the chunk's two ends as such tokens
        M = (A * P).tril(-1).double()
        e, f = (inter_q * q).double().sum(-1), (inter_v * v).double().sum(-1)
        ends = whole.double() * (G * S).sum((-1, -2), dtype=torch.float64)
        dg = ends[..., None] + _back_sum(e + M.sum(-1) - M.sum(-2)) + f.cumsum(-1) - f
        dg = _flat(dg[..., None], L)[..., 0]
        if st["gate"] == "head":
            out["dg_log"] = dg.sum((0, 1)).float()
        else:
            out["dg_log"] = (dg * (torch.exp(st["g"]) > 0)).float()
    return out


def _keep(st):
    """What dropout multiplies by: 0 or 1 / (1 - p), p to the nearest 65536th.  Sixteen bits an element from a
    counter-based generator of ten rounds (Salmon et al., SC 2011), eight elements of a row to a counter."""
    N, D = st["rows"], st["width"]
    drop = round(st["p"] * 65536)
    if drop == 0:
        return torch.ones((N, D), device="cuda")
    if drop == 65536:
        return torch.zeros((N, D), device="cuda")
    blocks = -(-D // 8)
    low = (1 << 32) - 1
    n = torch.arange(N * blocks, device="cuda")
    c = [n & low, n >> 32, torch.full_like(n, st["offset"] & low), torch.full_like(n, st["offset"] >> 32)]
    k0, k1 = st["seed"] & low, st["seed"] >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # 64-bit products, wrapped; the shift's sign is cleared
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    u = torch.stack([w >> s & 0xFFFF for w in c for s in (0, 16)], -1).view(N, blocks * 8)[:, :D]
    return (u >= drop).float() * (65536.0 / (65536 - drop))


def _normed(s):
    s = s.float()
    d = s - s.mean(-1, keepdim=True)
    return d, 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)


def _plain(st):
    op = st["op"]
    if op == "lin_fwd":
        return _lin_fwd(st)
    if op == "lin_bwd":
        return _lin_bwd(st)
    if op == "lin_decode":
        H, q, k, v = st["H"], st["q"][:, 0].float(), st["k"][:, 0].float(), st["v"][:, 0].float()
        q, k = (x.repeat_interleave(H // st["Hk"], 1) for x in (q, k))
        S = st["S0"]
        if st["g"] is not None:
            S.mul_(torch.exp(st["g"]).reshape(-1, H, 1, 1))
        S.add_(k[..., None] * v[:, :, None])
        O = st["scale"] * (q[..., None] * S).sum(2)
        return {"O": O[:, None].to(st["v"].dtype), "S": S}
    if op == "dropout":
        y = st["x"].float() * _keep(st)
        return {"y": (y if st["r"] is None else st["r"].float() + y).to(st["x"].dtype)}
    w = st["w"]
    if op == "ln_fwd":
        s = (st["r"].float() + st["x"].float() * _keep(st)).to(st["x"].dtype)
        d, rstd = _normed(s)
        y = d * rstd * w
        return {"sum": s, "y": (y if st["b"] is None else y + st["b"]).to(s.dtype)}
    d, rstd = _normed(st["s"])
    z, dy = d * rstd, st["dy"].float()
    wd = w * dy
    ds = st["ds"].float() + rstd * (wd - wd.mean(-1, keepdim=True) - z * (wd * z).mean(-1, keepdim=True))
    out = {"dresidual": ds.to(st["s"].dtype), "dx": (ds * _keep(st)).to(st["s"].dtype),
           "dw": (dy * z).sum(0, dtype=torch.float64).float()}
    if st["b"] is not None:
        out["db"] = dy.sum(0, dtype=torch.float64).float()
    return out


def run(state):
    if not own:
        return _plain(state)
    delta, st, op = _pkg(), state, state["op"]
    if op == "lin_fwd":
        O, S = delta.fwd_lin(st["q"], st["k"], st["v"], st["g"], st["S0"], scale=st["scale"])
        return {"O": O, "S": S}
    if op == "lin_bwd":
        g = delta.bwd_lin(st["q"], st["k"], st["v"], st["g"], st["S0"], st["dO"], st["dS"], scale=st["scale"])
        return {n: t for n, t in g.items() if t is not None}
    if op == "lin_decode":
        return {"O": delta.decode_lin(st["q"], st["k"], st["v"], st["g"], st["S0"], scale=st["scale"]), "S": st["S0"]}
    rng = dict(p=st["p"], seed=st["seed"], offset=st["offset"])
    if op == "dropout":
        return {"y": delta.layer_dropout(st["x"], st["r"], **rng)}
    if op == "ln_fwd":
        s, y = delta.layer_layernorm(st["x"], st["w"], st["b"], st["r"], eps=EPS, **rng)
        return {"sum": s, "y": y}
    g = delta.layer_layernorm_bwd(st["dy"], st["s"], st["w"], st["ds"], eps=EPS, want_dbias=st["b"] is not None, **rng)
    out = {"dresidual": g["dresidual"], "dx": g["dx"], "dw": g["dweight"]}
    if st["b"] is not None:
        out["db"] = g["dbias"]
    return out


def work(case):
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("lin"):
        B, L, Hk, H, dk, dv = case["B"], case.get("L", 1), case["Hk"], case["H"], case["dk"], case["dv"]
        qk, vo, state = 2 * B * L * Hk * dk * e, 2 * B * L * H * dv * e, 2 * B * H * dk * dv * 4
        g = {"token": 4 * B * L * H, "head": 4 * H, "none": 0}[case["gate"]]
        if op == "lin_bwd":
            return {"bytes": 2 * qk + vo * 3 // 2 + 2 * g + state * 3 // 2, "flops": 10 * B * L * H * dk * dv}
        return {"bytes": qk + vo + g + state, "flops": 4 * B * L * H * dk * dv}
    n, D = case["rows"] * case["width"], case["width"]
    if op == "dropout":
        return {"bytes": (3 if case["residual"] else 2) * e * n, "flops": 2 * n}
    if op == "ln_fwd":
        return {"bytes": 4 * e * n + 4 * D * (2 if case["bias"] else 1), "flops": 10 * n}
    return {"bytes": 5 * e * n + 4 * D * (3 if case["bias"] else 2), "flops": 16 * n}


# ---- the definitions, token by token and row by row, in 64 bits -------------------------------------

def _mask64(case, st):
    """Dropout's factor from the generator's definition, on the host in 64-bit unsigned integers."""
    N, D = case["rows"], case["width"]
    share = round(case["p"] * 65536)
    if share in (0, 65536):
        return torch.full((N, D), 1.0 if share == 0 else 0.0, dtype=torch.float64, device="cuda")
    u64, half = np.uint64, np.uint64(32)
    per_row = (D + 7) // 8
    ctr = np.zeros((4, N * per_row), u64)
    at = np.arange(N * per_row, dtype=u64)
    word = lambda a: a & u64(0xFFFFFFFF)
    ctr[0], ctr[1] = word(at), at >> half
    ctr[2], ctr[3] = st["offset"] % 2**32, st["offset"] // 2**32
    key = [st["seed"] % 2**32, st["seed"] // 2**32]
    for r in range(10):
        m0, m1 = u64(0xD2511F53) * ctr[0], u64(0xCD9E8D57) * ctr[2]
        ks = [u64((key[i] + r * bump) % 2**32) for i, bump in enumerate((0x9E3779B9, 0xBB67AE85))]
        ctr = np.stack([(m1 >> half) ^ ctr[1] ^ ks[0], word(m1), (m0 >> half) ^ ctr[3] ^ ks[1], word(m0)])
    bits = ctr.T.astype("<u4").copy().view("<u2").reshape(N, per_row * 8)[:, :D].astype(np.int64)
    kept = torch.from_numpy(bits >= share).to("cuda")
    return kept.double() / (1.0 - share / 65536)


def _exact_lin(case, st):
    f64, op = torch.float64, case["op"]
    L, H, scale = st["q"].shape[1], case["H"], st["scale"]
    if op == "lin_bwd" and L > 20000:
        return None
    many = H // case["Hk"]
    q, k = (st[n].to(f64)[:, :, torch.arange(H, device="cuda") // many] for n in ("q", "k"))
    v, S = st["v"].to(f64), st["S0"].to(f64)
    a = torch.ones((1, 1, H), dtype=f64, device="cuda") if st["g"] is None else st["g"].to(f64).exp().view(-1, 1 if case["gate"] == "head" else L, H)
    a = a.expand(v.shape[0], L, H)[..., None, None]
    every, kept = 64, []
    O = torch.empty_like(v)
    for t in range(L):
        if op == "lin_bwd" and t % every == 0:
            kept.append(S)
        S = torch.addcmul(a[:, t] * S, k[:, t, :, :, None], v[:, t, :, None, :])
        if op != "lin_bwd":
            O[:, t] = scale * (q[:, t, :, None, :] @ S)[:, :, 0]
    if op != "lin_bwd":
        return {"O": O, "S": S}
    dO, flow = st["dO"].to(f64), st["dS"].to(f64)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty(v.shape[:3], dtype=f64, device="cuda")
    for first in reversed(range(0, L, every)):
        S, before = kept.pop(), []
        for t in range(first, min(first + every, L)):
            before.append(S)
            S = torch.addcmul(a[:, t] * S, k[:, t, :, :, None], v[:, t, :, None, :])
        for t in reversed(range(first, min(first + every, L))):
            w = scale * dO[:, t]
            dq[:, t] = (S @ w[..., None])[..., 0]
            flow = torch.addcmul(flow, q[:, t, :, :, None], w[:, :, None])
            dk[:, t] = (flow @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = (k[:, t, :, None, :] @ flow)[:, :, 0]
            S = before.pop()
            back = a[:, t] * flow
            dg[:, t] = (back * S).sum((-1, -2))
            flow = back
    fold = lambda x: x.unflatten(2, (case["Hk"], many)).sum(3)
    out = {"dq": fold(dq), "dk": fold(dk), "dv": dv, "dS0": flow}
    if st["g"] is not None:
        out["dg_log"] = dg.sum((0, 1)) if case["gate"] == "head" else dg
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op.startswith("lin"):
        return _exact_lin(case, st)
    m = _mask64(case, st)
    if op == "dropout":
        y = m * st["x"].to(f64)
        return {"y": y if st["r"] is None else y + st["r"].to(f64)}
    w = st["w"].to(f64)
    if op == "ln_fwd":
        s = (st["r"].to(f64) + m * st["x"].to(f64)).to(st["x"].dtype)
        t = s.to(f64)
        y = (t - t.mean(1, keepdim=True)) / torch.sqrt(t.var(1, keepdim=True, correction=0) + EPS) * w
        return {"sum": s, "y": y if st["b"] is None else y + st["b"].to(f64)}
    s, dy = st["s"].to(f64), st["dy"].to(f64)
    root = torch.sqrt(s.var(1, keepdim=True, correction=0) + EPS)
    z = (s - s.mean(1, keepdim=True)) / root
    dz = dy * w
    dr = st["ds"].to(f64) + (dz - dz.mean(1, keepdim=True) - z * (dz * z).mean(1, keepdim=True)) / root
    out = {"dresidual": dr, "dx": m * dr, "dw": (dy * z).sum(0)}
    if case["bias"]:
        out["db"] = dy.sum(0)
    return out
