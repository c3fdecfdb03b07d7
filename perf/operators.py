"""Measured cases of the gated delta rule (ss_gdr_fwd, ss_gdr_bwd, ss_gdr_step) and of the layer norm
(ss_norm_fwd, ss_norm_bwd).

`run` computes them in plain fp32 torch where `own` is false and through the library where it is true;
`exact` recomputes them in 64 bits from their definitions.

The gated delta rule, per batch entry and value head h (key head h // (nheads / nheads_k)), from S_-1 = initial state:
  Δ_t = softplus(dt_t + dt_bias_h),  α_t = exp(Δ_t A_h),  β_t = sigmoid(beta_t),  q, k rows scaled to unit length,
  e_t = v_t - α_t S_t-1 k_t,   S_t = α_t S_t-1 + β_t e_t k_tᵀ,   y_t = scale · S_t q_t      (S is d_v x d_k)
"""
import math

import torch

own = False

EPS_L2 = 1e-6   # added to a row's sum of squares before its square root
CHUNK = 64      # steps that the plain form treats as one set of dense products


# ------------------------------------------------------------------------------------------------ cases
def gdr(op, name, batch, seqlen, heads, heads_k, dk, dv, dtype="bf16", ragged=False, init=False, unit=True):
    return {"name": name, "op": op, "batch": batch, "seqlen": seqlen, "heads": heads, "heads_k": heads_k, "dk": dk,
            "dv": dv, "dtype": dtype, "ragged": ragged, "init": init, "unit": unit}


def norm(op, name, rows, cols, dtype):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # a short prompt in fp32, its length no multiple of anything
        gdr("gdr_fwd", "fwd short prompt fp32", 1, 77, 4, 2, 64, 128, dtype="fp32"),
        # the 130M-shaped layer (d_inner 1536 as 12 heads of 128), a padded batch of prompts that continue a state
        gdr("gdr_fwd", "fwd 130M-shaped ragged", 8, 2048, 12, 12, 128, 128, ragged=True, init=True),
        # the 2.8B-shaped layer (d_inner 5120 as 40 heads of 128), two value heads to a key head
        gdr("gdr_fwd", "fwd 2.8B-shaped", 4, 8192, 40, 20, 128, 128),
        # one long document: few rows, a long axis
        gdr("gdr_fwd", "fwd one long sequence", 1, 32768, 16, 8, 128, 128),
        # a small training batch of unequal lengths, heads of unequal widths
        gdr("gdr_bwd", "bwd small ragged", 2, 333, 6, 3, 64, 128, ragged=True, init=True),
        # a training step of the 130M-shaped layer
        gdr("gdr_bwd", "bwd 130M-shaped", 8, 2048, 12, 12, 128, 128),
        # one token of one sequence: latency
        gdr("gdr_step", "step one sequence fp32", 1, 1, 12, 6, 128, 128, dtype="fp32"),
        # a decode batch of the 2.8B-shaped layer
        gdr("gdr_step", "step batch of 256", 256, 1, 40, 20, 128, 128),
        # odd sizes, fp32
        norm("norm_fwd", "norm fwd odd fp32", 333, 1537, "fp32"),
        # the block's input of the 2.8B-shaped layer (4 x 8192 tokens, d_model 2560)
        norm("norm_fwd", "norm fwd d_model 2560", 32768, 2560, "bf16"),
        norm("norm_bwd", "norm bwd odd fp32", 1000, 777, "fp32"),
        norm("norm_bwd", "norm bwd d_model 2560", 32768, 2560, "bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("gdr_fwd", "gdr_fwd", "gdr_bwd", "gdr_step", "norm_fwd", "norm_bwd"))
    if op.startswith("norm"):
        cols = _spread(rng, 64, 8192)
        rows = _spread(rng, 1, min(65536, (1 << 26) // cols))
        c = norm(op, "", rows, cols, rng.choice(("bf16", "fp32")))
    else:
        heads_k = _spread(rng, 1, 20)
        heads = heads_k * rng.choice((1, 1, 2, 3))
        dk, dv = rng.choice((64, 128)), rng.choice((64, 128))
        if op == "gdr_step":
            c = gdr(op, "", _spread(rng, 1, 256 * 40 // heads if heads > 40 else 256), 1, heads, heads_k, dk, dv,
                    dtype=rng.choice(("bf16", "fp32")), unit=rng.random() < 0.7)
        else:
            dtype = "fp32" if op == "gdr_fwd" and rng.random() < 0.2 else "bf16"
            tokens = {"gdr_fwd": 1 << 19, "gdr_bwd": 1 << 17}[op] // heads     # tokens x heads of a drawn case
            seqlen = _spread(rng, 1, min(tokens, 1024 if dtype == "fp32" else 16384))
            batch = _spread(rng, 1, max(1, min(32, tokens // seqlen)))
            c = gdr(op, "", batch, seqlen, heads, heads_k, dk, dv, dtype=dtype, ragged=rng.random() < 0.4,
                    init=rng.random() < 0.5, unit=rng.random() < 0.7)
    del c["name"]
    return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "norm_fwd":
        n, c = case["rows"] * case["cols"], case["cols"]
        return {"bytes": 2 * n * e + 8 * c + 8 * case["rows"], "flops": 8 * n}
    if case["op"] == "norm_bwd":
        n, c = case["rows"] * case["cols"], case["cols"]
        return {"bytes": 3 * n * e + 12 * c + 8 * case["rows"], "flops": 14 * n}
    B, L, H, Hk, dk, dv = (case[n] for n in ("batch", "seqlen", "heads", "heads_k", "dk", "dv"))
    qk, v, gates, state = B * L * Hk * dk * e, B * L * H * dv * e, B * L * H * e, B * H * dk * dv * 4
    if case["op"] == "gdr_bwd":   # q, k, v, dy, dt, beta read, their gradients written; the states' gradients
        by = 4 * qk + 3 * v + 4 * gates + state * (3 if case["init"] else 1)
        return {"bytes": by, "flops": 16 * B * L * H * dk * dv}
    by = 2 * qk + 2 * v + 2 * gates + state * (2 if case["init"] or case["op"] == "gdr_step" else 1)
    return {"bytes": by, "flops": 6 * B * L * H * dk * dv}


# ----------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed * 7919 + 13)
    io = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev).mul_(std)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=dev)

    s = {"op": case["op"]}
    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = (normal(rows, cols) * (0.5 + rand(rows, 1)) + normal(rows, 1)).to(io)   # rows of unequal means
        s["weight"] = 1.0 + normal(cols, std=0.2)
        s["bias"] = normal(cols, std=0.2)
        if case["op"] == "norm_bwd":   # what the forward pass left, and the gradient of its output
            s["dy"] = normal(rows, cols).to(io)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + 1e-5).rsqrt().float()
        return s
    B, L, H, Hk, dk, dv = (case[n] for n in ("batch", "seqlen", "heads", "heads_k", "dk", "dv"))
    tok = (B,) if case["op"] == "gdr_step" else (B, L)
    q, k = normal(*tok, Hk, dk), normal(*tok, Hk, dk)
    if not case["unit"]:   # the user's own normalisation, before the call
        q, k = (t / t.square().sum(-1, keepdim=True).sqrt() for t in (q, k))
    s["q"], s["k"], s["v"] = q.to(io), k.to(io), normal(*tok, H, dv).to(io)
    s["dt"] = normal(*tok, H, std=0.5).to(io)
    s["beta"] = normal(*tok, H).to(io)
    s["A"] = -(1.0 + 15.0 * rand(H))
    d0 = torch.exp(math.log(1e-3) + rand(H).double() * (math.log(1e-1) - math.log(1e-3)))
    s["dt_bias"] = torch.log(torch.expm1(d0)).float()   # steps between 1e-3 and 1e-1 at dt = 0
    s["unit"], s["scale"] = case["unit"], dk ** -0.5
    if case["op"] == "gdr_step":
        s["state"] = normal(B, H, dv, dk, std=0.3)
        return s
    s["initial_state"] = normal(B, H, dv, dk, std=0.3) if case["init"] else None
    s["seqlens"] = None
    if case["ragged"]:
        n = (1 + rand(B) * L).floor().clamp(1, L)
        n[0] = L
        s["seqlens"] = n.to(torch.int32)
    if case["op"] == "gdr_bwd":
        s["dy"] = normal(B, L, H, dv).to(io)
        s["dfinal_state"] = normal(B, H, dv, dk)
    else:
        s["y"] = torch.zeros(B, L, H, dv, dtype=io, device=dev)   # rows behind a sequence's end stay zero
    return s


# ------------------------------------------------------------------------------------------ plain forms
def _unit_inverse(A):
    """(I + A)^-1 for strictly lower triangular A [..., n, n], n a power of two: [[P, 0], [-Q A21 P, Q]] of the two
    halves' inverses P and Q."""
    n = A.shape[-1]
    if n == 1:
        return torch.ones_like(A)
    h = n // 2
    P, Q = _unit_inverse(torch.stack((A[..., :h, :h], A[..., h:, h:]))).unbind(0)
    low = torch.cat((-(Q @ A[..., h:, :h] @ P), Q), -1)
    return torch.cat((torch.cat((P, torch.zeros_like(P)), -1), low), -2)


def _gdr_plain(q, k, v, dt, A, beta, dt_bias, S, seqlens, scale, unit):
    """y [B, L, H, dv] (zero behind a sequence's end) and the final state, in fp32.  Everything that does not need the
    state is computed for all chunks at once; the loop carries the state from chunk to chunk, which depends on it."""
    B, L, H, dv = v.shape
    rep = H // q.shape[2]
    q, k, v, beta = q.float(), k.float(), v.float(), torch.sigmoid(beta.float())
    g = torch.nn.functional.softplus(dt.float() + dt_bias) * A
    if unit:
        q, k = (t / (t.square().sum(-1, keepdim=True) + EPS_L2).sqrt() for t in (q, k))
    if seqlens is not None:   # a step behind the end changes nothing: its decay is 1, its β is 0
        live = torch.arange(L, device=v.device)[None, :] < seqlens[:, None]
        q, k, v = (torch.where(live[..., None, None], t, 0.0) for t in (q, k, v))
        g, beta = (torch.where(live[..., None], t, 0.0) for t in (g, beta))
    n = -(-L // CHUNK)

    def chunks(t, times=1):   # [B, L, heads, ...] -> [B, H, n, CHUNK, ...]
        t = torch.nn.functional.pad(t, (0, 0) * (t.dim() - 2) + (0, n * CHUNK - L))
        t = t.reshape(B, n, CHUNK, *t.shape[2:]).movedim(3, 1)
        return t.repeat_interleave(times, 1) if times > 1 else t

    q, k, v, g, beta = chunks(q, rep), chunks(k, rep), chunks(v), chunks(g), chunks(beta)
    G = g.double().cumsum(-1)   # 64 bits: differences of a long decay's prefix
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=v.device).tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf)).float()
    kk = k @ k.mT
    T = _unit_inverse((kk * D * beta[..., None, :]).tril(-1))
    P = q @ k.mT * D * scale
    eG, end = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    last = torch.exp(G[..., -1]).float()[..., None, None]
    keG, qeG, kend = k * eG, q * eG * scale, k * end
    S = torch.zeros(B, H, dv, k.shape[-1], device=v.device) if S is None else S
    ys = []
    for c in range(n):
        e = T[:, :, c] @ (v[:, :, c] - keG[:, :, c] @ S.mT)
        w = beta[:, :, c, :, None] * e
        ys.append(qeG[:, :, c] @ S.mT + P[:, :, c] @ w)
        S = last[:, :, c] * S + w.mT @ kend[:, :, c]
    y = torch.stack(ys, 2).movedim(1, 3).reshape(B, n * CHUNK, H, dv)[:, :L]
    if seqlens is not None:
        y = torch.where(live[..., None, None], y, 0.0)
    return y, S


def _args(s):
    return s["q"], s["k"], s["v"], s["dt"], s["A"], s["beta"], s["dt_bias"]


def _plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = (d.square().mean(1) + 1e-5).rsqrt()
        return {"y": (d * rstd[:, None] * s["weight"] + s["bias"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        wdy = dy * s["weight"]
        dx = s["rstd"][:, None] * (wdy - wdy.mean(1, keepdim=True) - xh * (wdy * xh).mean(1, keepdim=True))
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}
    if op == "gdr_step":
        S = s["state"]
        rep = S.shape[1] // s["q"].shape[1]
        q, k, v, beta = s["q"].float(), s["k"].float(), s["v"].float(), torch.sigmoid(s["beta"].float())
        if s["unit"]:
            q, k = (t / (t.square().sum(-1, keepdim=True) + EPS_L2).sqrt() for t in (q, k))
        q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
        S.mul_(torch.exp(torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"]) * s["A"])[..., None, None])
        e = v - (S @ k[..., None])[..., 0]
        S.add_((beta[..., None] * e)[..., None] * k[..., None, :])
        return {"y": ((S @ q[..., None])[..., 0] * s["scale"]).to(s["v"].dtype), "state": S}
    if op == "gdr_fwd":
        y, S = _gdr_plain(*_args(s), s["initial_state"], s["seqlens"], s["scale"], s["unit"])
        return {"y": s["y"].copy_(y), "final_state": S}
    leaves = [t.detach().float().requires_grad_() for t in _args(s)]
    if s["initial_state"] is not None:
        leaves.append(s["initial_state"].detach().requires_grad_())
    y, S = _gdr_plain(*leaves[:7], leaves[7] if len(leaves) > 7 else None, s["seqlens"], s["scale"], s["unit"])
    got = torch.autograd.grad((y, S), leaves, (s["dy"].float(), s["dfinal_state"]))
    io = [t.dtype for t in _args(s)]
    names = ("dq", "dk", "dv", "ddt", "dA", "dbeta", "ddt_bias", "dinitial_state")
    return {n: t.to(io[i]) if i < 7 else t for i, (n, t) in enumerate(zip(names, got))}


def run(state):
    if not own:
        return _plain(state)
    import selective_state_space_37_b200 as ss
    s, op = state, state["op"]
    if op == "norm_fwd":
        y, mean, rstd = ss.ss_norm_fwd(s["x"], s["weight"], s["bias"], eps=1e-5)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        return ss.ss_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
    q, k, v, dt, A, beta, dt_bias = _args(s)
    if op == "gdr_step":
        y = ss.ss_gdr_step(s["state"], q, k, v, dt, A, beta, dt_bias=dt_bias, scale=s["scale"], qk_l2norm=s["unit"])
        return {"y": y, "state": s["state"]}
    if op == "gdr_fwd":
        y, S = ss.ss_gdr_fwd(q, k, v, dt, A, beta, dt_bias=dt_bias, initial_state=s["initial_state"],
                             seqlens=s["seqlens"], scale=s["scale"], qk_l2norm=s["unit"], y=s["y"])
        return {"y": y, "final_state": S}
    return ss.ss_gdr_bwd(q, k, v, dt, A, beta, s["dy"], dt_bias=dt_bias, initial_state=s["initial_state"],
                         dfinal_state=s["dfinal_state"], seqlens=s["seqlens"], scale=s["scale"], qk_l2norm=s["unit"])


# -------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The recurrence step by step and its adjoint step by step, in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("norm"):
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        if op == "norm_fwd":
            mean = x.sum(1) / x.shape[1]
            rstd = 1.0 / (((x - mean[:, None]) ** 2).sum(1) / x.shape[1] + 1e-5).sqrt()
            return {"y": (x - mean[:, None]) * rstd[:, None] * w + b, "mean": mean, "rstd": rstd}
        dy, mean, rstd = s["dy"].double(), s["mean"].double()[:, None], s["rstd"].double()[:, None]
        xh, c = (x - mean) * rstd, x.shape[1]
        dxh = dy * w
        dx = rstd / c * (c * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True))
        return {"dx": dx, "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}

    step = op == "gdr_step"
    q, k, v, dt, A, braw, dt_bias = (t.double() for t in _args(s))
    if step:
        q, k, v, dt, braw = (t[:, None] for t in (q, k, v, dt, braw))
    B, L, H, dv = v.shape
    rep, dk = H // q.shape[2], q.shape[3]
    pre = dt + dt_bias
    delta = torch.where(pre > 20, pre, torch.log1p(torch.exp(pre.clamp(max=20.0))))
    beta = 1.0 / (1.0 + torch.exp(-braw))
    lq, lk = (((t * t).sum(-1, keepdim=True) + EPS_L2).sqrt() if s["unit"] else torch.ones_like(t[..., :1]) for t in (q, k))
    qh, kh = q / lq, k / lk
    alpha = torch.exp(delta * A)
    lens = s.get("seqlens")
    live = torch.ones(B, L, dtype=torch.bool, device=v.device)
    if lens is not None:
        live = torch.arange(L, device=v.device)[None] < lens[:, None]
    alpha = torch.where(live[..., None], alpha, 1.0)
    beta_l = torch.where(live[..., None], beta, 0.0)
    qr, kr = qh.repeat_interleave(rep, 2) * s["scale"], kh.repeat_interleave(rep, 2)
    first = s["state"] if step else s["initial_state"]
    S = torch.zeros(B, H, dv, dk, dtype=torch.float64, device=v.device) if first is None else first.double()

    def forward(S, t):
        Sd = S * alpha[:, t, :, None, None]
        e = v[:, t] - (Sd @ kr[:, t, :, :, None])[..., 0]
        return Sd, e, Sd + (beta_l[:, t, :, None] * e)[..., None] * kr[:, t, :, None, :]

    if op != "gdr_bwd":
        y = torch.zeros_like(v)
        for t in range(L):
            S = forward(S, t)[2]
            y[:, t] = torch.where(live[:, t, None, None], (S @ qr[:, t, :, :, None])[..., 0], 0.0)
        return {"y": y[:, 0], "state": S} if step else {"y": y, "final_state": S}

    seg, starts = 64, []
    for t in range(L):
        if t % seg == 0:
            starts.append(S)
        S = forward(S, t)[2]
    dS = s["dfinal_state"].double()
    dy = torch.where(live[..., None, None], s["dy"].double(), 0.0)
    dq, dk_, dv_ = torch.zeros_like(qr), torch.zeros_like(kr), torch.zeros_like(v)
    db, dla = torch.zeros_like(beta), torch.zeros_like(beta)
    for c in reversed(range(len(starts))):
        S, kept = starts[c], []
        for t in range(c * seg, min(L, (c + 1) * seg)):
            Sd, e, S1 = forward(S, t)
            kept.append((S, Sd, e, S1))
            S = S1
        for t in reversed(range(c * seg, min(L, (c + 1) * seg))):
            S0, Sd, e, S1 = kept[t - c * seg]
            kt, qt, b1 = kr[:, t], qr[:, t], beta_l[:, t, :, None]
            dS = dS + dy[:, t, :, :, None] * qt[..., None, :]
            dq[:, t] = (dy[:, t, :, None, :] @ S1)[..., 0, :] * s["scale"]
            dSk = (dS @ kt[..., None])[..., 0]
            de = b1 * dSk
            db[:, t] = (dSk * e).sum(-1)
            dSd = dS - de[..., None] * kt[..., None, :]
            dk_[:, t] = b1 * (e[..., None, :] @ dS)[..., 0, :] - (de[..., None, :] @ Sd)[..., 0, :]
            dv_[:, t] = de
            dla[:, t] = (dSd * Sd).sum((-1, -2))
            dS = alpha[:, t, :, None, None] * dSd
    m = live[..., None]
    db, dla = torch.where(m, db, 0.0), torch.where(m, dla, 0.0)
    dk_, dv_ = torch.where(m[..., None], dk_, 0.0), torch.where(m[..., None], dv_, 0.0)
    share = lambda t: t.reshape(B, L, H // rep, rep, dk).sum(3)  # noqa: E731
    dq, dk_ = share(dq), share(dk_)
    if s["unit"]:
        dq = (dq - qh * (qh * dq).sum(-1, keepdim=True)) / lq
        dk_ = (dk_ - kh * (kh * dk_).sum(-1, keepdim=True)) / lk
    ddt = dla * A * (1.0 / (1.0 + torch.exp(-pre)))
    out = {"dq": dq, "dk": dk_, "dv": dv_, "ddt": ddt, "dA": (dla * delta).sum((0, 1)), "dbeta": db * beta * (1 - beta),
           "ddt_bias": ddt.sum((0, 1))}
    if first is not None:
        out["dinitial_state"] = dS
    return out
