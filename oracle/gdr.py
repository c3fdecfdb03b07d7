"""Oracle of the gated delta rule and of the layer norm -- TEST INFRASTRUCTURE ONLY.

Float64 numpy, straight from the definitions, token by token (no chunks, no inverse, no tensor cores):

  Δ_t = softplus(dt_t + bias),  α_t = exp(Δ_t A),  β_t = σ(beta_t),  k̂ = k / sqrt(|k|² + 1e-6)  (q likewise)
  e_t = v_t - α_t S_{t-1} k̂_t,  S_t = α_t S_{t-1} + β_t e_t k̂_tᵀ,  y_t = scale S_t q̂_t

and its adjoint, the same steps differentiated one by one in reverse."""
import numpy as np

L2_EPS = 1e-6


def _softplus(x):
    return np.where(x > 20.0, x, np.log1p(np.exp(np.minimum(x, 20.0))))


def _sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x))


class _Prep:
    """The per-token quantities of a call, masked behind each sequence's end."""

    def __init__(self, q, k, v, dt, A, beta, dt_bias, seqlens, scale, softplus, beta_sigmoid, qk_l2norm):
        B, L, H = dt.shape
        self.rep = H // q.shape[2]
        self.live = np.ones((B, L), bool) if seqlens is None else np.arange(L)[None] < np.clip(seqlens, 0, L)[:, None]
        m = self.live[..., None]
        # what lies behind a sequence's end is not used, whatever it holds
        q, k, v = (np.where(m[..., None], t, 0.0) for t in (q, k, v))
        dt, beta = np.where(m, dt, 0.0), np.where(m, beta, 0.0)
        self.pre = dt + (0.0 if dt_bias is None else dt_bias)
        self.delta = _softplus(self.pre) if softplus else self.pre
        self.alpha = np.where(m, np.exp(self.delta * A), 1.0)
        self.beta = np.where(m, _sigmoid(beta) if beta_sigmoid else beta, 0.0)
        one = np.ones(q.shape[:-1] + (1,))
        self.lq = np.sqrt((q * q).sum(-1, keepdims=True) + L2_EPS) if qk_l2norm else one
        self.lk = np.sqrt((k * k).sum(-1, keepdims=True) + L2_EPS) if qk_l2norm else one
        self.qh, self.kh = q / self.lq, k / self.lk
        self.qr, self.kr = np.repeat(self.qh, self.rep, 2) * scale, np.repeat(self.kh, self.rep, 2)
        self.v = v

    def step(self, S, t):
        Sd = S * self.alpha[:, t, :, None, None]
        e = self.v[:, t] - np.einsum("bhvk,bhk->bhv", Sd, self.kr[:, t])
        return Sd, e, Sd + (self.beta[:, t, :, None] * e)[..., None] * self.kr[:, t, :, None, :]


def gdr_fwd(q, k, v, dt, A, beta, dt_bias=None, h_init=None, seqlens=None, scale=1.0, softplus=True,
            beta_sigmoid=True, qk_l2norm=True):
    """y [B, L, H, d_v] (zero behind a sequence's end) and the final state [B, H, d_v, d_k]."""
    p = _Prep(q, k, v, dt, A, beta, dt_bias, seqlens, scale, softplus, beta_sigmoid, qk_l2norm)
    B, L, H, dv = v.shape
    S = np.zeros((B, H, dv, q.shape[3])) if h_init is None else np.array(h_init, dtype=np.float64)
    y = np.zeros(v.shape)
    for t in range(L):
        S = p.step(S, t)[2]
        y[:, t] = np.where(p.live[:, t, None, None], np.einsum("bhvk,bhk->bhv", S, p.qr[:, t]), 0.0)
    return y, S


def gdr_bwd(q, k, v, dt, A, beta, dy, dt_bias=None, h_init=None, dfinal=None, seqlens=None, scale=1.0, softplus=True,
            beta_sigmoid=True, qk_l2norm=True):
    """Gradients of sum(dy y) + sum(dfinal final_state) as a dict, and of each token Δ, the gradient of log α, and the
    sum of absolute values whose signed sum that gradient is (what a rounding of its terms is relative to)."""
    p = _Prep(q, k, v, dt, A, beta, dt_bias, seqlens, scale, softplus, beta_sigmoid, qk_l2norm)
    B, L, H, dv = v.shape
    dk = q.shape[3]
    S = np.zeros((B, H, dv, dk)) if h_init is None else np.array(h_init, dtype=np.float64)
    kept = []
    for t in range(L):
        Sd, e, S = p.step(S, t)
        kept.append((Sd, e, S))
    dy = np.where(p.live[..., None, None], dy, 0.0)
    dS = np.zeros_like(S) if dfinal is None else np.array(dfinal, dtype=np.float64)
    dq, dk_, dv_ = np.zeros(p.qr.shape), np.zeros(p.kr.shape), np.zeros(v.shape)
    db, dla, size = np.zeros(dt.shape), np.zeros(dt.shape), np.zeros(dt.shape)
    for t in reversed(range(L)):
        Sd, e, S1 = kept[t]
        kt, qt, b1 = p.kr[:, t], p.qr[:, t], p.beta[:, t, :, None]
        dS = dS + dy[:, t, :, :, None] * qt[..., None, :]
        dq[:, t] = scale * np.einsum("bhv,bhvk->bhk", dy[:, t], S1)
        dSk = np.einsum("bhvk,bhk->bhv", dS, kt)
        de = b1 * dSk
        db[:, t] = (dSk * e).sum(-1)
        dSd = dS - de[..., None] * kt[..., None, :]
        dk_[:, t] = b1 * np.einsum("bhv,bhvk->bhk", e, dS) - np.einsum("bhv,bhvk->bhk", de, Sd)
        dv_[:, t] = de
        dla[:, t] = (dSd * Sd).sum((-1, -2))
        size[:, t] = np.abs(dSd * Sd).sum((-1, -2))
        dS = p.alpha[:, t, :, None, None] * dSd
    m = p.live[..., None]
    db, dla = np.where(m, db, 0.0), np.where(m, dla, 0.0)
    dk_, dv_ = np.where(m[..., None], dk_, 0.0), np.where(m[..., None], dv_, 0.0)
    dq, dk_ = (t.reshape(B, L, H // p.rep, p.rep, dk).sum(3) for t in (dq, dk_))
    if qk_l2norm:
        dq = (dq - p.qh * (p.qh * dq).sum(-1, keepdims=True)) / p.lq
        dk_ = (dk_ - p.kh * (p.kh * dk_).sum(-1, keepdims=True)) / p.lk
    ddt = dla * A * (_sigmoid(p.pre) if softplus else 1.0)
    return {"dq": dq, "dk": dk_, "dv": dv_, "ddt": ddt, "dA": (dla * p.delta).sum((0, 1)),
            "dbeta": db * (p.beta * (1.0 - p.beta) if beta_sigmoid else 1.0), "ddt_bias": ddt.sum((0, 1)),
            "dinitial_state": dS, "delta": p.delta, "dlog_alpha": dla, "dlog_alpha_size": size}


def norm_fwd(x, weight=None, bias=None, eps=1e-5):
    mean = x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    y = (x - mean) * rstd
    y = y if weight is None else y * weight
    return (y if bias is None else y + bias), mean[..., 0], rstd[..., 0]


def norm_bwd(dy, x, mean, rstd, weight=None):
    xh = (x - mean[..., None]) * rstd[..., None]
    g = dy if weight is None else dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return {"dx": dx, "dweight": (dy * xh).sum(axes), "dbias": dy.sum(axes)}
