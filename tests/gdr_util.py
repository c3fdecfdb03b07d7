"""Inputs and comparisons for the gated delta rule's tests."""
import numpy as np
import torch

from ss_inputs import to_f64

SEQ = ("q", "k", "v", "dt", "beta")


def gdr_inputs(B, L, H, Hk, dk, dv, dtype=torch.bfloat16, seed=0, device="cuda:0", init=False, unit=True, step=False):
    """Inputs of one call: q, k, v, beta ~ N(0, 1), dt ~ N(0, 0.5²), A = -U[1, 16], steps of 1e-3 .. 1e-1 at
    dt = 0.  unit=False normalises q and k here instead of in the call."""
    g = torch.Generator(device="cpu").manual_seed(seed * 131 + 7)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    tok = (B,) if step else (B, L)
    x = {"q": n(*tok, Hk, dk), "k": n(*tok, Hk, dk), "v": n(*tok, H, dv), "dt": 0.5 * n(*tok, H), "beta": n(*tok, H)}
    if not unit:
        for name in ("q", "k"):
            x[name] = x[name] / x[name].square().sum(-1, keepdim=True).sqrt()
    x = {name: t.to(dtype) for name, t in x.items()}
    x["A"] = -(1.0 + 15.0 * torch.rand(H, generator=g))
    x["dt_bias"] = torch.log(torch.expm1(torch.exp(-6.9 + 4.6 * torch.rand(H, generator=g))))
    if init or step:
        x["state"] = 0.3 * n(B, H, dv, dk)
    return {name: t.to(device) for name, t in x.items()}


def call_args(x):
    return (x["q"], x["k"], x["v"], x["dt"], x["A"], x["beta"])


def f64(x):
    return {name: to_f64(t) for name, t in x.items()}


def max_err(got, ref):
    """max |got - ref| / max |ref| (absolute where the reference is zero)."""
    got, ref = np.asarray(to_f64(got)), np.asarray(ref)
    if not ref.size:
        return 0.0
    err, den = np.max(np.abs(got - ref)), np.max(np.abs(ref))
    return float(err / den) if den > 0 else float(err)


def rms_err(got, ref):
    got, ref = np.asarray(to_f64(got)), np.asarray(ref)
    den = np.linalg.norm(ref)
    return float(np.linalg.norm(got - ref) / den) if den > 0 else float(np.linalg.norm(got - ref))


U32 = 2.0 ** -24


def state_tol(L, dtype):
    """Bound on the state's largest error over its largest entry.

    Token by token in fp32 a step rounds a dot product of d_k <= 128 terms (16 in a chain, 3 shuffles), the
    correction and the update: under 40 half-steps of 2^-24, and I - β k̂ k̂ᵀ does not enlarge an earlier error.
    In chunks (bf16 inputs) the three products in series of 64 steps read their fp32 operands as two bf16 terms:
    each is off by at most 2^-16 of its operands' norms, and a row's norm is at most 8 times what its largest
    entry shows here (128 entries of one size: 11.3 at most, of normal values far less)."""
    if dtype == torch.float32:
        return 40 * U32 * max(L, 1)
    return max(40 * U32 * max(L, 1), (L // 64 + 1) * 3 * 8 * 2.0 ** -16)


def y_tol(L, dtype):
    """The state's bound, y's own dot product being of the same kind, plus half a step of y's type.  bf16 chunks
    also round the chunk's attention weights and values to bf16 in the part of y that they give: 2 · 2^-9 of it."""
    if dtype == torch.float32:
        return 2 * state_tol(L, dtype)
    return 2 * state_tol(L, dtype) + 2.0 ** -8 + 2 * 2.0 ** -8
