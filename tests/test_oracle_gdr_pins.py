"""Pins of the gated delta rule's and the layer norm's oracle (no GPU): worked special cases, linearity, and
every gradient against central differences of the forward."""
import numpy as np
import pytest

from oracle import gdr


def inputs(seed, B=2, L=7, H=4, Hk=2, dk=5, dv=3):
    r = np.random.default_rng(seed)
    return dict(q=r.normal(size=(B, L, Hk, dk)), k=r.normal(size=(B, L, Hk, dk)), v=r.normal(size=(B, L, H, dv)),
                dt=r.normal(size=(B, L, H)), A=-r.uniform(0.2, 2.0, H), beta=r.normal(size=(B, L, H)),
                dt_bias=r.normal(size=H), h_init=r.normal(size=(B, H, dv, dk)))


def test_no_decay_unit_beta_stores_and_returns_values():
    """α = 1, β = 1 and orthonormal keys: the state is a table, and reading key i gives value i."""
    L, d = 5, 6
    k = np.eye(d)[None, :L, None, :]
    v = np.random.default_rng(0).normal(size=(1, L, 1, 4))
    y, S = gdr.gdr_fwd(k, k, v, np.zeros((1, L, 1)), np.zeros(1), np.ones((1, L, 1)), softplus=False,
                       beta_sigmoid=False, qk_l2norm=False)
    assert np.allclose(y, v)
    # writing a key again replaces its value
    k2 = np.concatenate([k, k[:, :1]], 1)
    v2 = np.concatenate([v, -v[:, :1]], 1)
    _, S2 = gdr.gdr_fwd(k2, k2, v2, np.zeros((1, L + 1, 1)), np.zeros(1), np.ones((1, L + 1, 1)), softplus=False,
                        beta_sigmoid=False, qk_l2norm=False)
    assert np.allclose(S2[0, 0] @ k[0, 0, 0], -v[0, 0, 0])


def test_beta_zero_only_decays():
    x = inputs(1)
    x["beta"] = np.full_like(x["beta"], -np.inf)
    _, S = gdr.gdr_fwd(**x)
    pre = x["dt"] + x["dt_bias"]
    g = (np.log1p(np.exp(pre)) * x["A"]).sum(1)
    assert np.allclose(S, x["h_init"] * np.exp(g)[..., None, None])


def test_linear_in_values_and_state_and_split():
    x, z = inputs(2), inputs(3)
    y1, S1 = gdr.gdr_fwd(**x)
    y2, S2 = gdr.gdr_fwd(**{**x, "v": z["v"], "h_init": z["h_init"]})
    y3, S3 = gdr.gdr_fwd(**{**x, "v": x["v"] + 2 * z["v"], "h_init": x["h_init"] + 2 * z["h_init"]})
    assert np.allclose(y3, y1 + 2 * y2) and np.allclose(S3, S1 + 2 * S2)
    cut = lambda s: {n: (t[:, s] if n in ("q", "k", "v", "dt", "beta") else t) for n, t in x.items()}  # noqa: E731
    ya, Sa = gdr.gdr_fwd(**cut(slice(0, 3)))
    yb, Sb = gdr.gdr_fwd(**{**cut(slice(3, None)), "h_init": Sa})
    assert np.allclose(np.concatenate([ya, yb], 1), y1) and np.allclose(Sb, S1)


def test_lengths_ignore_what_lies_behind():
    x = inputs(4)
    lens = np.array([3, 0])
    for n in ("q", "k", "v", "dt", "beta"):
        x[n][0, 3:] = np.nan
        x[n][1] = np.inf
    y, S = gdr.gdr_fwd(**x, seqlens=lens)
    cut = {n: (t[:1, :3] if n in ("q", "k", "v", "dt", "beta") else t[:1] if n == "h_init" else t)
           for n, t in x.items()}
    y0, S0 = gdr.gdr_fwd(**cut)
    assert np.allclose(y[:1, :3], y0) and np.allclose(S[:1], S0)
    assert not y[0, 3:].any() and not y[1].any() and np.array_equal(S[1], x["h_init"][1])


@pytest.mark.parametrize("opts", [dict(), dict(softplus=False, beta_sigmoid=False, qk_l2norm=False)])
def test_gradients_against_differences(opts):
    x = inputs(5)
    if opts:
        x["dt"] = np.abs(x["dt"]) + 0.1
        x["dt_bias"] = np.abs(x["dt_bias"])
        x["k"] /= np.linalg.norm(x["k"], axis=-1, keepdims=True)
    r = np.random.default_rng(6)
    dy, dS = r.normal(size=x["v"].shape), r.normal(size=x["h_init"].shape)
    lens = np.array([7, 5])

    def J(z):
        y, S = gdr.gdr_fwd(**z, seqlens=lens, scale=0.7, **opts)
        return (y * dy).sum() + (S * dS).sum()

    g = gdr.gdr_bwd(**x, dy=dy, dfinal=dS, seqlens=lens, scale=0.7, **opts)
    names = {"q": "dq", "k": "dk", "v": "dv", "dt": "ddt", "A": "dA", "beta": "dbeta", "dt_bias": "ddt_bias",
             "h_init": "dinitial_state"}
    for n, gn in names.items():
        d = r.normal(size=x[n].shape)
        h = 1e-5
        num = (J({**x, n: x[n] + h * d}) - J({**x, n: x[n] - h * d})) / (2 * h)
        ana = (g[gn] * d).sum()
        # central differences: h² f''' and rounding 1e-16 / h, both far below 1e-7 of the value's scale
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), (n, num, ana)


def test_norm_oracle():
    r = np.random.default_rng(7)
    x, w, b, dy = r.normal(size=(5, 9)), r.normal(size=9), r.normal(size=9), r.normal(size=(5, 9))
    y, mean, rstd = gdr.norm_fwd(x, w, b, 1e-3)
    assert np.allclose(((y - b) / w).mean(1), 0) and np.allclose(((y - b) / w).std(1) ** 2, 1 - 1e-3 * rstd ** 2)
    g = gdr.norm_bwd(dy, x, mean, rstd, w)
    J = lambda x_, w_, b_: (gdr.norm_fwd(x_, w_, b_, 1e-3)[0] * dy).sum()  # noqa: E731
    for i, n in enumerate(("dx", "dweight", "dbias")):
        args = [x, w, b]
        d = r.normal(size=args[i].shape)
        hi, lo = list(args), list(args)
        hi[i], lo[i] = args[i] + 1e-5 * d, args[i] - 1e-5 * d
        num, ana = (J(*hi) - J(*lo)) / 2e-5, (g[n] * d).sum()
        assert abs(num - ana) <= 1e-6 * max(1.0, abs(ana)), n
