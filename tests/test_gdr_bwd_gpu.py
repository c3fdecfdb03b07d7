"""GPU tests of the gated delta rule's backward pass against the 64-bit oracle (token by token), and of the passes
together."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, f64, gdr_inputs, max_err, rms_err
from oracle import gdr
from ss_inputs import to_f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DEV = "cuda:0"
SEQ_GRADS = ("dq", "dk", "dv", "ddt", "dbeta")


def upstream(x, seed, final=True):
    g = torch.Generator(device="cpu").manual_seed(seed)
    B, L, H, dv = x["v"].shape
    dk = x["q"].shape[-1]
    dy = torch.randn(B, L, H, dv, generator=g).to(BF).to(DEV)
    dS = torch.randn(B, H, dv, dk, generator=g).to(DEV) if final else None
    return dy, dS


def oracle_bwd(x, dy, dS, seqlens=None, scale=None, **opt):
    z = f64(x)
    return gdr.gdr_bwd(z["q"], z["k"], z["v"], z["dt"], z["A"], z["beta"], to_f64(dy), dt_bias=z.get("dt_bias"),
                       h_init=z.get("state"), dfinal=to_f64(dS), seqlens=seqlens, scale=scale, **opt)


def gate_bound(want, x, dy, seqlens=None, scale=1.0, **opt):
    """Bound on dA's and ddt_bias' error.  A token's gradient of log α is <S, dS> of its chunk's end and up to 64
    terms dO·Y and dV·V; each is computed from products whose fp32 operands enter as two bf16 terms: off by under
    2^-15 of the sum of absolute values (three such products in a row, 2^-17 each, and fp32 sums)."""
    z = f64(x)
    y, _ = gdr.gdr_fwd(z["q"], z["k"], z["v"], z["dt"], z["A"], z["beta"], dt_bias=z.get("dt_bias"),
                       h_init=z.get("state"), seqlens=seqlens, scale=scale, **opt)
    B, L, H, _ = y.shape
    m = np.abs(np.nan_to_num(to_f64(dy)) * y).sum(-1) + np.abs(want["dv"] * np.nan_to_num(z["v"])).sum(-1)
    n = -(-L // 64)
    pad = lambda t: np.pad(t, ((0, 0), (0, n * 64 - L), (0, 0))).reshape(B, n, 64, H)  # noqa: E731
    per = pad(m).sum(2) + pad(want["dlog_alpha_size"]).max(2)
    err = 2.0 ** -15 * np.repeat(per, 64, 1)[:, :L]
    sig = np.abs(want["ddt"]) / np.maximum(np.abs(want["dlog_alpha"] * z["A"]), 1e-300)   # softplus' slope
    return (err * np.abs(want["delta"])).sum((0, 1)), (err * np.abs(z["A"]) * np.minimum(sig, 1.0)).sum((0, 1))


def check(x, seed=0, seqlens=None, scale=None, final=True, **kw):
    opt = {n: kw.pop(n) for n in ("softplus", "beta_sigmoid", "qk_l2norm") if n in kw}
    dy, dS = kw.pop("up", None) or upstream(x, seed, final)
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device=DEV)
    g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x.get("dt_bias"), initial_state=x.get("state"), dfinal_state=dS,
                      seqlens=lens, scale=scale, sync_check=True, **opt, **kw)
    want = oracle_bwd(x, dy, dS, None if seqlens is None else np.array(seqlens), scale, **opt)
    for n in SEQ_GRADS:
        # bf16 outputs (half a step: 1.7e-3 on average) of products whose operands are rounded once to bf16 (two of
        # them for dq and dk, E for dbeta): 2.9e-3 on average; a single value at four half-steps of the largest
        assert rms_err(g[n], want[n]) <= 5e-3, n
        assert max_err(g[n], want[n]) <= 4 * 2.0 ** -8, n
    bA, bb = gate_bound(want, x, dy, None if seqlens is None else np.array(seqlens), scale, **opt)
    assert np.all(np.abs(to_f64(g["dA"]) - want["dA"]) <= bA + 1e-30)
    if "dt_bias" in x:
        assert np.all(np.abs(to_f64(g["ddt_bias"]) - want["ddt_bias"]) <= bb + 1e-6 * np.abs(want["ddt_bias"]) + 1e-30)
    if "state" in x:
        assert rms_err(g["dinitial_state"], want["dinitial_state"]) <= 1e-5
    return g, want


@pytest.mark.parametrize("L", [1, 2, 15, 63, 64, 65, 128, 129, 200])
def test_lengths(L):
    check(gdr_inputs(2, L, 4, 2, 128, 128, seed=L, init=L % 2 == 0), L)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (2, 2), (6, 2)])
def test_heads_and_widths(H, Hk, dk, dv):
    check(gdr_inputs(2, 150, H, Hk, dk, dv, seed=dk + H, init=H == 2), H)


def test_without_initial_and_final_gradients():
    x = gdr_inputs(2, 100, 2, 2, 128, 128, seed=9)
    g, _ = check(x, 1, final=False)
    assert "dinitial_state" not in g
    x.pop("dt_bias")
    g, _ = check(x, 1)
    assert "ddt_bias" not in g


def test_options():
    x = gdr_inputs(2, 100, 2, 1, 64, 128, seed=11, unit=False, init=True)
    check(x, 2, qk_l2norm=False, scale=0.37)
    x["dt"] = (x["dt"].float().abs() * 0.1).to(BF)
    x["beta"] = torch.rand_like(x["beta"].float()).to(BF)
    x.pop("dt_bias")
    check(x, 2, qk_l2norm=False, softplus=False, beta_sigmoid=False)
    x["beta"][:, ::7] = 0.0   # β's gradient where β is zero
    check(x, 2, qk_l2norm=False, softplus=False, beta_sigmoid=False)


@pytest.mark.parametrize("L", [20, 200])
def test_padded_batch_ignores_what_lies_behind(L):
    lens = [L, 0, 1, L // 2, L - 1, 5]
    x = gdr_inputs(6, L, 4, 2, 128, 128, seed=3, init=True)
    dy, dS = upstream(x, 5)
    for b, n in enumerate(lens):
        for name, bad in (("q", np.nan), ("k", np.inf), ("v", np.nan), ("dt", np.nan), ("beta", -np.inf)):
            x[name][b, n:] = bad
        dy[b, n:] = np.nan
    g, want = check(x, seqlens=lens, up=(dy, dS))
    for b, n in enumerate(lens):
        for name in SEQ_GRADS:
            assert not g[name][b, n:].any(), name
    assert torch.equal(g["dinitial_state"][1], dS[1])


@pytest.mark.parametrize("A", [0.0, -1e-4, -1000.0])
def test_extreme_decays(A):
    x = gdr_inputs(2, 140, 2, 2, 128, 128, seed=21, init=True)
    x["A"].fill_(A)
    dy, dS = upstream(x, 7)
    g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS, sync_check=True)
    want = oracle_bwd(x, dy, dS, scale=128 ** -0.5)
    for n in ("dq", "dk", "dv", "dbeta"):
        assert rms_err(g[n], want[n]) <= 5e-3, n
    assert rms_err(g["dinitial_state"], want["dinitial_state"]) <= 1e-5
    bA, _ = gate_bound(want, x, dy, scale=128 ** -0.5)
    assert np.all(np.abs(to_f64(g["dA"]) - want["dA"]) <= bA + 1e-30)


@pytest.mark.parametrize("dt", [400.0, 3.0e38])
def test_steps_that_empty_the_state(dt):
    """Gates so large that Δ A, and its sums, leave fp32's range: no gradient passes them, and they have none."""
    x = gdr_inputs(2, 140, 3, 3, 128, 128, seed=23, init=True)
    x["dt"][0, ::9, 0] = dt
    x["dt"][1, 5, :] = dt
    x["dt"][:, -3:, 2] = dt
    check(x, 3)


def test_refusals():
    x = gdr_inputs(2, 20, 2, 2, 64, 64, seed=2)
    dy, _ = upstream(x, 1)
    with pytest.raises(TypeError, match="float16"):
        ss.ss_gdr_bwd(x["q"].half(), *call_args(x)[1:], dy)
    with pytest.raises(TypeError, match="dy"):
        ss.ss_gdr_bwd(*call_args(x), dy.float())
    with pytest.raises(ValueError, match="dq"):
        ss.ss_gdr_bwd(*call_args(x), dy, grads={"dq": x["q"][:1].contiguous()})
    with pytest.raises(ValueError, match="ddt_bias"):
        ss.ss_gdr_bwd(*call_args(x), dy, grads={"ddt_bias": x["A"]})
    with pytest.raises(ValueError, match="contiguous"):
        ss.ss_gdr_bwd(x["q"].transpose(0, 1).contiguous().transpose(0, 1), *call_args(x)[1:], dy)
    with pytest.raises(ss.SelscanError):
        ss.ss_gdr_bwd(*call_args(x), dy, workspace=torch.empty(512, dtype=torch.uint8, device=DEV))


def test_against_differences():
    """The gradients of the library's own forward: central differences of J along random directions of the fp32
    inputs (A, dt_bias, the states), whose outputs are fp32 where they matter (J of the final state alone)."""
    x = gdr_inputs(2, 70, 2, 1, 64, 64, seed=14, init=True)
    dS = torch.randn(x["state"].shape, device=DEV)
    dy = torch.zeros_like(x["v"])
    g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS)

    def J(**change):
        z = {**x, **change}
        _, S = ss.ss_gdr_fwd(*call_args(z), dt_bias=z["dt_bias"], initial_state=z["state"])
        return float((S.double() * dS.double()).sum())

    size = float((dS.abs().double() * ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"],
                                                    initial_state=x["state"])[1].abs().double()).sum())
    for name, grad in (("A", "dA"), ("dt_bias", "ddt_bias"), ("state", "dinitial_state")):
        d = torch.randn_like(x[name])
        h = 1e-2
        num = (J(**{name: x[name] + h * d}) - J(**{name: x[name] - h * d})) / (2 * h)
        ana = float((g[grad].double() * d.double()).sum())
        # J's rounding over h, and the differences' own h² term (a third derivative of a few J)
        assert abs(num - ana) <= 2.0 ** -16 * size / h / 10 + 20 * h * h * size + 1e-3 * abs(ana), (name, num, ana)


def test_same_call_same_bits_and_graphs():
    xs = [gdr_inputs(2, 200, 4, 2, 128, 128, seed=s, init=True) for s in (1, 2)]
    ups = [upstream(x, s) for s, x in enumerate(xs)]
    call = lambda x, u: ss.ss_gdr_bwd(*call_args(x), u[0], dt_bias=x["dt_bias"], initial_state=x["state"],  # noqa: E731
                                      dfinal_state=u[1])
    want = [call(x, u) for x, u in zip(xs, ups)]
    again = [call(x, u) for x, u in zip(xs, ups)]
    for a, b in zip(want, again):
        assert all(torch.equal(a[n], b[n]) for n in a)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x, u in zip(xs, ups):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x, u))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(2):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_zero_length_and_empty():
    x = gdr_inputs(2, 0, 3, 3, 64, 64, init=True)
    dy, dS = upstream(x, 1)
    g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS, sync_check=True)
    assert not g["dA"].any() and not g["ddt_bias"].any() and torch.equal(g["dinitial_state"], dS)
    x = gdr_inputs(0, 5, 3, 3, 64, 64)
    g = ss.ss_gdr_bwd(*call_args(x), x["v"], dt_bias=x["dt_bias"], sync_check=True)
    assert not g["dA"].any()


def test_bounded_wait_reports_timeout_and_context_survives():
    x = gdr_inputs(2, 300, 2, 2, 128, 128, seed=5)
    dy, dS = upstream(x, 1)
    need = ss.lib().ss_gdr_bwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(2, 300, 2, 2, 128, 128)), ss.SS_BF16)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], dfinal_state=dS, workspace=ws, timeout_iters=2000,
                  extra_flags=ss.SS_TEST_DROP_CARRY)
    assert ss.ss_check(ws) == ss.SS_ERR_TIMEOUT
    check(x, 1, workspace=ws)


def test_layer_of_the_operators_together():
    """Norm -> projections -> gated delta rule -> norm over each head, forward and backward, against the same layer
    in 64 bits by automatic differentiation; and the step continues what the sequence left."""
    B, L, H, Hk, d, m = 2, 130, 4, 2, 64, 96
    g = torch.Generator(device="cpu").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    x = rnd(B, L, m).to(BF)
    w1, b1, w2, b2 = 1 + 0.1 * rnd(m), 0.1 * rnd(m), 1 + 0.1 * rnd(d), 0.1 * rnd(d)
    W = (rnd(2 * Hk * d + H * d + 2 * H, m) / m ** 0.5).to(BF)
    A, bias = -(1 + rnd(H).abs()), rnd(H) - 3
    sizes = (Hk * d, Hk * d, H * d, H, H)

    def parts(p):
        q, k, v, dt, be = p.split(sizes, -1)
        return [t.contiguous() for t in (q.unflatten(-1, (Hk, d)), k.unflatten(-1, (Hk, d)), v.unflatten(-1, (H, d)), dt, be)]

    n1, mu1, r1 = ss.ss_norm_fwd(x, w1, b1)
    q, k, v, dt, be = parts(n1 @ W.T)
    y, S = ss.ss_gdr_fwd(q, k, v, dt, A, be, dt_bias=bias)
    out, mu2, r2 = ss.ss_norm_fwd(y, w2, b2)
    dout = rnd(B, L, H, d).to(BF)
    gn2 = ss.ss_norm_bwd(dout, y, mu2, r2, w2)
    gd = ss.ss_gdr_bwd(q, k, v, dt, A, be, gn2["dx"], dt_bias=bias)
    dp = torch.cat([gd[n].flatten(2) if n in ("dq", "dk", "dv") else gd[n] for n in ("dq", "dk", "dv", "ddt", "dbeta")], -1)
    gn1 = ss.ss_norm_bwd((dp @ W).contiguous(), x, mu1, r1, w1)

    D = torch.float64
    lx, lw1, lb1, lw2, lb2, lA, lbias = (t.to(D).detach().requires_grad_() for t in (x, w1, b1, w2, b2, A, bias))
    rt = lambda t: t + (t.to(BF).to(D) - t).detach()   # rounded where the layer stores bf16  # noqa: E731
    ln = lambda t, w, b: (t - t.mean(-1, keepdim=True)) / (t.var(-1, unbiased=False, keepdim=True) + 1e-5).sqrt() * w + b  # noqa: E731
    rq, rk, rv, rdt, rbe = parts(rt(rt(ln(lx, lw1, lb1)) @ W.to(D).T))
    unit = lambda t: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    uq, uk = (unit(t).repeat_interleave(H // Hk, 2) for t in (rq, rk))
    al, bt = torch.exp(torch.nn.functional.softplus(rdt + lbias) * lA), torch.sigmoid(rbe)
    St, ys = torch.zeros(B, H, d, d, dtype=D, device=DEV), []
    for t in range(L):
        St = St * al[:, t, :, None, None]
        e = rv[:, t] - (St @ uk[:, t, :, :, None])[..., 0]
        St = St + (bt[:, t, :, None] * e)[..., None] * uk[:, t, :, None, :]
        ys.append((St @ uq[:, t, :, :, None])[..., 0] * d ** -0.5)
    ry = rt(torch.stack(ys, 1))
    ref = ln(ry, lw2, lb2)
    rg = torch.autograd.grad(ref, (lx, lw1, lb1, lw2, lb2, lA, lbias), dout.to(D))
    num = lambda t: t.detach().cpu().numpy()  # noqa: E731
    assert rms_err(S, num(St)) <= 2 * 2.0 ** -8          # (the projections' own rounding may fall either way)
    assert rms_err(out, num(ref)) <= 3 * 2.0 ** -8
    # a chain of six roundings to bf16 (each 1.7e-3 on average) between dout and the last gradients
    got = (gn1["dx"], gn1["dweight"], gn1["dbias"], gn2["dweight"], gn2["dbias"], gd["dA"], gd["ddt_bias"])
    for name, a, r in zip(("dx", "dw1", "db1", "dw2", "db2", "dA", "dbias"), got, rg):
        assert rms_err(a, num(r)) <= 6 * 2.0 ** -8, name
    st = S.clone()
    y1 = ss.ss_gdr_step(st, *(t[:, -1].contiguous() for t in (q, k, v, dt)), A, be[:, -1].contiguous(), dt_bias=bias)
    y2, S2 = ss.ss_gdr_fwd(*(t[:, -1:].contiguous() for t in (q, k, v, dt)), A, be[:, -1:].contiguous(), dt_bias=bias,
                           initial_state=S)
    assert torch.equal(st, S2) and torch.equal(y1, y2[:, 0])
