"""GPU tests of the gated delta rule's gradients against differences of its own forward pass, along each gradient's own
direction, with a bound well under the derivative itself."""
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, gdr_inputs

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H_STEP = 2.0 ** -5


def slow_inputs(L, dtype, device="cuda:0"):
    """Decays so slow that the entering state reaches the end: Δ near 0.02, A between -0.5 and -2."""
    x = gdr_inputs(2, L, 4, 2, 64, 64, dtype, seed=L, init=True, device=device)
    x["A"] = -torch.linspace(0.5, 2.0, 4).to(device)
    x["dt_bias"] = torch.full_like(x["A"], -4.0)
    return x


def derivative(J, x, name, grad):
    """(the derivative that the gradient claims, Richardson's difference of J) along the gradient's direction, one unit
    being the input's own size (1 for dt_bias, in whose unit Δ changes e-fold)."""
    unit = 1.0 if name == "dt_bias" else float(x[name].double().norm())
    d = grad.double() / grad.double().norm() * unit * (2.0 if name == "dt_bias" else 1.0)   # (4 heads: norm 2 is 1 each)

    def central(h):
        lo, hi = (J(**{name: (x[name].double() + s * h * d).to(x[name].dtype)}) for s in (-1, 1))
        return (hi - lo) / (2 * h)

    return float((grad.double() * d).sum()), (4 * central(H_STEP / 2) - central(H_STEP)) / 3


def compare(x, J, grads, size, off):
    """J is off by at most `off` of `size`, so Richardson's difference by 3 off / h of it; its own remainder is a fifth
    derivative times h^4 / 480 (J changes by less than itself per unit: under h^4 of size)."""
    bound = (3 * off / H_STEP + H_STEP ** 4) * size
    for name, grad in grads.items():
        ana, num = derivative(J, x, name, grad)
        assert bound <= abs(ana) / 10, (name, bound, ana)      # a gradient of zero, or of the wrong sign, fails
        assert abs(num - ana) <= bound, (name, num, ana, bound)


@pytest.mark.parametrize("L", [70, 200])
def test_chunks_against_differences_of_the_final_state(L):
    x = slow_inputs(L, BF)
    g = torch.Generator().manual_seed(L)
    dS = torch.randn(x["state"].shape, generator=g).to("cuda:0")

    def state(**change):
        z = {**x, **change}
        return ss.ss_gdr_fwd(*call_args(z), dt_bias=z["dt_bias"], initial_state=z["state"])[1].double()

    J = lambda **change: float((state(**change) * dS.double()).sum())  # noqa: E731
    got = ss.ss_gdr_bwd(*call_args(x), torch.zeros_like(x["v"]), dt_bias=x["dt_bias"], initial_state=x["state"],
                        dfinal_state=dS)
    # the state's own error, T's two terms of 2^-9 each and fp32 sums: under 2^-18 of it, in directions that dS does
    # not know (64 x 64 x 8 values: a hundredth of the product of the norms)
    size = float(state().norm() * dS.double().norm())
    compare(x, J, {"A": got["dA"], "dt_bias": got["ddt_bias"], "state": got["dinitial_state"]}, size, 2.0 ** -18 / 100)


@pytest.mark.parametrize("L", [30])
def test_fp32_against_differences_of_both_outputs(L):
    x = slow_inputs(L, F32)
    g = torch.Generator().manual_seed(L)
    dS, dy = (torch.randn(t.shape, generator=g).to("cuda:0") for t in (x["state"], x["v"]))

    def out(**change):
        z = {**x, **change}
        return [t.double() for t in ss.ss_gdr_fwd(*call_args(z), dt_bias=z["dt_bias"], initial_state=z["state"])]

    def J(**change):
        y, S = out(**change)
        return float((y * dy.double()).sum() + (S * dS.double()).sum())

    got = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS)
    y, S = out()
    size = float(S.norm() * dS.double().norm() + y.norm() * dy.double().norm())
    # 40 half-steps of 2^-24 a token, independent ones, against directions that do not know them
    names = {"A": "dA", "dt_bias": "ddt_bias", "state": "dinitial_state", "q": "dq", "k": "dk", "v": "dv", "dt": "ddt",
             "beta": "dbeta"}
    compare(x, J, {n: got[m] for n, m in names.items()}, size, 40 * 2.0 ** -24 * L ** 0.5 / 100)
