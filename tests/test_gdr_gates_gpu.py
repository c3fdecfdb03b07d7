"""GPU tests of the gates' gradients (ddt, dA, ddt_bias) where decays are strong, weak and mixed, against the 64-bit
oracle."""
import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, f64, gdr_inputs, rms_err
from oracle import gdr
from ss_inputs import to_f64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
# A path's share of log α's gradient passes at most six fp32 operands that enter a product as two bf16 terms (T, X, E, S
# before it, dE, dS behind it), each off by at most 2^-18 of itself; the paths of a head, and the heads, are independent,
# so that the norm over heads is off by no more than one path is.
GATES = 6 * 2.0 ** -18


def bwd(x, seed, **kw):
    g = torch.Generator(device="cpu").manual_seed(seed)
    dy = torch.randn(x["v"].shape, generator=g).to(x["v"].dtype).to(DEV)
    dS = torch.randn(x["state"].shape, generator=g).to(DEV)
    got = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS,
                        sync_check=True, **kw)
    z = f64(x)
    want = gdr.gdr_bwd(z["q"], z["k"], z["v"], z["dt"], z["A"], z["beta"], to_f64(dy), dt_bias=z["dt_bias"],
                       h_init=z["state"], dfinal=to_f64(dS), scale=x["q"].shape[-1] ** -0.5)
    return got, want


def check(x, seed, dtype=BF):
    got, want = bwd(x, seed)
    # ddt's own rounding, half a step, and what it is rounded from
    assert rms_err(got["ddt"], want["ddt"]) <= (2.0 ** -8 if dtype == BF else 2.0 ** -24) + GATES
    assert rms_err(got["dA"], want["dA"]) <= GATES
    assert rms_err(got["ddt_bias"], want["ddt_bias"]) <= GATES
    return got, want


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("A,bias", [(-16.0, 1.5), (-20.0, 1.0), (-1000.0, -3.0), (-4.0, 0.0), (-1e-4, -3.0)])
def test_one_decay(A, bias, dtype):
    """Δ A near -29, -27, -50, -3 and -5e-6: what is left of a path after one token, from 1e-22 of it to all."""
    x = gdr_inputs(2, 140, 8, 8, 64, 64, dtype, seed=int(-A) + 1, init=True)
    x["A"].fill_(A)
    x["dt_bias"].fill_(bias)
    check(x, 1, dtype)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64)])
def test_heads_of_unlike_decays(dk, dv):
    """Two value heads to a key head, from hardly any decay to one that empties the state in a token."""
    x = gdr_inputs(2, 200, 8, 4, dk, dv, seed=dk, init=True)
    x["A"] = -torch.tensor([1e-3, 0.1, 1, 4, 16, 16, 64, 200], device=DEV)
    x["dt_bias"] = torch.tensor([-3, -3, -3, -1, 0, 1.5, -0.5, -1], device=DEV, dtype=F32)
    got, want = check(x, 2)
    for h in range(8):   # each head by itself: its own sums are no larger than it is
        assert rms_err(got["ddt"][..., h], want["ddt"][..., h]) <= 2.0 ** -8 + 8 * GATES, h


def test_resets_between_slow_tokens():
    """Every ninth token empties the state; the others keep it."""
    x = gdr_inputs(2, 200, 8, 4, 128, 128, seed=5, init=True)
    x["A"].fill_(-1.0)
    x["dt_bias"].fill_(-4.0)
    x["dt"][:, ::9] = 34.0
    check(x, 3)


def test_key_heads_that_no_value_head_reads():
    """No value head: q's and k's gradients are written all the same."""
    x = gdr_inputs(2, 20, 0, 3, 64, 64, seed=1)
    g = {n: torch.full_like(x[n[1:]], 7.0) for n in ("dq", "dk")}
    ss.ss_gdr_bwd(*call_args(x), x["v"], grads=g, sync_check=True)
    assert not g["dq"].any() and not g["dk"].any()
