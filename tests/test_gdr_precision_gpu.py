"""GPU tests of how exact the gated delta rule in chunks is: bounds from the terms that its operands enter products with,
which a product with one term fewer does not meet."""
import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, f64, gdr_inputs, max_err, rms_err, state_tol, y_tol
from oracle import gdr
from ss_inputs import to_f64

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
DEV = "cuda:0"
# A rounding to bf16 is off by at most 2^-8 of the value; evenly spread, by 2^-8 / sqrt(3) on average where all values
# stand just above a power of two, and by less elsewhere.  Operands in two terms add 2^-16 at most, four in a row here.
ROUNDED = 2.0 ** -8 / 3 ** 0.5 + 4 * 2.0 ** -16
# What is rounded is off by under 2^-16 of itself, so that it falls to the other side of a rounding in at most 2 · 2^-16
# / step of all cases, a step being at most 2^-7, and is one step off there: sqrt(2 · 2^-16 · 2^-7) on average.  A
# product with one term (2^-9 off on average) is off by more than that everywhere.
OTHER_SIDE = 2.0 ** -11
# An operand in two terms is off by at most 2^-16 (both rounded to nearest: 2^-8 of 2^-8), on average by a third of it
# twice over; what a chain carries has three, and one operand beside it (T) two.
STATE = 2.0 ** -16 / 9
# The gates' gradients pass two such operands more (dV, and T on the way back).
GATES = 3 * 2.0 ** -16 / 9


def case(B, L, H, Hk, dk, dv, seed, **kw):
    x = gdr_inputs(B, L, H, Hk, dk, dv, seed=seed, init=True, **kw)
    g = torch.Generator().manual_seed(seed)
    dy = torch.randn(x["v"].shape, generator=g).to(BF).to(DEV)
    dS = torch.randn(x["state"].shape, generator=g).to(DEV)
    return x, dy, dS


@pytest.mark.parametrize("B,L,H,Hk,dk,dv", [(2, 400, 8, 8, 128, 128), (2, 333, 8, 4, 64, 128), (3, 250, 9, 3, 128, 64),
                                            (2, 150, 12, 12, 64, 64)])
@pytest.mark.parametrize("seed", [1, 2])
def test_outputs_and_gradients(B, L, H, Hk, dk, dv, seed):
    x, dy, dS = case(B, L, H, Hk, dk, dv, seed)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], sync_check=True)
    got = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS,
                        sync_check=True)
    z = f64(x)
    args = [z[n] for n in ("q", "k", "v", "dt", "A", "beta")]
    yr, Sr = gdr.gdr_fwd(*args, dt_bias=z["dt_bias"], h_init=z["state"], scale=dk ** -0.5)
    want = gdr.gdr_bwd(*args, to_f64(dy), dt_bias=z["dt_bias"], h_init=z["state"], dfinal=to_f64(dS), scale=dk ** -0.5)
    assert rms_err(y, yr) <= ROUNDED
    for n in ("dq", "dk", "dv", "ddt", "dbeta"):
        assert rms_err(got[n], want[n]) <= ROUNDED, n
    for n, t, r in (("y", y, yr), *((n, got[n], want[n]) for n in ("dq", "dk", "dv"))):
        off = to_f64(t) - to_f64(torch.tensor(r).to(BF))
        assert np.linalg.norm(off) <= OTHER_SIDE * np.linalg.norm(r), n
    assert rms_err(S, Sr) <= STATE
    assert rms_err(got["dinitial_state"], want["dinitial_state"]) <= STATE
    for n in ("dA", "ddt_bias"):
        assert rms_err(got[n], want[n]) <= GATES, n


def test_segments_keep_the_state():
    """The fold of the segments' maps adds nothing that shows."""
    x, _, _ = case(1, 2048, 4, 4, 128, 128, 3)
    z = f64(x)
    _, Sr = gdr.gdr_fwd(*(z[n] for n in ("q", "k", "v", "dt", "A", "beta")), dt_bias=z["dt_bias"], h_init=z["state"],
                        scale=128 ** -0.5)
    for seg in (1 << 30, 512, 128):
        _, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], chunk_len=seg, sync_check=True)
        assert rms_err(S, Sr) <= STATE, seg


@pytest.mark.parametrize("dtype,L", [(F32, 1), (F32, 9), (F32, 40), (BF, 2), (BF, 15)])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(6, 16, 8, 128, 128), (6, 16, 16, 64, 128), (12, 16, 4, 128, 64)])
def test_many_items_token_by_token(B, H, Hk, dk, dv, dtype, L):
    """Enough (batch, head) items for four rows of the state per thread, in a sequence and for single tokens."""
    x = gdr_inputs(B, L, H, Hk, dk, dv, dtype, seed=L, init=True)
    lens = torch.tensor([L, 0, 1, L // 2, L, L] * (B // 6), dtype=torch.int32, device=DEV)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], seqlens=lens, sync_check=True)
    z = f64(x)
    yr, Sr = gdr.gdr_fwd(*(z[n] for n in ("q", "k", "v", "dt", "A", "beta")), dt_bias=z["dt_bias"], h_init=z["state"],
                         seqlens=lens.cpu().numpy(), scale=dk ** -0.5)
    assert max_err(y, yr) <= (y_tol(L, F32) if dtype == F32 else y_tol(L, F32) + 2.0 ** -8)
    assert max_err(S, Sr) <= state_tol(L, F32)
    for b, n in enumerate(lens.tolist()):
        assert not y[b, n:].any()
    assert np.array_equal(to_f64(S[1]), z["state"][1])
