"""GPU tests of the gated delta rule's backward pass token by token (fp32 of any length, short bf16 sequences)."""
import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import U32, call_args, gdr_inputs, max_err, rms_err
from ss_inputs import to_f64
from test_gdr_bwd_gpu import BF, DEV, SEQ_GRADS, gate_bound, oracle_bwd, upstream

pytestmark = pytest.mark.gpu
F32 = torch.float32


def check(x, seed=0, seqlens=None, scale=None, final=True, up=None, **opt):
    dtype = x["q"].dtype
    dy, dS = up or upstream(x, seed, final)
    dy = dy.to(dtype)
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    L = x["q"].shape[1]
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device=DEV)
    g = ss.ss_gdr_bwd(*call_args(x), dy, dt_bias=x.get("dt_bias"), initial_state=x.get("state"), dfinal_state=dS,
                      seqlens=lens, scale=scale, sync_check=True, **opt)
    np_lens = None if seqlens is None else np.array(seqlens)
    want = oracle_bwd(x, dy, dS, np_lens, scale, **opt)
    # The state, its adjoint and the product of the two: three series of under 40 half-steps of 2^-24 a token, which
    # add up like independent errors over the tokens; bf16 outputs round once more (half a step).
    tol = 3 * 40 * U32 * max(L, 1) ** 0.5
    out = 2.0 ** -8 if dtype == BF else 0.0
    for n in SEQ_GRADS:
        assert g[n].dtype == dtype
        assert rms_err(g[n], want[n]) <= tol + out, n
        assert max_err(g[n], want[n]) <= 4 * tol + out, n
    bA, bb = gate_bound(want, x, dy, np_lens, scale, **opt)   # (made for 2^-15 per product; here 120 · 2^-24 < 2^-17)
    assert np.all(np.abs(to_f64(g["dA"]) - want["dA"]) <= bA / 4 + 1e-30)
    if "dt_bias" in x:
        assert np.all(np.abs(to_f64(g["ddt_bias"]) - want["ddt_bias"]) <= bb / 4 + 1e-6 * np.abs(want["ddt_bias"]) + 1e-30)
    if "state" in x:
        assert rms_err(g["dinitial_state"], want["dinitial_state"]) <= tol
    return g, want


@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 16, 63, 130])
def test_lengths_fp32(L):
    check(gdr_inputs(2, L, 4, 2, 64, 128, F32, seed=L, init=True), L)


@pytest.mark.parametrize("L", [1, 2, 5, 7])
def test_short_bf16(L):
    check(gdr_inputs(3, L, 4, 2, 128, 64, seed=L, init=True), L)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2)])
def test_heads_and_widths(H, Hk, dk, dv):
    check(gdr_inputs(2, 21, H, Hk, dk, dv, F32, seed=H + dk, init=H != 3), H, final=H != 1)


def test_options():
    x = gdr_inputs(2, 30, 2, 1, 64, 64, F32, seed=8, unit=False)
    x["dt"] = x["dt"].abs() * 0.1
    x["beta"] = torch.sigmoid(x["beta"])
    x["beta"][:, ::7] = 0.0   # β's gradient where β is zero
    del x["dt_bias"]
    check(x, 2, qk_l2norm=False, softplus=False, beta_sigmoid=False, scale=0.3)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_padded_batch_ignores_what_lies_behind(dtype):
    L, lens = (7, [7, 0, 1, 4, 6, 5]) if dtype == BF else (29, [29, 0, 1, 14, 28, 8])
    x = gdr_inputs(6, L, 4, 2, 128, 128, dtype, seed=3, init=True)
    dy, dS = upstream(x, 5)
    dy = dy.to(dtype)
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
    x = gdr_inputs(2, 40, 2, 2, 128, 128, F32, seed=21, init=True)
    x["A"].fill_(A)
    check(x, 7)


def test_steps_that_empty_the_state():
    x = gdr_inputs(2, 40, 3, 3, 128, 128, F32, seed=23, init=True)
    x["dt"][0, ::9, 0] = 3.0e38
    x["dt"][1, 5, :] = 400.0
    x["dt"][:, -3:, 2] = 3.0e38
    check(x, 3)


def test_both_ways_agree_at_the_border():
    """The last length that runs token by token and the first that runs in chunks, on the same tokens: the longer call's
    last token does not count."""
    x = gdr_inputs(2, 8, 2, 2, 128, 128, seed=5, init=True)
    dy, dS = upstream(x, 2)
    lens = torch.tensor([7, 7], dtype=torch.int32, device=DEV)
    kw = dict(dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS)
    a = ss.ss_gdr_bwd(*call_args(x), dy, seqlens=lens, **kw)
    short = [t[:, :7].contiguous() if t.dim() > 1 else t for t in call_args(x)]
    b = ss.ss_gdr_bwd(*short, dy[:, :7].contiguous(), **kw)
    for n in SEQ_GRADS:
        assert rms_err(a[n][:, :7], to_f64(b[n])) <= 5e-3, n
    assert rms_err(a["dinitial_state"], to_f64(b["dinitial_state"])) <= 1e-5


def test_same_bits_and_captured_graphs():
    x = gdr_inputs(2, 20, 4, 2, 64, 64, F32, seed=9, init=True)
    dy, dS = upstream(x, 4)
    dy = dy.float()
    kw = dict(dt_bias=x["dt_bias"], initial_state=x["state"], dfinal_state=dS)
    want = ss.ss_gdr_bwd(*call_args(x), dy, **kw)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        ss.ss_gdr_bwd(*call_args(x), dy, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = ss.ss_gdr_bwd(*call_args(x), dy, **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n, t in want.items():
        assert torch.equal(got[n], t), n
