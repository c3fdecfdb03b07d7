"""GPU tests of the gated delta rule's forward and step against the 64-bit oracle (token by token)."""
import ctypes

import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import call_args, f64, gdr_inputs, max_err, rms_err, state_tol, y_tol
from oracle import gdr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
OPT = dict(softplus=True, beta_sigmoid=True, qk_l2norm=True)


def oracle_fwd(x, scale, seqlens=None, **opt):
    z = f64(x)
    return gdr.gdr_fwd(z["q"], z["k"], z["v"], z["dt"], z["A"], z["beta"], dt_bias=z.get("dt_bias"),
                       h_init=z.get("state"), seqlens=seqlens, scale=scale, **opt)


def check(x, L, dtype, seqlens=None, scale=None, **kw):
    opt = {**OPT, **{n: kw.pop(n) for n in tuple(kw) if n in OPT}}
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    lens = None if seqlens is None else torch.tensor(seqlens, dtype=torch.int32, device="cuda:0")
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x.get("dt_bias"), initial_state=x.get("state"), seqlens=lens,
                         scale=scale, sync_check=True, **opt, **kw)
    yr, Sr = oracle_fwd(x, scale, seqlens, **opt)
    assert max_err(y, yr) <= y_tol(L, dtype)
    assert max_err(S, Sr) <= state_tol(L, dtype)
    assert rms_err(S, Sr) <= 1e-5
    return y, S


LENGTHS = [1, 2, 7, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 333]


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_lengths(L, dtype):
    x = gdr_inputs(2, L, 4, 2, 128, 128, dtype, seed=L, init=L % 2 == 0)
    check(x, L, dtype)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2)])
@pytest.mark.parametrize("L", [5, 150])
def test_heads_and_widths(L, H, Hk, dk, dv):
    for dtype in (BF, F32):
        x = gdr_inputs(3, L, H, Hk, dk, dv, dtype, seed=dk + H, init=H == 3)
        check(x, L, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("L", [9, 100])
def test_options(dtype, L):
    x = gdr_inputs(2, L, 2, 2, 64, 128, dtype, seed=11, unit=False)
    check(x, L, dtype, qk_l2norm=False, scale=0.37)
    x["dt"] = (x["dt"].float().abs() * 0.1).to(dtype)
    x["beta"] = torch.rand_like(x["beta"].float()).to(dtype)
    x.pop("dt_bias")
    check(x, L, dtype, qk_l2norm=False, softplus=False, beta_sigmoid=False)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("L", [12, 200])
def test_padded_batch_ignores_what_lies_behind(dtype, L):
    """Lengths from zero to all; NaN and infinities behind the ends; rows of y behind the ends stay."""
    lens = [L, 0, 1, L // 2, L - 1, 5]
    x = gdr_inputs(6, L, 4, 2, 128, 128, dtype, seed=3, init=True)
    for b, n in enumerate(lens):
        for name, bad in (("q", np.nan), ("k", np.inf), ("v", np.nan), ("dt", np.nan), ("beta", -np.inf)):
            x[name][b, n:] = bad
    y = torch.full_like(x["v"], 7.0)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda:0")
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], seqlens=lt, y=y,
                         sync_check=True)
    yr, Sr = oracle_fwd(x, 128 ** -0.5, np.array(lens), **OPT)
    for b, n in enumerate(lens):
        assert bool((y[b, n:] == 7.0).all())
        assert max_err(y[b, :n], yr[b, :n]) <= y_tol(L, dtype)
    assert max_err(S, Sr) <= state_tol(L, dtype)
    assert torch.equal(S[1], x["state"][1])


def test_lengths_out_of_range_are_clamped():
    x = gdr_inputs(3, 70, 2, 2, 64, 64, seed=5)
    a = ss.ss_gdr_fwd(*call_args(x), seqlens=torch.tensor([-3, 1000, 70], dtype=torch.int32, device="cuda:0"))
    b = ss.ss_gdr_fwd(*call_args(x), seqlens=torch.tensor([0, 70, 70], dtype=torch.int32, device="cuda:0"))
    assert all(torch.equal(s, t) for s, t in zip(a, b))


@pytest.mark.parametrize("L", [10, 130])
def test_state_in_place_and_pieces(L):
    """final_state may be initial_state, and a sequence in two pieces gives the whole."""
    x = gdr_inputs(2, 2 * L, 4, 4, 128, 128, seed=8, init=True)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"])
    st = x["state"].clone()
    part = lambda s: [t[:, s].contiguous() if t.dim() > 1 else t for t in call_args(x)]  # noqa: E731
    ys = [ss.ss_gdr_fwd(*part(s), dt_bias=x["dt_bias"], initial_state=st, final_state=st)[0]
          for s in (slice(0, L), slice(L, None))]
    assert rms_err(st, S.double().cpu().numpy()) <= 1e-5
    assert max_err(torch.cat(ys, 1), y.double().cpu().numpy()) <= 2 * y_tol(2 * L, BF)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("A", [0.0, -1e-4, -1000.0])
def test_extreme_decays(dtype, A):
    """No decay at all, hardly any, and one that empties the state within a token."""
    x = gdr_inputs(2, 140, 2, 2, 128, 128, dtype, seed=21, init=True)
    x["A"].fill_(A)
    check(x, 140, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("dt", [400.0, 3.0e38, float("inf")])
@pytest.mark.parametrize("L", [10, 140])
def test_steps_that_empty_the_state(L, dt, dtype):
    """Gates so large that Δ A, and its sums, leave fp32's range: α is zero there and nowhere else."""
    x = gdr_inputs(2, L, 3, 3, 128, 128, dtype, seed=23, init=True)
    x["dt"][0, ::9, 0] = dt
    x["dt"][1, 5, :] = dt
    x["dt"][:, -3:, 2] = dt
    check(x, L, dtype)


def test_arguments_by_name_and_zeros_on_the_calls_stream():
    """y, made by the call, is cleared on the stream that the call is given."""
    x = gdr_inputs(3, 200, 2, 2, 64, 64, seed=41)
    lens = torch.tensor([200, 3, 0], dtype=torch.int32, device="cuda:0")
    names = ("q", "k", "v", "dt", "A", "beta", "dt_bias")
    want, S = ss.ss_gdr_fwd(**{n: x[n] for n in names}, seqlens=lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.empty_like(want).fill_(7.0)      # what the allocator hands out next
        torch.cuda.synchronize()
        y, S2 = ss.ss_gdr_fwd(**{n: x[n] for n in names}, seqlens=lens, stream=st)
        st.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(S, S2)
        assert not y[1, 3:].any() and not y[2].any()


def test_equal_keys():
    """One key again and again with β = 1: the chunk's triangular system has no small entry."""
    x = gdr_inputs(1, 130, 2, 2, 128, 128, seed=31)
    x["k"] = x["k"][:, :1].expand_as(x["k"]).contiguous()
    x["A"].zero_()
    x["beta"].fill_(1.0)
    check(x, 130, BF, beta_sigmoid=False)


def test_zero_length_and_empty():
    x = gdr_inputs(2, 0, 3, 3, 64, 64, init=True)
    y, S = ss.ss_gdr_fwd(*call_args(x), initial_state=x["state"], sync_check=True)
    assert y.shape == x["v"].shape and torch.equal(S, x["state"])
    _, S = ss.ss_gdr_fwd(*call_args(x), sync_check=True)
    assert not S.any()
    x = gdr_inputs(0, 5, 3, 3, 64, 64)
    y, S = ss.ss_gdr_fwd(*call_args(x), sync_check=True)
    assert y.numel() == 0 and S.numel() == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 1, 1, 64, 64), (3, 6, 2, 128, 64), (2, 4, 4, 64, 128), (70, 8, 4, 128, 128)])
def test_step(dtype, B, H, Hk, dk, dv):
    x = gdr_inputs(B, 1, H, Hk, dk, dv, dtype, seed=B + H, step=True)
    st = x["state"].clone()
    y = ss.ss_gdr_step(st, *call_args(x), dt_bias=x["dt_bias"], sync_check=True)
    z = {n: (t[:, None] if n in ("q", "k", "v", "dt", "beta") else t) for n, t in x.items()}
    yr, Sr = oracle_fwd(z, dk ** -0.5, **OPT)
    assert max_err(y, yr[:, 0]) <= (80 * 2.0 ** -24 if dtype == F32 else 2.0 ** -8 + 80 * 2.0 ** -24)
    assert max_err(st, Sr) <= 40 * 2.0 ** -24


def test_steps_give_the_sequence():
    x = gdr_inputs(2, 100, 4, 2, 128, 128, seed=77, init=True)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"])
    st = x["state"].clone()
    ys = []
    for t in range(100):
        q, k, v, dt, beta = (x[n][:, t].contiguous() for n in ("q", "k", "v", "dt", "beta"))
        ys.append(ss.ss_gdr_step(st, q, k, v, dt, x["A"], beta, dt_bias=x["dt_bias"]))
    assert rms_err(st, S.double().cpu().numpy()) <= 1e-5
    assert max_err(torch.stack(ys, 1), y.double().cpu().numpy()) <= 2 * y_tol(100, BF)


@pytest.mark.parametrize("L", [8, 200])
def test_captured_and_replayed_and_other_stream(L):
    """Two graphs captured from two calls, replayed at once on two streams, and a call on a side stream."""
    xs = [gdr_inputs(2, L, 4, 2, 128, 128, seed=s, init=True) for s in (1, 2)]
    want = [ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"]) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (y, S), (yw, Sw) in zip(outs, want):
        assert torch.equal(y, yw) and torch.equal(S, Sw)
    y, S = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    ss.ss_gdr_fwd(*call_args(xs[0]), dt_bias=xs[0]["dt_bias"], initial_state=xs[0]["state"], y=y, final_state=S,
                  stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(y, want[0][0]) and torch.equal(S, want[0][1])


def test_bounded_wait_reports_timeout_and_context_survives():
    """A hand-over that is never signalled (SS_TEST_DROP_CARRY: the first block's first product) runs the bounded
    waits out: the call reports SS_ERR_TIMEOUT, and the next call on the same context is right."""
    x = gdr_inputs(2, 300, 2, 2, 128, 128, seed=5)
    need = ss.lib().ss_gdr_fwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(2, 300, 2, 2, 128, 128)), ss.SS_BF16, 0)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda:0")
    ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], workspace=ws, timeout_iters=200,
                  extra_flags=ss.SS_TEST_DROP_CARRY)
    assert ss.ss_check(ws) == ss.SS_ERR_TIMEOUT
    check(x, 300, BF, workspace=ws)
    assert ss.ss_check(ws) == ss.SS_OK


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("L,seg", [(130, 64), (320, 128), (1000, 64), (700, 200)])
def test_time_segments(L, seg, dk, dv):
    """Forced segments (2 to 16): a state pass, the fold and the segments from their entering states."""
    x = gdr_inputs(2, L, 4, 2, dk, dv, seed=L + dk, init=dv == 64)
    check(x, L, BF, chunk_len=seg)


def test_time_segments_of_a_padded_batch():
    """Segments behind a sequence's end pass its state on."""
    lens = [600, 0, 1, 64, 300, 599]
    x = gdr_inputs(6, 600, 2, 2, 128, 128, seed=4, init=True)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "dt", "beta"):
            x[name][b, n:] = np.nan
    y = torch.full_like(x["v"], 7.0)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda:0")
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], seqlens=lt, y=y, chunk_len=128,
                         sync_check=True)
    yr, Sr = oracle_fwd(x, 128 ** -0.5, np.array(lens), **OPT)
    for b, n in enumerate(lens):
        assert bool((y[b, n:] == 7.0).all())
        assert max_err(y[b, :n], yr[b, :n]) <= y_tol(600, BF)
    assert max_err(S, Sr) <= state_tol(600, BF)
    assert rms_err(S, Sr) <= 1e-5


def test_time_segments_with_the_state_in_place():
    """final_state = initial_state in segments: the first one's entering state is read from a copy."""
    x = gdr_inputs(2, 640, 4, 2, 128, 128, seed=12, init=True)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=x["state"], chunk_len=64)
    st = x["state"].clone()
    y2, S2 = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], initial_state=st, final_state=st, chunk_len=64)
    assert S2 is st and torch.equal(S, st) and torch.equal(y, y2)


def test_segments_of_the_last_wave():
    """More items than SMs: those of the last wave are cut, the others run whole; all give the whole sequence's
    results (which the oracle checks elsewhere)."""
    x = gdr_inputs(20, 512, 8, 4, 64, 64, seed=6)
    y, S = ss.ss_gdr_fwd(*call_args(x), dt_bias=x["dt_bias"], sync_check=True)
    st = None
    ys = []
    for i in range(0, 512, 64):   # token pieces of one chunk: no segments
        part = [t[:, i:i + 64].contiguous() if t.dim() > 1 else t for t in call_args(x)]
        yy, st = ss.ss_gdr_fwd(*part, dt_bias=x["dt_bias"], initial_state=st)
        ys.append(yy)
    assert rms_err(S, st.double().cpu().numpy()) <= 1e-5
    assert max_err(y, torch.cat(ys, 1).double().cpu().numpy()) <= 2 * y_tol(512, BF)
