"""Host-side checks of the gated delta rule's and the layer norm's entry points: refusals before anything is
launched, workspace sizes, and the binding's own checks (no GPU)."""
import ctypes

import pytest
import torch

import selective_state_space_37_b200 as ss

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    return ss.lib()


def fwd(L, dims=(2, 64, 4, 2, 128, 64), flags=ss.SS_BF16, ws=(0x90000, 1 << 30), launch=True, **ptr):
    a = dict(q=0x10000, k=0x20000, v=0x30000, dt=0x40000, dt_bias=None, A=0x50000, beta=0x60000, h_init=None,
             seqlens=None, y=0x70000, final_state=None)
    a.update(ptr)
    la = ss.ss_launch(None, ws[0], ws[1], 0, 0)
    return L.ss_gdr_fwd(*(P(v) if v else None for v in a.values()), 1.0, flags,
                        None if dims is None else ctypes.byref(ss.ss_gdr_dims(*dims)),
                        ctypes.byref(la) if launch else None)


BAD_DIMS = [((-1, 64, 4, 2, 128, 64), ss.SS_ERR_INVALID_ARG), ((2, -1, 4, 2, 128, 64), ss.SS_ERR_INVALID_ARG),
            ((2, 64, -4, 2, 128, 64), ss.SS_ERR_INVALID_ARG), ((2, 64, 4, 3, 128, 64), ss.SS_ERR_INVALID_ARG),
            ((2, 64, 4, 0, 128, 64), ss.SS_ERR_INVALID_ARG), ((2, 64, 4, 8, 128, 64), ss.SS_ERR_INVALID_ARG),
            ((2, 64, 4, 2, 96, 64), ss.SS_ERR_UNSUPPORTED), ((2, 64, 4, 2, 128, 256), ss.SS_ERR_UNSUPPORTED),
            ((2, 64, 4, 2, 0, 64), ss.SS_ERR_UNSUPPORTED), ((1 << 27, 64, 4, 2, 128, 64), ss.SS_ERR_INVALID_ARG),
            ((1, 1 << 31, 4, 2, 128, 64), ss.SS_ERR_INVALID_ARG)]


@pytest.mark.parametrize("dims,want", BAD_DIMS)
def test_gdr_sizes_are_refused(L, dims, want):
    assert fwd(L, dims) == want
    assert L.ss_gdr_fwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(*dims)), ss.SS_BF16, 0) == 0


def test_gdr_fwd_refusals(L):
    bad = ss.SS_ERR_INVALID_ARG
    assert fwd(L, None) == bad
    assert fwd(L, launch=False) == bad
    for name in ("q", "k", "v", "dt", "A", "beta", "y"):
        assert fwd(L, **{name: None}) == bad, name
    for name in ("q", "dt", "dt_bias", "A", "beta", "h_init", "seqlens", "y", "final_state"):
        assert fwd(L, **{name: 0x70004}) == bad, name
    assert fwd(L, flags=ss.SS_BF16 | 1 << 12) == bad
    assert fwd(L, flags=ss.SS_BF16 | ss.SS_FORCE_GENERAL_A) == bad
    assert fwd(L, ws=(None, 0)) == ss.SS_ERR_WORKSPACE
    assert fwd(L, ws=(0x90000, 8)) == ss.SS_ERR_WORKSPACE
    assert fwd(L, ws=(0x90008, 1 << 30)) == ss.SS_ERR_WORKSPACE
    assert fwd(L, (0, 64, 4, 2, 128, 64)) == ss.SS_OK
    assert fwd(L, (2, 64, 0, 0, 128, 64)) == ss.SS_OK


def test_gdr_step_refusals(L):
    def step(dims=(2, 0, 4, 2, 128, 64), flags=0, **ptr):
        a = dict(state=0x8000, q=0x10000, k=0x20000, v=0x30000, dt=0x40000, dt_bias=None, A=0x50000, beta=0x60000,
                 y=0x70000)
        a.update(ptr)
        return L.ss_gdr_step(*(P(v) if v else None for v in a.values()), 1.0, flags,
                             ctypes.byref(ss.ss_gdr_dims(*dims)), ctypes.byref(ss.ss_launch(None, None, 0, 0, 0)))

    for name in ("state", "q", "k", "v", "dt", "A", "beta", "y"):
        assert step(**{name: None}) == ss.SS_ERR_INVALID_ARG, name
        assert step(**{name: 0x70002}) == ss.SS_ERR_INVALID_ARG, name
    assert step((2, 0, 4, 2, 32, 64)) == ss.SS_ERR_UNSUPPORTED
    assert step((2, 0, 4, 3, 64, 64)) == ss.SS_ERR_INVALID_ARG
    assert step(flags=1 << 20) == ss.SS_ERR_INVALID_ARG
    assert step((0, 0, 4, 2, 64, 64)) == ss.SS_OK


def test_gdr_bwd_refusals(L):
    d = (2, 64, 4, 2, 128, 64)
    need = L.ss_gdr_bwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(*d)), ss.SS_BF16)
    assert need > 0
    assert L.ss_gdr_bwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(*d)), 0) > 0

    def bwd(dims=d, flags=ss.SS_BF16, ws=(0x900000, need), launch=True, **ptr):
        names = ("q", "k", "v", "dt", "dt_bias", "A", "beta", "h_init", "seqlens", "dy", "dfinal_state", "dq", "dk",
                 "dv", "ddt", "dbeta", "dA", "ddt_bias", "dh_init")
        a = {n: 0x10000 * (i + 1) for i, n in enumerate(names)}
        a.update(ptr)
        la = ss.ss_launch(None, ws[0], ws[1], 0, 0)
        return L.ss_gdr_bwd(*(P(v) if v else None for v in a.values()), 1.0, flags,
                            None if dims is None else ctypes.byref(ss.ss_gdr_dims(*dims)),
                            ctypes.byref(la) if launch else None)

    bad = ss.SS_ERR_INVALID_ARG
    assert bwd(None) == bad and bwd(launch=False) == bad
    assert bwd(flags=0, ws=(0x900000, 4096)) == ss.SS_ERR_WORKSPACE
    assert bwd(flags=ss.SS_BF16 | 1 << 12) == bad
    for name in ("q", "k", "v", "dt", "A", "beta", "dy", "dq", "dk", "dv", "ddt", "dbeta", "dA"):
        assert bwd(**{name: None}) == bad, name
    for name in ("q", "dt_bias", "h_init", "seqlens", "dy", "dfinal_state", "dq", "dbeta", "dA", "ddt_bias", "dh_init"):
        assert bwd(**{name: 0x700004}) == bad, name
    assert bwd(dt_bias=None) == bad                       # a gradient of nothing
    assert bwd(ws=(0x900000, need - 1)) == ss.SS_ERR_WORKSPACE
    assert bwd(ws=(None, need)) == ss.SS_ERR_WORKSPACE
    assert bwd(ws=(0x900004, need)) == ss.SS_ERR_WORKSPACE
    for dims, want in BAD_DIMS:
        assert bwd(dims) == want, dims
        assert L.ss_gdr_bwd_workspace_bytes(ctypes.byref(ss.ss_gdr_dims(*dims)), ss.SS_BF16) == 0
    assert bwd((2, 64, 0, 0, 128, 64)) == ss.SS_OK


@pytest.mark.parametrize("L_,H", [(16, 1), (1000, 4), (100000, 16), (130, 300)])
def test_gdr_workspace_grows_with_the_segments(L, L_, H):
    """Records for every chunk, and states for the segments that a call is cut into; token by token needs neither."""
    size = lambda n, f=ss.SS_BF16, cl=0: L.ss_gdr_fwd_workspace_bytes(  # noqa: E731
        ctypes.byref(ss.ss_gdr_dims(1, n, H, H, 128, 128)), f, cl)
    chunks = -(-L_ // 64)
    whole = size(L_, cl=1 << 30)
    assert whole >= H * chunks * 33 * 1024
    assert size(L_, cl=64) >= whole + (H * min(chunks - 1, 1) * 3 * 65536 if chunks > 1 else 0)
    assert size(L_) >= whole
    assert size(L_, 0) == size(15) < 4096


def test_prenorm_refusals(L):
    w = ss.ss_block_weights()
    for n, v in (("d_model", 64), ("d_inner", 128), ("dt_rank", 8)):
        setattr(w, n, v)
    for i, n in enumerate(("in_proj_x", "in_proj_z", "conv_w", "x_proj_dt", "x_proj_B", "x_proj_C", "dt_proj", "dt_bias",
                           "A", "out_proj")):
        setattr(w, n, 0x100000 * (i + 1))
    need = L.ss_block_prenorm_scratch_bytes(ctypes.byref(w), 1, 16)
    assert need > L.ss_block_scratch_bytes(ctypes.byref(w), 1, 16) > 0
    assert L.ss_block_prenorm_scratch_bytes(ctypes.byref(w), -1, 16) == 0

    def call(hidden=0x10000, nw=None, nb=None, eps=1e-5, out=0x20000, batch=1, scratch=0x30000, size=need):
        return L.ss_block_fwd_prenorm(P(hidden) if hidden else None, P(nw) if nw else None, P(nb) if nb else None, eps,
                                      P(out) if out else None, ctypes.byref(w), batch, 16,
                                      P(scratch) if scratch else None, size, None)

    bad = ss.SS_ERR_INVALID_ARG
    assert call(hidden=None) == bad and call(out=None) == bad and call(batch=-1) == bad
    assert call(hidden=0x10004) == bad and call(out=0x20004) == bad
    assert call(nw=0x40004) == bad and call(nb=0x40004) == bad
    assert call(eps=-1.0) == bad and call(eps=float("nan")) == bad
    assert call(out=0x10000) == bad                       # out in hidden's place
    assert call(scratch=None) != ss.SS_OK and call(size=need - 1) != ss.SS_OK


def test_older_entry_points_refuse_the_new_flags(L):
    d = ss.ss_dims(0, 64, 128, 16)
    la = ss.ss_launch(None, None, 0, 0, 0)
    for f in (ss.SS_BETA_SIGMOID, ss.SS_QK_L2NORM):
        assert L.ss_fwd(*[None] * 10, f, ctypes.byref(d), ctypes.byref(la)) == ss.SS_ERR_INVALID_ARG


def test_norm_refusals(L):
    la = ss.ss_launch(None, 0x90000, 1 << 30, 0, 0)

    def fw(dims=(4, 64), eps=1e-5, flags=0, **ptr):
        a = dict(x=0x10000, weight=None, bias=None, y=0x20000, mean=None, rstd=None)
        a.update(ptr)
        return L.ss_norm_fwd(*(P(v) if v else None for v in a.values()), eps, flags,
                             ctypes.byref(ss.ss_norm_dims(*dims)), ctypes.byref(la))

    def bw(dims=(4, 64), flags=0, la=la, **ptr):
        a = dict(dy=0x10000, x=0x20000, mean=0x30000, rstd=0x40000, weight=None, dx=0x50000, dweight=0x60000, dbias=None)
        a.update(ptr)
        return L.ss_norm_bwd(*(P(v) if v else None for v in a.values()), flags, ctypes.byref(ss.ss_norm_dims(*dims)),
                             ctypes.byref(la))

    for f in (fw, bw):
        for dims in ((-1, 64), (4, -1), (4, 0), (1, 1 << 31)):
            assert f(dims) == ss.SS_ERR_INVALID_ARG, dims
        assert f(flags=ss.SS_DELTA_SOFTPLUS) == ss.SS_ERR_INVALID_ARG
        assert f(x=None) == ss.SS_ERR_INVALID_ARG
        assert f(x=0x10004) == ss.SS_ERR_INVALID_ARG
    assert fw((0, 64)) == ss.SS_OK
    assert fw(eps=-1.0) == ss.SS_ERR_INVALID_ARG
    assert fw(eps=float("nan")) == ss.SS_ERR_INVALID_ARG
    assert fw(weight=0x10004) == ss.SS_ERR_INVALID_ARG
    for name in ("dy", "mean", "rstd", "dx"):
        assert bw(**{name: None}) == ss.SS_ERR_INVALID_ARG, name
    need = L.ss_norm_bwd_workspace_bytes(ctypes.byref(ss.ss_norm_dims(4, 64)), 0)
    assert need >= 256
    assert bw(la=ss.ss_launch(None, 0x90000, need - 1, 0, 0)) == ss.SS_ERR_WORKSPACE
    assert bw(la=ss.ss_launch(None, None, 0, 0, 0)) == ss.SS_ERR_WORKSPACE
    assert L.ss_norm_bwd_workspace_bytes(ctypes.byref(ss.ss_norm_dims(4, -1)), 0) == 0


def test_binding_checks():
    x = torch.zeros(2, 8, 2, 64)
    g = torch.zeros(2, 8, 2)
    A = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_gdr_fwd(x, x, x, g, A, g)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_gdr_step(torch.zeros(2, 2, 64, 64), x[:, 0], x[:, 0], x[:, 0], g[:, 0], A, g[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_norm_fwd(torch.zeros(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_norm_bwd(torch.zeros(2, 8), torch.zeros(2, 8), torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_block_fwd_prenorm(torch.zeros(2, 8, 8), {})
    with pytest.raises(ValueError, match="CUDA"):   # every argument by name
        ss.ss_gdr_fwd(q=x, k=x, v=x, dt=g, A=A, beta=g)
    with pytest.raises(ValueError, match="CUDA"):
        ss.ss_norm_fwd(x=torch.zeros(2, 8))


def test_gdr_bwd_without_value_heads(L):
    """dq and dk are written, so they are asked for; nothing else is."""
    la = ss.ss_launch(None, None, 0, 0, 0)

    def bwd(hk, dq=None, dk=None, batch=2):
        a = [None] * 11 + [dq, dk] + [None] * 6
        return L.ss_gdr_bwd(*(P(v) if v else None for v in a), 1.0, ss.SS_BF16,
                            ctypes.byref(ss.ss_gdr_dims(batch, 64, 0, hk, 128, 64)), ctypes.byref(la))

    bad = ss.SS_ERR_INVALID_ARG
    assert bwd(2) == bad and bwd(2, 0x10000) == bad and bwd(2, 0x10000, 0x20004) == bad
    assert bwd(1 << 60, 0x10000, 0x20000) == bad
    assert bwd(0) == ss.SS_OK and bwd(2, batch=0) == ss.SS_OK
