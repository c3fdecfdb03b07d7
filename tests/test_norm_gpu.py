"""GPU tests of the layer norm's forward and backward against the 64-bit oracle, and of the block behind it."""
import numpy as np
import pytest
import torch

import selective_state_space_37_b200 as ss
from gdr_util import U32, max_err
from oracle import block as oracle_block
from oracle import gdr
from ss_inputs import block_inputs, to_f64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32

# cols: below and above a warp's reach (512), one vector more or less, odd, the widest held row (8192), beyond it
SHAPES = [(1, 1), (3, 2), (5, 7), (300, 64), (9, 511), (9, 512), (9, 520), (7, 777), (33, 1000), (2000, 1536), (5, 2560),
          (17, 4095), (3, 8192), (3, 8193), (4, 8200), (2, 20000)]


def inputs(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * (0.5 + torch.rand(rows, 1, generator=g))
         + torch.randn(rows, 1, generator=g)).to(dtype)
    w, b = 1 + 0.2 * torch.randn(cols, generator=g), 0.2 * torch.randn(cols, generator=g)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    return [t.to(DEV) for t in (x, w, b, dy)]


def half(dtype):
    return 2.0 ** -8 if dtype == BF else 2.0 ** -24


def chain(cols):
    """Roundings of a sum over a row: 16 values in a thread (or cols / 512 of them), 5 shuffles twice."""
    return max(16, cols // 512) + 12


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, dtype):
    x, w, b, dy = inputs(rows, cols, dtype, cols)
    y, mean, rstd = ss.ss_norm_fwd(x, w, b, eps=1e-5, sync_check=True)
    yr, mr, rr = gdr.norm_fwd(to_f64(x), to_f64(w), to_f64(b), 1e-5)
    scale = float(np.max(np.abs(to_f64(x))))
    assert np.max(np.abs(to_f64(mean) - mr)) <= chain(cols) * U32 * scale
    # |x - μ| carries the mean's error, its square twice that; 1 / sqrt halves a relative error.  A row that is
    # nearly constant has its error against eps.
    err = chain(cols) * U32 * scale
    dev = 4 * (err * rr + chain(cols) * U32)
    assert np.all(np.abs(to_f64(rstd) - rr) <= dev * rr)
    # y = x̂ w + b with x̂'s error that of (x - μ) r
    bound = (np.max(np.abs(to_f64(w))) * (4 * err * rr[:, None] + (dev[:, None] + 4 * U32) * np.abs(to_f64(x) - mr[:, None]) * rr[:, None])
             + (half(dtype) + U32) * np.abs(yr))
    assert np.all(np.abs(to_f64(y) - yr) <= bound + 1e-30)

    g = ss.ss_norm_bwd(dy, x, mean, rstd, w, sync_check=True)
    want = gdr.norm_bwd(to_f64(dy), to_f64(x), to_f64(mean), to_f64(rstd), to_f64(w))
    # x̂ from the same statistics: 2 roundings; the two means a row's chain; dx is a sum of three such terms
    big = float(np.max(np.abs(want["dx"]))) if cols > 1 else 1.0
    xh = np.max(np.abs((to_f64(x) - to_f64(mean)[:, None]) * to_f64(rstd)[:, None]))
    row = np.max(np.abs(to_f64(dy) * to_f64(w)), 1, keepdims=True) * to_f64(rstd)[:, None] * (2 + xh * xh)
    xerr = 2 * U32 * scale * to_f64(rstd)[:, None] * (1 + xh) * row   # x - μ where both are large
    tol = (chain(cols) + 8) * U32 * row + xerr + half(dtype) * np.abs(want["dx"]) + 1e-30
    assert np.all(np.abs(to_f64(g["dx"]) - want["dx"]) <= tol), big
    # a column's sum: rows / blocks terms in a chain, then the partial rows; each term |dy x̂|
    n = rows + 16
    for name, term in (("dweight", np.abs(to_f64(dy)) * np.abs((to_f64(x) - to_f64(mean)[:, None]) * to_f64(rstd)[:, None])),
                       ("dbias", np.abs(to_f64(dy)))):
        slack = 3 * U32 * scale * np.max(to_f64(rstd)) * np.abs(to_f64(dy)).sum(0) if name == "dweight" else 0.0
        assert np.all(np.abs(to_f64(g[name]) - want[name]) <= min(n, 200) * U32 * term.sum(0) + slack + 1e-30), name
    g2 = ss.ss_norm_bwd(dy, x, mean, rstd, w)
    assert all(torch.equal(g[k], g2[k]) for k in g)   # no order that changes


def test_without_parameters_in_place_and_empty():
    x, w, b, dy = inputs(40, 96, F32, 1)
    y, mean, rstd = ss.ss_norm_fwd(x)
    yr, _, _ = gdr.norm_fwd(to_f64(x))
    assert max_err(y, yr) <= 200 * U32
    z = x.clone()
    out, _, _ = ss.ss_norm_fwd(z, y=z)
    assert out is z and torch.equal(z, y)
    g = ss.ss_norm_bwd(dy, x, mean, rstd)
    d = dy.clone()
    g2 = ss.ss_norm_bwd(d, x, mean, rstd, dx=d)
    assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dweight"], g2["dweight"])
    wide, _, _, dwide = inputs(3, 20000, BF, 2)
    yw, mw, rw = ss.ss_norm_fwd(wide)
    zw = wide.clone()
    assert torch.equal(ss.ss_norm_fwd(zw, y=zw)[0], yw)
    gw = ss.ss_norm_bwd(dwide, wide, mw, rw)
    dw = dwide.clone()
    gw2 = ss.ss_norm_bwd(dw, wide, mw, rw, dx=dw)
    assert all(torch.equal(gw[k], gw2[k]) for k in gw)
    assert set(ss.ss_norm_bwd(dy, x, mean, rstd, sums=False)) == {"dx"}
    e = torch.empty(0, 64, device=DEV)
    s = torch.empty(0, device=DEV)
    assert ss.ss_norm_fwd(e)[0].shape == (0, 64)
    g = ss.ss_norm_bwd(e, e, s, s)
    assert not g["dweight"].any() and not g["dbias"].any()


def test_constant_rows_and_not_finite_values():
    x = torch.full((4, 640), 3.0, device=DEV)
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    y, mean, rstd = ss.ss_norm_fwd(x)
    assert not y[0].any() and not y[3].any()           # variance 0: eps alone
    assert torch.isnan(y[1:3]).any(1).all()            # and only the rows that hold them
    assert mean[0] == 3.0 and abs(float(rstd[0]) - 1e-5 ** -0.5) <= 2 * U32 * 1e-5 ** -0.5


def test_large_mean_keeps_the_variance():
    x = torch.randn(8, 1024, device=DEV) + 1000.0
    y, _, _ = ss.ss_norm_fwd(x)
    yr, _, _ = gdr.norm_fwd(to_f64(x))
    # x itself is exact; x - μ loses the mean's error of about 28 half-steps of 1000 at most
    assert max_err(y, yr) <= 28 * U32 * 1000 * 2 / 3


def test_captured_graphs_of_backward():
    xs = [inputs(500, 640, BF, s) for s in (1, 2)]
    st = [ss.ss_norm_fwd(x, w, b)[1:] for x, w, b, _ in xs]
    want = [ss.ss_norm_bwd(dy, x, *s, w) for (x, w, b, dy), s in zip(xs, st)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for (x, w, b, dy), s in zip(xs, st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ss.ss_norm_bwd(dy, x, *s, w))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(o[k], w[k]) for k in w)


def test_block_behind_its_norm():
    """out = hidden + block(norm(hidden)); the block's oracle rounds what the block stores in bf16."""
    hidden, w = block_inputs(2, 40, 64, seed=9, device=DEV)
    nw, nb = 1 + 0.1 * torch.randn(64, device=DEV), 0.1 * torch.randn(64, device=DEV)
    out = ss.ss_block_fwd_prenorm(hidden, w, nw, nb)
    x = oracle_block.round_bf16(gdr.norm_fwd(to_f64(hidden), to_f64(nw), to_f64(nb))[0])
    want = to_f64(hidden) + oracle_block.block_fwd(x, {k: to_f64(v) for k, v in w.items()})
    # the block's own bound, and one rounding of the sum
    assert max_err(out, want) <= 2e-2 + 2.0 ** -8
    plain = ss.ss_block_fwd(ss.ss_norm_fwd(hidden, nw, nb)[0], w)
    # the same block, its output rounded before the sum instead of after it
    assert max_err(out, to_f64(hidden) + to_f64(plain)) <= 2 * 2.0 ** -8
    with pytest.raises(ss.SelscanError):
        ss.ss_block_fwd_prenorm(hidden, w, out=hidden)
