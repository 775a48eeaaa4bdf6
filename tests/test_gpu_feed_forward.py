"""The gated activation, the residual norms and their gradients on the GPU against the plain 64-bit implementations.

Tolerances, from the arithmetic (eps = 2^-24, half a step of fp32):

* act(g) u: the exponential of the rounded product z log2(e) is within (2 + 1.5 |z|) eps of its value, 1 + e, the reciprocal
  and three products add one or two each, and an argument z that is rounded itself (GELU: 4 operations) changes the exponential by
  4 eps |z|; below (10 + 6 |z|) eps of the value.  A slope is a sum of two such terms and is held to their magnitudes.
* norms: a lane adds at most 16 squares, then 10 additions join lanes and waves; the square root halves that, five more
  operations follow, and the second norm inherits the first's error: below 80 eps of the magnitudes of the terms that
  are added (|residual| + |scale gate z| for the sum).
* column sums over the rows: chains of at most 16 rows and 16 + 64 partials more, below 200 eps of the terms' magnitudes.
* one rounding to the output's type: OUT_REL.
* quantized outputs are the library's quantizers of the fp32 values: the same bits as the fp32 call followed by them.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
import oracle
from gpu_util import device, say

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = [F32, BF16, F16]
EPS = 2.0 ** -24
OUT_REL = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
OUT_ABS = {F32: 2.0 ** -126, BF16: 2.0 ** -126, F16: 2.0 ** -25}   # exponentials below 2^-126 count as zero
OF = oracle.feed_forward


def host(t):
    return t.detach().double().cpu().numpy()


def rand(rng, *shape, dtype=F32, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(device=device(), dtype=dtype)


def near(got, want, tol, dtype, what=""):
    g = host(got)
    bad = ~(np.abs(g - want) <= tol + OUT_REL[dtype] * (np.abs(want) + tol) + OUT_ABS[dtype])
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, the first by {np.abs(g - want)[bad][0]:.3g}"


def same_bits(a, b, what=""):
    assert a.dtype == b.dtype and a.shape == b.shape, what
    n = a.element_size()
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[n]
    assert torch.equal(a.contiguous().view(view), b.contiguous().view(view)), what


def act_tol(pre, act):
    """(values, relative tolerance) of h."""
    g = pre[..., :pre.shape[-1] // 2]
    return (10 + 6 * np.abs(OF._arg(g, act)[0])) * EPS


# ---- the activation -------------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,n", [(1, 16), (3, 128), (17, 144), (130, 1040), (33, 4112), (5, 16400), (9, 1024), (3, 8192), (2, 8208)])
def test_act(rows, n, act):
    rng = np.random.default_rng(rows * n)
    for dtype in DTYPES:
        say("act", rows, n, act, dtype)
        pre = rand(rng, rows, 2 * n, dtype=dtype, scale=2.0)
        pre[0, :4] = torch.tensor([0.0, -0.0, 30.0, -30.0], device=device(), dtype=dtype)
        h = dg.dg_gated_act(pre, act=act)
        want = OF.gated(host(pre), act)
        near(h, want, act_tol(host(pre), act) * np.abs(want), dtype)
        same_bits(h, dg.dg_gated_act(pre, act=act))
        # quantized: the quantizers' bits of the fp32 values
        wide = dg.dg_gated_act(pre.float(), act=act)
        q, s = dg.dg_gated_act_fp8(pre, act=act)
        q2, s2 = dg.dg_quantize_per_token_group(wide)
        same_bits(q, q2, "fp8 codes")
        same_bits(s[:, :rows], s2[:, :rows], "fp8 scales")
        q, s = dg.dg_gated_act_int8(pre, act=act)
        q2, s2 = dg.dg_quantize_int8_per_token(wide)
        same_bits(q, q2, "int8 codes")
        same_bits(s, s2, "int8 scales")
        # the gradient
        dh = rand(rng, rows, n, dtype=dtype)
        dpre = dg.dg_gated_act_grad(dh, pre, act=act)
        hp, hd = host(pre), host(dh)
        a, b = OF.act_slope_terms(hp[:, :n], act)
        z = np.abs(OF._arg(hp[:, :n], act)[0])
        tol = np.concatenate((np.abs(hd * hp[:, n:]) * (np.abs(a) + np.abs(b)), np.abs(hd * OF.act_value(hp[:, :n], act))), 1)
        near(dpre, OF.gated_grad(hd, hp, act), tol * np.concatenate((12 + 6 * z, 12 + 6 * z), 1) * EPS, dtype, "gradient")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_act_limits(act):
    """Values whose exponentials leave fp32, infinities and NaN: the formula's limits, and nothing else's."""
    say("act limits", act)
    g = torch.tensor([100.0, -100.0, 3e38, -3e38, 1e20, -1e20, float("inf"), float("nan"), 1e-40, 0.0, 2.0, -87.0, -2.0, 88.0, 5.0, 6.0],
                     device=device())
    pre = torch.cat((g, torch.ones_like(g)))[None].contiguous()
    h = dg.dg_gated_act(pre, act=act)[0]
    assert torch.equal(h[[0, 2, 4, 13]], g[[0, 2, 4, 13]]) and torch.all(h[[1, 3, 5]] == 0) and h[6] == float("inf")
    assert torch.isnan(h[7]) and torch.isfinite(h[8:]).all() and h[9] == 0
    d = dg.dg_gated_act_grad(torch.ones_like(g)[None].contiguous(), pre, act=act)[0]
    slope = d[:16]
    assert torch.all(slope[[0, 2, 4, 6, 13]] == 1) and torch.all(slope[[1, 3, 5]] == 0) and torch.isnan(slope[7])
    assert slope[9] == 0.5 and torch.isfinite(slope[8:]).all()
    same_bits(d[16:], h, "the other half's gradient is the activation")
    # a NaN stays in its row
    pre = torch.randn((4, 256), device=device())
    clean = dg.dg_gated_act_int8(pre, act=act)
    pre[2, 5] = float("nan")
    q, s = dg.dg_gated_act_int8(pre, act=act)
    assert torch.isnan(s[2]) and torch.equal(s[[0, 1, 3]], clean[1][[0, 1, 3]]) and torch.equal(q[[0, 1, 3]], clean[0][[0, 1, 3]])


def test_act_of_zero_rows():
    say("act of zeros and of none")
    pre = torch.zeros((6, 512), device=device())
    q, s = dg.dg_gated_act_fp8(pre)
    assert torch.all(q == 0) and torch.all(s[:, :6] == 1)
    q, s = dg.dg_gated_act_int8(pre)
    assert torch.all(q == 0) and torch.all(s == 1)
    for f in (dg.dg_gated_act, dg.dg_gated_act_fp8, dg.dg_gated_act_int8):
        f(pre[:0])
    assert dg.dg_gated_act_grad(pre[:0, :256], pre[:0]).shape == (0, 512)
    dg.dg_gated_act_grad_fp8(pre[:0, :256], pre[:0])


@pytest.mark.parametrize("form", ["same", "fp8", "int8"])
@pytest.mark.parametrize("n", [80, 1024])
def test_act_masks(form, n):
    """Rows that are not computed stay as they were; the others have the bits of a call without a mask."""
    rng = np.random.default_rng(n)
    g, m = 5, 37
    pre = rand(rng, g, m, 2 * n, dtype=BF16)
    counts = torch.tensor([0, 37, 1, -3, 99], dtype=torch.int32, device=device())
    flat = pre.view(g * m, 2 * n)
    say("act masks", form, n)
    mi = torch.tensor(([3] * 20 + [-1] * 17) * g, dtype=torch.int32, device=device())
    keep_m = torch.arange(m, device=device())[None, :] < counts[:, None]

    def check(got, full, keep, untouched):
        full = full.view(got.shape)
        same_bits(got[keep], full[keep])
        assert torch.all(got[~keep] == untouched)

    if form == "same":
        full = dg.dg_gated_act(flat)
        check(dg.dg_gated_act(pre, h=torch.full((g, m, n), 7.0, dtype=BF16, device=device()), masked_m=counts), full, keep_m, 7.0)
        check(dg.dg_gated_act(flat, h=torch.full((g * m, n), 7.0, dtype=BF16, device=device()), m_indices=mi), full, mi >= 0, 7.0)
    elif form == "int8":
        fq, fs = dg.dg_gated_act_int8(flat)
        q, s = torch.full((g, m, n), 7, dtype=torch.int8, device=device()), torch.full((g, m), 7.0, device=device())
        dg.dg_gated_act_int8(pre, q=q, s=s, masked_m=counts)
        check(q, fq, keep_m, 7)
        check(s, fs, keep_m, 7.0)
        q, s = torch.full((g * m, n), 7, dtype=torch.int8, device=device()), torch.full((g * m,), 7.0, device=device())
        dg.dg_gated_act_int8(flat, q=q, s=s, m_indices=mi)
        check(q, fq, mi >= 0, 7)
        check(s, fs, mi >= 0, 7.0)
    else:
        fq, fs = dg.dg_gated_act_fp8(flat)
        kb = -(-n // 128)
        q, s = torch.full((g, m, n), 7, dtype=torch.uint8, device=device()), torch.full((g, kb, 40), 7.0, device=device())
        dg.dg_gated_act_fp8(pre, q=q, s=s, masked_m=counts)
        check(q, fq, keep_m, 7)
        check(s[..., :m].transpose(1, 2).contiguous(), fs[:, :g * m].t().contiguous(), keep_m, 7.0)
        assert torch.all(s[..., m:] == 7.0)
        q, s = torch.full((g * m, n), 7, dtype=torch.uint8, device=device()), torch.full((kb, 188), 7.0, device=device())
        dg.dg_gated_act_fp8(flat, q=q, s=s, m_indices=mi)
        check(q, fq, mi >= 0, 7)
        check(s[:, :g * m].t().contiguous(), fs[:, :g * m].t().contiguous(), mi >= 0, 7.0)
        assert torch.all(s[:, g * m:] == 7.0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,n", [(16, 128), (112, 256), (128, 128), (272, 384), (400, 1024)])
def test_act_grad_fp8(rows, n, act):
    """The bits of the fp32 gradient followed by the library's quantizers, in all three layouts and each alone."""
    rng = np.random.default_rng(rows + n)
    for dtype in DTYPES:
        say("act grad fp8", rows, n, act, dtype)
        pre, dh = rand(rng, rows, 2 * n, dtype=dtype, scale=1.5), rand(rng, rows, n, dtype=dtype)
        dh[:, 3] = 0.0       # a column and a row of zeros
        dh[5] = 0.0
        wide = dg.dg_gated_act_grad(dh.float(), pre.float(), act=act)
        h = dg.dg_gated_act(pre.float(), act=act)
        got = dg.dg_gated_act_grad_fp8(dh, pre, act=act)
        want = (*dg.dg_quantize_per_token_group(wide), *dg.dg_quantize_per_channel_group(wide),
                *dg.dg_quantize_per_channel_group(h))
        for i, (a, b) in enumerate(zip(got, want)):
            same_bits(a, b[..., :a.shape[-1]], f"output {i}")
        for wanted in ((True, False, False), (False, True, False), (False, False, True)):
            part = dg.dg_gated_act_grad_fp8(dh, pre, act=act, rows_wanted=wanted[0], columns_wanted=wanted[1], h_wanted=wanted[2])
            for i in range(6):
                assert (part[i] is not None) == wanted[i // 2]
                if part[i] is not None:
                    same_bits(part[i], got[i], f"output {i} alone")


# ---- residual norms -------------------------------------------------------------------------------

def norm_inputs(rng, rows, hidden, dtype, res, gates, post, weights):
    a = dict(x=rand(rng, rows, hidden, dtype=dtype), residual=rand(rng, rows, hidden, dtype=res, scale=2.0),
             weight=rand(rng, hidden, scale=0.2) + 1 if weights else None,
             gate=rand(rng, gates, hidden, dtype=dtype) if gates else None, post_norm=post,
             post_weight=rand(rng, hidden, scale=0.2) + 1 if post and weights else None, scale=0.75, eps=1e-5)
    if rows > 2:
        a["x"][1] *= 100
        a["x"][2] = 0
    return a


def on_host(a):
    return {k: host(v) if isinstance(v, torch.Tensor) else v for k, v in a.items()}


def norm_tolerances(a, want_sum):
    """Of the sum and of y, without the rounding to their types."""
    h = on_host(a)
    size = np.abs(h["residual"])
    if h["x"] is not None:
        size = size + np.abs(want_sum - h["residual"])
    rho = 1 / np.sqrt((want_sum ** 2).mean(1, keepdims=True) + h["eps"])
    w = 1.0 if h["weight"] is None else np.abs(h["weight"])
    y = np.abs(want_sum) * rho * w
    # the sum's rounding errors move its rms too, by at most their own rms
    moved = np.sqrt((size ** 2).mean(1, keepdims=True)) * rho
    return 80 * EPS * size, 80 * EPS * (y * (1 + moved) + rho * w * size)


SHAPES = [(1, 16), (5, 64), (7, 144), (66, 512), (9, 528), (33, 1024), (6, 2064), (12, 4096), (5, 4112), (7, 8192), (3, 8208),
          (4, 16384)]


@pytest.mark.parametrize("rows,hidden", SHAPES)
@pytest.mark.parametrize("post,gates,weights", [(False, 0, True), (True, 1, True), (True, -1, True), (False, 1, False), (True, 0, False)])
def test_norm(rows, hidden, post, gates, weights):
    rng = np.random.default_rng(rows * hidden + gates)
    for dtype, res in ((F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)):
        say("norm", rows, hidden, post, gates, weights, dtype, res)
        a = norm_inputs(rng, rows, hidden, dtype, res, rows if gates < 0 else gates, post, weights)
        total, y = dg.dg_residual_norm(**a)
        want_sum, want_y = OF.residual_norm(**on_host(a))
        tol_sum, tol_y = norm_tolerances(a, want_sum)
        near(total, want_sum, tol_sum, res, "sum")
        near(y, want_y, tol_y, dtype, "y")
        # quantized, from the fp32 values
        wide = {k: v.float() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
        exact = dg.dg_residual_norm(**wide)[1]
        t8, q, s = dg.dg_residual_norm_fp8(**a)
        q2, s2 = dg.dg_quantize_per_token_group(exact)
        same_bits(t8, total, "sum beside fp8")
        same_bits(q, q2, "fp8 codes")
        same_bits(s[:, :rows], s2[:, :rows], "fp8 scales")
        t8, q, s = dg.dg_residual_norm_int8(**a)
        q2, s2 = dg.dg_quantize_int8_per_token(exact)
        same_bits(t8, total, "sum beside int8")
        same_bits(q, q2, "int8 codes")
        same_bits(s, s2, "int8 scales")
        # in place
        mine = a["residual"].clone()
        t3, y3 = dg.dg_residual_norm(**{**a, "residual": mine}, sum=mine)
        assert t3.data_ptr() == mine.data_ptr()
        same_bits(mine, total, "in place")
        same_bits(y3, y, "y in place")


@pytest.mark.parametrize("rows,hidden", [(1, 16), (5, 528), (40, 7168)])
def test_norm_alone(rows, hidden):
    rng = np.random.default_rng(hidden)
    for res in DTYPES:
        say("norm alone", rows, hidden, res)
        r, w = rand(rng, rows, hidden, dtype=res), rand(rng, hidden, scale=0.2) + 1
        total, y = dg.dg_residual_norm(None, r, w)
        assert total is r
        a = dict(x=None, residual=r, weight=w, eps=1e-6)
        near(y, OF.residual_norm(**on_host(a))[1], norm_tolerances(a, host(r))[1], res)
        _, q, s = dg.dg_residual_norm_fp8(None, r, w)
        q2, s2 = dg.dg_quantize_per_token_group(dg.dg_residual_norm(None, r.float(), w)[1])
        same_bits(q, q2)
        same_bits(s[:, :rows], s2[:, :rows])
        dy, ds = rand(rng, rows, hidden, dtype=res), rand(rng, rows, hidden, dtype=res)
        got = dg.dg_residual_norm_grad(dy, ds, None, r, w)
        want = OF.residual_norm_grad(host(dy), host(ds), None, host(r), host(w))
        assert got.dx is None and got.dgate is None and got.dpost_weight is None
        near(got.dresidual, want["dresidual"], 80 * EPS * want["size_dresidual"], res, "dresidual")
        near(got.dweight, want["dweight"], 200 * EPS * want["size_dweight"], F32, "dweight")
    # a wider residual stream than the block's type
    r = rand(rng, rows, hidden)
    _, y = dg.dg_residual_norm(None, r, dtype=BF16)
    near(y, OF.residual_norm(None, host(r), None)[1], norm_tolerances(dict(x=None, residual=r, weight=None, eps=1e-6), host(r))[1], BF16)


@pytest.mark.parametrize("rows,hidden,gates", [(1, 16, 1), (5, 64, 5), (12, 144, 4), (66, 512, 3), (2500, 64, 1), (2500, 64, 5),
                                               (2499, 128, 833), (2500, 48, 1250), (3000, 32, 3000), (1050, 1024, 7),
                                               (1030, 2064, 2), (64, 4096, 0), (1060, 4112, 1), (600, 8192, 3), (520, 8208, 2),
                                               (300, 16384, 1), (1280, 64, 64), (1300, 1040, 20), (1000, 528, 100)])
@pytest.mark.parametrize("post", [False, True])
def test_norm_grad(rows, hidden, gates, post):
    rng = np.random.default_rng(rows + hidden + gates)
    types = ((F32, F32), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32)) if rows * hidden < 1 << 20 else ((BF16, F32), (F32, F32))
    for n, (dtype, res) in enumerate(types):
        say("norm grad", rows, hidden, gates, post, dtype, res)
        weights = n != 2
        a = norm_inputs(rng, rows, hidden, dtype, res, gates, post, weights)
        del a["residual"]
        x = a.pop("x")
        s, dy = rand(rng, rows, hidden, dtype=res, scale=2.0), rand(rng, rows, hidden, dtype=dtype)
        ds = rand(rng, rows, hidden, dtype=res) if n != 1 else None
        got = dg.dg_residual_norm_grad(dy, ds, x, s, **a)
        want = OF.residual_norm_grad(host(dy), None if ds is None else host(ds), host(x), host(s), **on_host(a))
        near(got.dresidual, want["dresidual"], 80 * EPS * want["size_dresidual"], res, "dresidual")
        near(got.dx, want["dx"], 160 * EPS * want["size_dx"], dtype, "dx")
        # the terms' own errors (80 eps) and those of adding them
        for name, t in (("dweight", F32), ("dgate", dtype), ("dpost_weight", F32)):
            g = getattr(got, name)
            assert (g is None) == (want[name] is None)
            if g is not None:
                near(g, want[name], (80 + 200) * EPS * want["size_" + name], t, name)
        again = dg.dg_residual_norm_grad(dy, ds, x, s, **a)
        for u, v in zip(got, again):
            if u is not None:
                same_bits(u, v, "the same bits again")
        if ds is not None:
            mine = ds.clone()
            inplace = dg.dg_residual_norm_grad(dy, mine, x, s, dresidual=mine, **a)
            same_bits(mine, got.dresidual, "in place")
            same_bits(inplace.dx, got.dx, "dx in place")


def test_norm_of_no_rows():
    d = device()
    say("norm of no rows")
    x = torch.zeros((0, 64), dtype=BF16, device=d)
    w, gate = torch.ones(64, device=d), torch.ones((1, 64), dtype=BF16, device=d)
    dg.dg_residual_norm(x, x, w)
    got = dg.dg_residual_norm_grad(x, x, x, x, w, gate=gate[0], post_norm=True, post_weight=w)
    assert torch.all(got.dweight == 0) and torch.all(got.dpost_weight == 0) and torch.all(got.dgate == 0)


def test_norm_nan_stays_in_its_row():
    d = device()
    say("norm nan")
    x, r = torch.randn((5, 256), device=d), torch.randn((5, 256), device=d)
    clean = dg.dg_residual_norm(x, r, post_norm=True)
    x[3, 9] = float("nan")
    total, y = dg.dg_residual_norm(x, r, post_norm=True)
    assert torch.isnan(y[3]).all() and torch.isnan(total[3]).all()
    for i in (0, 1, 2, 4):
        same_bits(y[i], clean[1][i])


# ---- streams, graphs ------------------------------------------------------------------------------

def test_streams_and_graphs():
    """The calls on a side stream and captured, replayed on new inputs, against eager calls."""
    d = device()
    say("streams and graphs")
    rng = np.random.default_rng(3)
    x, r, w = rand(rng, 70, 1024, dtype=BF16), rand(rng, 70, 1024), rand(rng, 1024)
    gate, dy, ds = rand(rng, 1, 1024, dtype=BF16), rand(rng, 70, 1024, dtype=BF16), rand(rng, 70, 1024)
    pre, dh = rand(rng, 80, 512, dtype=BF16), rand(rng, 80, 256, dtype=BF16)

    def step():
        total, q, s = dg.dg_residual_norm_fp8(x, r, w, gate=gate, post_norm=True)
        grad = dg.dg_residual_norm_grad(dy, ds, x, r, w, gate=gate, post_norm=True, post_weight=w)
        return [total, q, s[:, :70], *grad, dg.dg_gated_act(pre), *dg.dg_gated_act_int8(pre), *dg.dg_gated_act_grad_fp8(dh, pre)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        same_bits(a, b, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in range(3):
        for t in (x, dy, ds, pre, dh):
            t.copy_(rand(rng, *t.shape, dtype=t.dtype))
        graph.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same_bits(a, b, f"replay {n}")
