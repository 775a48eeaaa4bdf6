"""Expert routing, expert row layout, dispatch and combine on the GPU against the plain 64-bit
implementations.

Tolerances, from the arithmetic: a routing weight is an exponential (2 ulp of its argument's rounding and
1 of its own), a quotient, a sum of up to 64 such terms and a product, each rounded to 24 bits - below
80 * 2^-24 = 4.8e-6 of its value.  A combined value is a chain of top_k fused multiply-adds (each within
2^-24 of the sum of magnitudes so far) and one rounding to the output's type (2^-24, 2^-8, 2^-11 relative,
2^-25 absolute for fp16 near zero).
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
OUT_REL = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}   # half a unit of 24, 8, 11 significant bits
OUT_ABS = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -25}
W_TOL = 80 * 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def dev(x, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(x))
    return t.to(device=device(), dtype=dtype or t.dtype)


# ---- routing --------------------------------------------------------------------------------------

def check_choice(x, ids, bias, g, tg, top, score, top_k):
    """Every token's ids against its choice values in 64 bits: exactly where the values are further
    apart than their fp32 rounding (4 ulp of values up to 2), else any order among the close ones."""
    close = 4 * 2.0 ** -23
    for i in range(x.shape[0]):
        v = oracle.moe.choice_values(x[i], score, bias, g, top)
        mine = ids[i][ids[i] >= 0]
        assert np.unique(mine).size == mine.size and np.all(ids[i][mine.size:] == -1)
        if g > 1:
            # a group judged within rounding of the last kept one may stand in for it
            per = v.reshape(g, -1)
            sums = np.array([np.sort(r[r != -np.inf])[::-1][:top].sum() if (r != -np.inf).any() else -np.inf for r in per])
            order = np.sort(sums)[::-1]
            used = np.unique(mine // per.shape[1])
            assert used.size <= tg and np.all(sums[used] >= order[tg - 1] - 2 * close)
            if order[min(tg, g - 1)] < order[tg - 1] - 2 * close or tg == g:
                keep = oracle.moe.kept_groups(v, g, tg, top)
            else:
                continue
            v = np.where(keep, v, -np.inf)
        want = np.sort(v)[::-1][:top_k]
        assert mine.size == (want != -np.inf).sum()
        assert np.all(np.abs(v[mine] - want[:mine.size]) <= close)


ROUTES = [  # experts, top_k, groups, topk_groups, group_top, bias
    (1, 1, 1, 1, 1, False), (3, 3, 1, 1, 1, True), (64, 6, 1, 1, 1, False), (65, 8, 1, 1, 1, True), (100, 7, 4, 3, 2, True),
    (128, 64, 1, 1, 1, False), (160, 6, 8, 3, 1, False), (256, 8, 8, 4, 2, True), (256, 8, 64, 9, 1, False),
    (300, 5, 3, 1, 2, False), (512, 8, 16, 16, 2, True), (1000, 10, 5, 2, 1, True), (1024, 16, 1, 1, 1, False)]


@pytest.mark.parametrize("experts,top_k,g,tg,top,bias", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(experts, top_k, g, tg, top, bias, score):
    rng = np.random.default_rng(experts * 7 + top_k)
    for n, (tokens, dtype) in enumerate([(1, BF16), (5, F16), (67, F32), (66, BF16)]):
        say("route", experts, top_k, g, tg, top, bias, score, tokens, dtype)
        x = dev(rng.standard_normal((tokens, experts)) * 2, dtype)
        if tokens > 5:   # some experts off, a row with a few left, a row with none
            x = torch.where(dev(rng.random((tokens, experts)) < 0.1), torch.full_like(x, -np.inf), x)
            x[3, 2:] = -np.inf
            x[4] = -np.inf
        b = dev(rng.standard_normal(experts) * 0.05, F32) if bias else None
        renorm, scale = n % 2 == 0, (1.0, 2.5)[n % 2]
        ids, w = dg.dg_moe_route(x, top_k, bias=b, num_groups=g, topk_groups=tg, group_top=top, score=score,
                                 renormalize=renorm, scale=scale)
        again = dg.dg_moe_route(x, top_k, bias=b, num_groups=g, topk_groups=tg, group_top=top, score=score,
                                renormalize=renorm, scale=scale)
        assert torch.equal(ids, again[0]) and torch.equal(w, again[1])
        hx, hi = host(x), ids.cpu().numpy()
        check_choice(hx, hi, None if b is None else host(b), g, tg, top, score, top_k)
        want = oracle.moe.weights_of(hx, hi, score, renorm, scale)
        np.testing.assert_allclose(host(w), want, rtol=W_TOL, atol=1e-37)
        # the gradient of the weights
        dw = dev(rng.standard_normal((tokens, top_k)), F32)
        dx = dg.dg_moe_route_grad(dw, x, ids, score=score, renormalize=renorm, scale=scale)
        want = oracle.moe.route_grad(host(dw), hx, hi, score, renorm, scale)
        # each term is a product of rounded factors; differences of terms as large as scale * s * max|dw|
        size = scale * np.abs(host(dw)).max() * 2
        assert np.all(np.abs(host(dx) - want) <= OUT_REL[dtype] * np.abs(want) + OUT_ABS[dtype] + 2 * W_TOL * size)


def test_route_ties_and_special_values():
    d = device()
    say("route ties and special values")
    x = torch.zeros((6, 200), device=d)
    x[0, 150] = 1.0
    x[1, ::2] = -0.0                     # -0 and +0 are equal
    x[2] = float("nan")
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    x[5] = -1000.0                       # sigmoid underflows
    ids, w = dg.dg_moe_route(x, 4, score="softmax")
    assert ids.tolist() == [[150, 0, 1, 2], [0, 1, 2, 3], [-1] * 4, [0, 1, 2, 3], [9, 0, 1, 2], [0, 1, 2, 3]]
    assert torch.all(w[2] == 0) and torch.isnan(w[3]).all() and torch.allclose(w[1], torch.full((4,), 0.25, device=d))
    ids, w = dg.dg_moe_route(x, 4, score="sigmoid")
    assert ids.tolist()[5] == [0, 1, 2, 3] and torch.all(w[5] == 0)    # no score left: weight 0
    assert torch.isnan(w[3]).all() and not torch.isnan(w[4]).any()
    # many equal logits across registers and lanes, and among groups
    q = torch.randint(0, 3, (50, 256), device=d, generator=torch.Generator(device=d).manual_seed(1)).float()
    ids, _ = dg.dg_moe_route(q, 8, num_groups=8, topk_groups=3)
    want, _ = oracle.moe.route(host(q), 8, num_groups=8, topk_groups=3)
    assert np.array_equal(ids.cpu().numpy(), want)
    # a bias of -inf switches an expert off, one of NaN marks the token
    bias = torch.zeros(200, device=d)
    bias[0] = -float("inf")
    ids, w = dg.dg_moe_route(x[:2], 2, bias=bias, score="sigmoid")
    assert ids.tolist() == [[150, 1], [1, 2]]
    # fewer experts than places in the kept group
    ids, w = dg.dg_moe_route(torch.zeros((1, 8), device=d), 5, num_groups=4, topk_groups=2)
    assert ids.tolist() == [[0, 1, 2, 3, -1]] and w[0, 4] == 0


def test_route_strided_and_other_stream():
    d = device()
    say("route strided")
    wide = torch.randn((33, 205), device=d).to(BF16)
    view = wide[:, 3:70]                 # rows 205 elements apart, starting at an odd element
    ids, w = dg.dg_moe_route(view, 4)
    ids2, w2 = dg.dg_moe_route(view.contiguous(), 4)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    out = torch.full((33, 80), 7.0, dtype=BF16, device=d)
    dw = torch.randn((33, 4), device=d)
    got = dg.dg_moe_route_grad(dw, view, ids, dlogits=out[:, 1:68])
    assert torch.equal(got, dg.dg_moe_route_grad(dw, view.contiguous(), ids))
    assert torch.all(out[:, 0] == 7) and torch.all(out[:, 68:] == 7)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids3, w3 = dg.dg_moe_route(view, 4)
        layout = dg.dg_moe_layout(ids3, 67)
        y = dg.dg_moe_combine(dg.dg_moe_dispatch(torch.ones((33, 32), device=d), layout), layout, weights=w3)
    s.synchronize()
    assert torch.equal(ids, ids3) and torch.equal(w, w3) and torch.allclose(y, torch.ones_like(y), atol=1e-6)
    for bad in (wide.t(), wide[0], wide.double(), wide.cpu()):
        with pytest.raises(ValueError):
            dg.dg_moe_route(bad, 1)
    with pytest.raises(dg.DGError):
        dg.dg_moe_route(view, 68)
    ids, w = dg.dg_moe_route(torch.empty((0, 16), device=d), 2)
    assert ids.shape == (0, 2) and dg.dg_moe_route_grad(w, torch.empty((0, 16), device=d), ids).shape == (0, 16)


def test_route_grad_of_odd_ids():
    """Ids outside the experts count as not chosen; a token with none gets zeros."""
    d = device()
    say("route grad of odd ids")
    x = torch.randn((3, 10), device=d)
    ids = torch.tensor([[1, -1], [10, 2 ** 30], [-5, 4]], dtype=torch.int32, device=d)
    dw = torch.ones((3, 2), device=d)
    for score in ("softmax", "sigmoid"):
        for renorm in (False, True):
            dx = dg.dg_moe_route_grad(dw, x, ids, score=score, renormalize=renorm)
            clean = np.where((ids.cpu().numpy() < 0) | (ids.cpu().numpy() >= 10), -1, ids.cpu().numpy())
            want = oracle.moe.route_grad(host(dw), host(x), clean, score, renorm, 1.0)
            assert np.all(np.abs(host(dx) - want) <= 4 * W_TOL)
            assert torch.all(dx[1] == 0)


# ---- layout ---------------------------------------------------------------------------------------

def make_ids(rng, tokens, top_k, experts, skew=0.0, dropped=0.1):
    p = np.arange(1, experts + 1, dtype=np.float64) ** -skew
    gumbel = rng.gumbel(size=(tokens, experts)) + np.log(p)
    ids = np.argsort(-gumbel, axis=1)[:, :top_k].astype(np.int32)
    if top_k > experts:
        ids = np.concatenate([ids, np.full((tokens, top_k - experts), -1, np.int32)], axis=1)
    ids[rng.random((tokens, top_k)) < dropped] = -1
    return ids


LAYOUTS = [  # tokens, top_k, experts, rows_per_expert, skew
    (0, 2, 8, 0, 0.0), (1, 1, 1, 0, 0.0), (1, 8, 256, 0, 0.0), (3, 2, 5, 4, 0.0), (128, 1, 1, 0, 0.0), (129, 1, 1, 0, 0.0),
    (4095, 1, 7, 0, 1.0), (4097, 1, 3, 0, 0.0), (1024, 4, 64, 0, 1.1), (1025, 4, 64, 96, 1.1), (2731, 3, 1024, 0, 0.5),
    (5000, 6, 1000, 8, 0.0), (700, 64, 129, 0, 0.3), (0, 1, 3, 5, 0.0), (45000, 6, 37, 0, 0.8), (70001, 5, 300, 0, 0.2)]


@pytest.mark.parametrize("tokens,top_k,experts,per,skew", LAYOUTS)
def test_layout(tokens, top_k, experts, per, skew):
    rng = np.random.default_rng(tokens + experts)
    ids = make_ids(rng, tokens, top_k, experts, skew)
    if ids.size > 4:   # whatever is not an expert gets no row
        ids.reshape(-1)[1] = experts
        ids.reshape(-1)[3] = 2 ** 31 - 1
        ids.reshape(-1)[ids.size // 2] = -2 ** 31
    say("layout", tokens, top_k, experts, per)
    lay = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    again = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    rows, sources, m_indices, counts = oracle.moe.layout(ids, experts, per)
    assert np.array_equal(lay.rows.cpu().numpy(), rows) and np.array_equal(lay.counts.cpu().numpy(), counts)
    n = len(sources)
    got = lay.sources.cpu().numpy()
    assert np.array_equal(got[:n], sources) and np.all(got[n:] == -1) and lay.rows_total == got.size
    if per:
        assert lay.m_indices is None and n == got.size
    else:
        mi = lay.m_indices.cpu().numpy()
        assert np.array_equal(mi[:n], m_indices) and np.all(mi[n:] == -1)
    assert torch.equal(lay.sources, again.sources) and torch.equal(lay.rows, again.rows)


def test_layout_larger_capacity_and_refusals():
    ids = dev(np.array([[0, 2], [2, 1]], dtype=np.int32))
    say("layout capacity")
    lay = dg.dg_moe_layout(ids, 4, rows_total=1280)
    assert lay.rows.tolist() == [[0, 256], [257, 128]] and lay.m_indices[384:].tolist() == [-1] * 896
    with pytest.raises(dg.DGError):
        dg.dg_moe_layout(ids, 4, rows_total=256)
    with pytest.raises(ValueError):
        dg.dg_moe_layout(ids.long(), 4)
    with pytest.raises(ValueError):
        dg.dg_moe_layout(ids.t(), 4)
    x = torch.zeros((2, 64), device=device())
    with pytest.raises(dg.DGError):
        dg.dg_moe_dispatch(torch.zeros((2, 40), device=device()), lay)
    with pytest.raises(ValueError):
        dg.dg_moe_dispatch(x[:1], lay)
    with pytest.raises(ValueError):
        dg.dg_moe_combine(torch.zeros((128, 64), device=device()), lay)
    with pytest.raises(ValueError):
        dg.dg_moe_combine(dg.dg_moe_dispatch(x, lay), lay, weights=torch.ones((2, 3), device=device()))


# ---- dispatch and combine -------------------------------------------------------------------------

ROWS = [  # tokens, top_k, experts, rows_per_expert, hidden
    (1, 1, 1, 0, 16), (1, 8, 64, 0, 7168), (7, 2, 3, 4, 48), (33, 3, 5, 0, 128), (40, 2, 4, 16, 400), (150, 4, 9, 0, 1040),
    (21, 11, 16, 0, 2064), (90, 8, 32, 24, 4112), (300, 2, 130, 0, 272), (0, 2, 4, 8, 64)]


@pytest.mark.parametrize("tokens,top_k,experts,per,hidden", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dispatch(tokens, top_k, experts, per, hidden, dtype):
    rng = np.random.default_rng(hidden + tokens)
    ids = make_ids(rng, tokens, top_k, experts, 0.5)
    x = dev(rng.standard_normal((tokens, hidden)) * 3, dtype)
    if tokens > 5:
        x[2] = 0
        x[3] *= 1000
    say("dispatch", tokens, top_k, experts, per, hidden, dtype)
    lay = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    sources = lay.sources.cpu().numpy()
    owned = sources >= 0 if per else lay.m_indices.cpu().numpy() >= 0     # rows that are written
    lead = lay.lead()
    xr = oracle.moe.dispatch(x.float().cpu().numpy(), sources, top_k)
    # copy: written rows exact, the others as they were
    out = torch.full((*lead, hidden), 9.0, dtype=dtype, device=device())
    dg.dg_moe_dispatch(x, lay, out=out)
    got = out.view(-1, hidden).float().cpu().numpy()
    assert np.array_equal(got[owned], xr[owned]) and np.all(got[~owned] == 9)
    # int8: the codes and scales of the per-row quantizer
    q = torch.full((*lead, hidden), 99, dtype=torch.int8, device=device())
    s = torch.full(lead, 5.0, device=device())
    dg.dg_moe_dispatch_int8(x, lay, q=q, s=s)
    wq, ws = oracle.int8.quantize(xr)
    gq, gs = q.view(-1, hidden).cpu().numpy(), s.view(-1).cpu().numpy()
    assert np.array_equal(gq[owned], wq[owned]) and np.array_equal(gs[owned], ws[owned])
    assert np.all(gq[~owned] == 99) and np.all(gs[~owned] == 5)
    # FP8: the codes and scales of the per-token-group quantizer
    kb = -(-hidden // 128)
    ld = dg.dg_get_scale_ld(lead[-1]) + 4
    q = torch.full((*lead, hidden), 0x55, dtype=torch.uint8, device=device())
    sa = torch.full((*lead[:-1], kb, ld), 5.0, device=device())
    dg.dg_moe_dispatch_fp8(x, lay, q=q, sa=sa)
    wq, ws = oracle.quant.quantize_per_token_group(xr)
    gq = q.view(-1, hidden).cpu().numpy()
    gs = sa.cpu().numpy()[..., :lead[-1]].swapaxes(-1, -2).reshape(-1, kb)
    assert np.array_equal(gq[owned], wq[owned]) and np.array_equal(gs[owned], ws[owned])
    assert np.all(gq[~owned] == 0x55) and np.all(gs[~owned] == 5) and torch.all(sa[..., lead[-1]:] == 5)


@pytest.mark.parametrize("tokens,top_k,experts,per,hidden", [(4097, 8, 20, 0, 1040), (700, 6, 9, 0, 8400), (3000, 3, 7, 999, 4112),
                                                              (8200, 8, 20, 0, 1040), (1500, 7, 9, 0, 8400),
                                                              (6000, 3, 7, 1999, 4112)])
def test_dispatch_of_many_scales(tokens, top_k, experts, per, hidden):
    """With its workspace the FP8 form moves the scales in a launch of their own: the same bits as without."""
    rng = np.random.default_rng(tokens)
    ids = make_ids(rng, tokens, top_k, experts, 0.5)
    x = dev(rng.standard_normal((tokens, hidden)), BF16)
    say("dispatch of many scales", tokens, top_k, experts, per, hidden)
    lay = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    need = dg.dg_moe_dispatch_fp8_workspace_size(tokens, top_k, hidden)
    assert need > 0 or tokens * top_k * -(-hidden // 128) < 1 << 19
    lead, kb = lay.lead(), -(-hidden // 128)
    got = []
    for ws in (torch.full((need,), 0xFF, dtype=torch.uint8, device=device()), torch.empty(0, dtype=torch.uint8, device=device())):
        q = torch.full((*lead, hidden), 0x55, dtype=torch.uint8, device=device())
        sa = torch.full((*lead[:-1], kb, dg.dg_get_scale_ld(lead[-1])), 5.0, device=device())
        got.append(dg.dg_moe_dispatch_fp8(x, lay, q=q, sa=sa, workspace=ws))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    wq, ws = dg.dg_quantize_per_token_group(x)
    for t, k in ((0, 0), (tokens - 1, top_k - 1), (tokens // 2, 1)):
        r = int(lay.rows[t, k])
        if r >= 0:
            sa = got[0][1].view(-1, kb, got[0][1].shape[-1])
            g, at = (r // per, r % per) if per else (0, r)
            assert torch.equal(sa[g, :, at], ws[:, t]) and torch.equal(got[0][0].view(-1, hidden)[r], wq[t])


@pytest.mark.parametrize("tokens,top_k,experts,per,hidden", ROWS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_and_gradients(tokens, top_k, experts, per, hidden, dtype):
    rng = np.random.default_rng(hidden * 3 + tokens)
    ids = make_ids(rng, tokens, top_k, experts, 0.5)
    say("combine", tokens, top_k, experts, per, hidden, dtype)
    lay = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    rows, sources = lay.rows.cpu().numpy(), lay.sources.cpu().numpy()
    out = dev(rng.standard_normal((lay.rows_total, hidden)), dtype)
    out[dev(sources < 0)] = float("nan")     # rows of no token are never read
    w = dev(rng.random((tokens, top_k)), F32)
    w = torch.where(lay.rows < 0, torch.full_like(w, float("nan")), w)   # nor the weights of entries without one
    hout, hw = host(out), host(w)
    size = oracle.moe.combine(np.abs(hout), rows, np.abs(hw))
    chain = (top_k + 1) * 2.0 ** -24
    y = dg.dg_moe_combine(out.view(*lay.lead(), hidden), lay, weights=w)
    want = oracle.moe.combine(hout, rows, hw)
    assert np.all(np.abs(host(y) - want) <= OUT_REL[dtype] * np.abs(want) + OUT_ABS[dtype] + 2 * chain * size)
    # without weights: the gradient of dispatch
    y1 = dg.dg_moe_combine(out, lay)
    want = oracle.moe.combine(hout, rows)
    size1 = oracle.moe.combine(np.abs(hout), rows)
    assert np.all(np.abs(host(y1) - want) <= OUT_REL[dtype] * np.abs(want) + OUT_ABS[dtype] + 2 * chain * size1)
    # gradients
    dy = dev(rng.standard_normal((tokens, hidden)), dtype)
    dout = torch.full((lay.rows_total, hidden), 9.0, dtype=dtype, device=device())
    dg.dg_moe_combine_grad(dy, out, lay, w, dout=dout)
    dout2, dw = dg.dg_moe_combine_grad(dy, out, lay, w, dout=dout.clone())
    assert torch.equal(dout, dout2)
    want_out, want_w = oracle.moe.combine_grad(host(dy), np.nan_to_num(hout), rows, hw)
    owned = sources >= 0 if per else lay.m_indices.cpu().numpy() >= 0
    got = host(dout)
    near = (OUT_REL[dtype] + 2.0 ** -23) * np.abs(want_out) + OUT_ABS[dtype]
    assert np.all(np.abs(got - want_out)[owned] <= near[owned]) and np.all(got[~owned] == 9)
    _, mag = oracle.moe.combine_grad(np.abs(host(dy)), np.abs(np.nan_to_num(hout)), rows, hw)
    # a sum of `hidden` products in 32 bits, in lanes: within hidden / 64 + 16 roundings of its magnitude
    assert np.all(np.abs(host(dw) - want_w) <= (hidden / 64 + 16) * 2.0 ** -24 * mag + 1e-37)


def test_rows_outside_the_layout_are_ignored():
    """Rows arrays are the caller's: what is not a row of the layout counts as none."""
    d = device()
    say("rows outside the layout")
    ids = dev(np.array([[0, 1], [1, 0]], dtype=np.int32))
    lay = dg.dg_moe_layout(ids, 2)
    lay.rows[0, 1] = lay.rows_total
    lay.rows[1, 0] = 2 ** 31 - 1
    x = torch.ones((2, 64), device=d)
    out = dg.dg_moe_dispatch(x, lay, out=torch.full((lay.rows_total, 64), 3.0, device=d))
    assert torch.all(out[0] == 1) and torch.all(out[1] == 1) and torch.all(out[128:130] == 3)
    y = dg.dg_moe_combine(out, lay, weights=torch.ones((2, 2), device=d))
    assert torch.all(y == 1)


def test_rows_past_32_bit_offsets():
    """Row data of more than 2^32 bytes: dispatch and combine reach its end."""
    d = device()
    tokens, top_k, hidden = 9000, 8, 32768
    say("rows past 32-bit offsets", tokens, top_k, hidden)
    ids = torch.arange(top_k, dtype=torch.int32, device=d).repeat(tokens, 1)
    lay = dg.dg_moe_layout(ids, top_k)
    x = torch.randn((tokens, hidden), device=d).to(BF16)
    xr = dg.dg_moe_dispatch(x, lay)
    assert xr.numel() * 2 > 2 ** 32 and int(lay.rows[-1, -1]) * hidden * 2 > 2 ** 32
    for k in (0, top_k - 1):
        r = int(lay.rows[0, k])
        assert torch.equal(xr[r:r + tokens], x)
    y = dg.dg_moe_combine(xr, lay, weights=torch.full((tokens, top_k), 0.125, device=d))
    assert torch.equal(y, x)
    q, s = dg.dg_moe_dispatch_int8(x, lay)
    wq, ws = dg.dg_quantize_int8_per_token(x)
    r = int(lay.rows[0, top_k - 1])
    assert torch.equal(q[r:r + tokens], wq) and torch.equal(s[r:r + tokens], ws)


def test_moe_graph_replays_match_eager():
    """Route, layout, dispatch and combine captured in a HIP graph: every replay gives the eager bits."""
    d = device()
    tokens, experts, top_k, hidden = 600, 32, 8, 512
    say("moe graph")
    x = torch.empty((tokens, hidden), dtype=BF16, device=d)
    logits = torch.empty((tokens, experts), device=d)
    total = dg.dg_moe_layout_rows(tokens, top_k, experts)
    q, s = torch.zeros((total, hidden), dtype=torch.int8, device=d), torch.zeros(total, device=d)
    rows = torch.zeros((total, hidden), dtype=BF16, device=d)

    def step(x, logits, q, s, rows):
        ids, w = dg.dg_moe_route(logits, top_k, score="sigmoid")
        lay = dg.dg_moe_layout(ids, experts)
        dg.dg_moe_dispatch_int8(x, lay, q=q, s=s)
        dg.dg_moe_dispatch(x, lay, out=rows)
        return ids, w, lay.rows, lay.m_indices, dg.dg_moe_combine(rows, lay, weights=w)

    gen = torch.Generator(device=d)
    fill = lambda seed: (gen.manual_seed(seed), x.copy_(torch.randn((tokens, hidden), generator=gen, device=d)),
                         logits.copy_(torch.randn((tokens, experts), generator=gen, device=d)))
    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, logits, q, s, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, logits, q, s, rows)
    for seed in (1, 2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        q2, s2, rows2 = q.clone(), s.clone(), rows.clone()
        ref = step(x, logits, q2, s2, rows2)
        torch.cuda.synchronize()
        for a, b in zip((*out, q, s, rows), (*ref, q2, s2, rows2)):
            assert torch.equal(a, b), seed
