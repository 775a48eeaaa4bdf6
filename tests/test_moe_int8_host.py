"""Expert routing, expert rows and 8-bit integer GEMMs without a GPU: what the entry points refuse, the
sizes they report, and the plain implementations against facts outside them (torch's autograd and
elementary operations, differences, closed forms)."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
import oracle

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P, MIS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)   # never dereferenced: the checks come first


@pytest.fixture(scope="module")
def lib():
    return dg.lib()


def test_route_refusals(lib):
    def route(logits=P, dtype=0, ld=256, bias=None, t=4, e=256, k=8, g=8, tg=4, top=2, score=1, ids=P, w=P):
        return lib.dg_moe_route(logits, dtype, ld, bias, t, e, k, g, tg, top, score, 1, 1.0, ids, w, None)

    assert route(t=0, logits=None, ids=None, w=None) == OK
    for bad in (dict(t=-1), dict(e=0), dict(e=1025, ld=2000), dict(k=0), dict(k=65), dict(e=4, k=5, g=1, tg=1), dict(ld=255),
                dict(g=0), dict(g=65), dict(g=7), dict(tg=0), dict(tg=9), dict(top=0), dict(top=3), dict(score=2),
                dict(dtype=3), dict(dtype=-1), dict(logits=None), dict(ids=None), dict(w=None), dict(logits=MIS),
                dict(bias=MIS), dict(ids=MIS)):
        assert route(**bad) == INVALID, bad

    def grad(dw=P, logits=P, dtype=1, ld=64, ids=P, t=4, e=64, k=6, score=0, out=P, ldo=64):
        return lib.dg_moe_route_grad(dw, logits, dtype, ld, ids, t, e, k, score, 1, 1.0, out, ldo, None)

    assert grad(t=0, dw=None, logits=None, ids=None, out=None) == OK
    for bad in (dict(dw=None), dict(logits=None), dict(ids=None), dict(out=None), dict(ld=63), dict(ldo=63), dict(k=65),
                dict(e=2000, ld=2000, ldo=2000), dict(dtype=7), dict(score=-1), dict(dw=MIS), dict(dtype=0, logits=MIS)):
        assert grad(**bad) == INVALID, bad


def test_layout_refusals_and_sizes(lib):
    def layout(ids=P, t=4, k=2, e=8, per=0, total=1024, rows=P, src=P, mi=P, counts=P, ws=None, nws=0):
        return lib.dg_moe_layout(ids, t, k, e, per, total, rows, src, mi, counts, ws, nws, None)

    for bad in (dict(t=-1), dict(k=0), dict(k=65), dict(e=0), dict(e=1025), dict(per=-1), dict(total=896), dict(total=1000),
                dict(total=-128), dict(mi=None), dict(per=32, total=256), dict(per=32, total=255, mi=None), dict(ids=None),
                dict(rows=None), dict(src=None), dict(counts=None), dict(ids=MIS), dict(counts=MIS)):
        assert layout(**bad) == INVALID, bad
    need = lib.dg_moe_layout_workspace_size(1 << 20, 2, 8)
    assert need > 0
    big = dict(t=1 << 20, total=(1 << 21) + 1024)
    assert layout(**big) == WORKSPACE and layout(**big, ws=P, nws=need - 1) == WORKSPACE
    assert layout(t=1 << 30, k=4, total=(1 << 32) + 1024) == UNSUPPORTED
    # the contiguous layout of the worst choice fits, and is reached: one entry past a block for each expert
    assert dg.dg_moe_layout_rows(0, 8, 4) == 0 and dg.dg_moe_layout_rows(1, 8, 256) == 8 * 128
    for t, k, e in ((129, 4, 4), (1, 1, 1), (57, 3, 64), (1000, 8, 256)):
        n = t * k
        worst, rest = 0, n
        for i in range(min(e, n)):
            take = 1 if i else rest - (min(e, n) - 1)
            worst += -(-take // 128) * 128
        assert worst <= dg.dg_moe_layout_rows(t, k, e) < n + min(e, n) * 128


def test_dispatch_and_combine_refusals(lib):
    def disp(x=P, dtype=1, rows=P, src=P, mi=P, t=4, k=2, h=64, total=1024, per=0, out=P):
        return lib.dg_moe_dispatch(x, dtype, rows, src, mi, t, k, h, total, per, out, None)

    for bad in (dict(x=None), dict(out=None), dict(rows=None), dict(src=None), dict(h=0), dict(h=40), dict(dtype=3), dict(k=65),
                dict(t=-1), dict(per=128), dict(mi=None), dict(mi=None, per=100, total=1024), dict(x=MIS), dict(out=MIS)):
        assert disp(**bad) == INVALID, bad
    assert disp(total=0, t=0, x=None, out=None) == OK

    def fp8(ld=1024, s=P, per=0, mi=P, total=1024, ws=None):
        return lib.dg_moe_dispatch_fp8(P, 1, P, P, mi, 4, 2, 64, total, per, P, s, ld, ws, 0, None)

    assert dg.dg_moe_dispatch_fp8_workspace_size(4, 2, 64) == 0 and dg.dg_moe_dispatch_fp8_workspace_size(4, 2, 60) == 0
    assert dg.dg_moe_dispatch_fp8_workspace_size(1 << 16, 8, 7168) == (1 << 16) * 56 * 4
    for bad in (dict(ws=MIS), dict(ld=1020), dict(ld=1026), dict(s=None), dict(per=32, mi=None, ld=28)):
        assert fp8(**bad) == INVALID, bad
    assert lib.dg_moe_dispatch_int8(P, 1, P, P, P, 4, 2, 64, 1024, 0, P, None, None) == INVALID

    def comb(out=P, dtype=1, rows=P, w=P, t=4, k=2, h=64, total=1024, y=P):
        return lib.dg_moe_combine(out, dtype, rows, w, t, k, h, total, y, None)

    for bad in (dict(out=None), dict(rows=None), dict(y=None), dict(h=24), dict(total=-1), dict(w=MIS), dict(y=MIS), dict(dtype=9)):
        assert comb(**bad) == INVALID, bad
    assert comb(t=0, out=None, y=None, rows=None) == OK

    def cg(dy=P, out=P, rows=P, src=P, mi=P, w=P, dout=P, dw=P, h=64):
        return lib.dg_moe_combine_grad(dy, out, 1, rows, src, mi, w, 4, 2, h, 1024, dout, dw, None)

    for bad in (dict(dy=None), dict(out=None), dict(w=None), dict(dout=None), dict(dw=None), dict(src=None), dict(h=8),
                dict(dy=MIS), dict(dw=MIS)):
        assert cg(**bad) == INVALID, bad


def test_int8_refusals(lib):
    q = lambda x=P, dt=1, r=4, k=64, c=P, s=P: lib.dg_quantize_int8_per_token(x, dt, r, k, c, s, None)
    for bad in (dict(x=None), dict(c=None), dict(s=None), dict(k=0), dict(k=40), dict(r=-1), dict(dt=5), dict(x=MIS), dict(s=MIS)):
        assert q(**bad) == INVALID, bad
    assert q(r=0, x=None, c=None, s=None) == OK

    def nt(a=P, sa=P, b=P, sb=P, d=P, dt=1, m=4, n=8, k=64, ws=None):
        return lib.dg_gemm_int8_nt(a, sa, b, sb, d, dt, m, n, k, ws, 0, None)

    for bad in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(d=None), dict(dt=3), dict(m=-1), dict(n=-1),
                dict(k=0), dict(k=24), dict(a=MIS), dict(d=MIS), dict(sa=MIS), dict(ws=MIS)):
        assert nt(**bad) == INVALID, bad
    assert nt(k=131072) == UNSUPPORTED
    assert nt(m=0, a=None, sa=None, d=None) == OK and nt(n=0, b=None) == OK

    def aq(x=P, dt=1, m=4, ws=P, nws=1 << 30, k=64):
        return lib.dg_gemm_int8_nt_act_quant(x, dt, P, P, P, 1, m, 8, k, ws, nws, None)

    for bad in (dict(x=None), dict(dt=3), dict(k=40), dict(ws=MIS), dict(m=-2)):
        assert aq(**bad) == INVALID, bad
    assert aq(k=1 << 20) == UNSUPPORTED
    assert dg.dg_gemm_int8_nt_act_quant_workspace_size(4, 8, 40) == 0
    assert dg.dg_gemm_int8_workspace_size(4, 8, 1 << 20) == 0

    def cont(mi=P, g=2, m=256, k=64, a=P):
        return lib.dg_gemm_int8_grouped_contiguous(a, P, P, P, mi, g, P, 1, m, 8, k, None)

    for bad in (dict(mi=None), dict(m=200), dict(g=-1), dict(k=8), dict(a=None)):
        assert cont(**bad) == INVALID, bad
    assert cont(g=0) == OK and cont(m=0) == OK

    def mask(mm=P, g=2, m=16, k=64):
        return lib.dg_gemm_int8_grouped_masked(P, P, P, P, P, 1, mm, g, m, 8, k, None, 0, None)

    for bad in (dict(mm=None), dict(g=-1), dict(g=1025), dict(k=8), dict(m=-1)):
        assert mask(**bad) == INVALID, bad
    assert mask(g=0) == OK and mask(m=0) == OK


def test_binding_refusals():
    z = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt)
    with pytest.raises(ValueError):
        dg.dg_moe_route(z(4, 8), 2)   # not on the GPU
    with pytest.raises(ValueError):
        dg.dg_moe_layout(z(4, 2, dt=torch.int64), 8)
    with pytest.raises(ValueError):
        dg.dg_quantize_int8_per_token(z(4, 64))
    with pytest.raises(ValueError):
        dg.dg_gemm_int8_nt(z(4, 64), z(4), z(8, 64, dt=torch.int8), z(8))
    with pytest.raises(ValueError):
        dg.dg_gemm_int8_nt(z(4, 64, dt=torch.int8), z(5), z(8, 64, dt=torch.int8), z(8))
    with pytest.raises(ValueError):
        dg.dg_gemm_int8_nt_act_quant(z(4, 64), z(8, 32, dt=torch.int8), z(8))


# ---- the plain implementations ------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_plain_route_against_torch(score, renormalize):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((9, 24))
    ids, w = oracle.moe.route(x, 5, score=score, renormalize=renormalize, scale=2.0)
    t = torch.from_numpy(x).requires_grad_(True)
    s = torch.softmax(t, 1) if score == "softmax" else torch.sigmoid(t)
    top = torch.topk(s, 5, dim=1)
    assert np.array_equal(ids, top.indices.numpy())
    tw = 2.0 * (top.values / top.values.sum(1, keepdim=True) if renormalize else top.values)
    np.testing.assert_allclose(w, tw.detach().numpy(), rtol=1e-12)
    g = rng.standard_normal(w.shape)
    (tw * torch.from_numpy(g)).sum().backward()
    dx = oracle.moe.route_grad(g, x, ids, score, renormalize, 2.0)
    np.testing.assert_allclose(dx, t.grad.numpy(), rtol=1e-10, atol=1e-14)
    # and by differences, the choice held fixed
    for _ in range(6):
        d = rng.standard_normal(x.shape)
        h = 1e-5
        lhs = sum(sign * (g * oracle.moe.weights_of(x + sign * h * d, ids, score, renormalize, 2.0)).sum()
                  for sign in (1, -1)) / (2 * h)
        assert abs(lhs - (dx * d).sum()) <= 1e-8 * max(1.0, abs(lhs))


def test_plain_route_rules():
    inf = np.inf
    x = np.array([[1.0, 3.0, 3.0, -inf], [-inf] * 4, [0.0, -0.0, 0.0, 0.0]])
    ids, w = oracle.moe.route(x, 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 1, 2]]
    assert np.allclose(w[0].sum(), 1) and np.all(w[1] == 0) and np.allclose(w[2], 1 / 3)
    # bias moves the choice, not the weight
    ids, w = oracle.moe.route(np.zeros((1, 4)), 1, bias=np.array([0, 0, 0.5, 0]), score="sigmoid", renormalize=False)
    assert ids.tolist() == [[2]] and w[0, 0] == 0.5
    # groups of two, scores (0.9, 0.01) and (0.5, 0.6): judged by one expert the first stays, by two the second
    x = np.array([[0.9, 0.01, 0.5, 0.6]])
    logit = np.log(x / (1 - x))
    assert oracle.moe.route(logit, 1, num_groups=2, score="sigmoid")[0].tolist() == [[0]]
    assert oracle.moe.route(logit, 2, num_groups=2, group_top=2, score="sigmoid")[0].tolist() == [[3, 2]]


def test_plain_layout_dispatch_combine():
    rng = np.random.default_rng(6)
    ids = rng.integers(-1, 5, (40, 3)).astype(np.int32)
    rows, sources, m_indices, counts = oracle.moe.layout(ids, 5)
    assert len(sources) % 128 == 0 and len(m_indices) == len(sources) and counts.sum() == (ids >= 0).sum()
    there = ids >= 0
    assert np.array_equal(m_indices[rows[there]], ids[there])
    assert np.array_equal(sources[rows[there]], np.flatnonzero(there.reshape(-1)))
    assert np.all(rows[~there] == -1) and (sources >= 0).sum() == there.sum()
    for e in range(5):   # in order within the expert
        mine = rows.reshape(-1)[ids.reshape(-1) == e]
        assert np.all(np.diff(mine) == 1) and (mine.size == 0 or mine[0] % 128 == 0)
    x = rng.standard_normal((40, 16))
    w = rng.random((40, 3))
    xr = oracle.moe.dispatch(x, sources, 3)
    # combining what was dispatched gives each row times the weights of its entries that have a row
    np.testing.assert_allclose(oracle.moe.combine(xr, rows, w), x * (w * there).sum(1)[:, None], rtol=1e-12)
    # gradients: <dy, combine> differentiated in out and in w
    dy = rng.standard_normal((40, 16))
    dout, dw = oracle.moe.combine_grad(dy, xr, rows, w)
    d_out, d_w = rng.standard_normal(xr.shape), rng.standard_normal(w.shape)
    h = 1e-6
    f = lambda a, b: (dy * oracle.moe.combine(a, rows, b)).sum()
    assert abs((f(xr + h * d_out, w) - f(xr - h * d_out, w)) / (2 * h) - (dout * d_out).sum()) < 1e-6
    assert abs((f(xr, w + h * d_w) - f(xr, w - h * d_w)) / (2 * h) - (dw * d_w).sum()) < 1e-6
    # masked: fixed pitch, the surplus dropped
    rows, sources, m_indices, counts = oracle.moe.layout(ids, 5, rows_per_expert=16)
    assert m_indices is None and len(sources) == 80
    assert (rows >= 0).sum() == np.minimum(counts, 16).sum() == (sources >= 0).sum()
    got = rows[rows >= 0]
    assert np.array_equal(got // 16, ids[rows >= 0])


def test_plain_int8():
    q, s = oracle.int8.quantize(np.array([[0, 0, 0], [127, -127, 63.5], [1, 0.5, -0.25], [254, 1, -3]], dtype=np.float32))
    assert s.tolist() == [1.0, 1.0, np.float32(1) / np.float32(127), 2.0]
    assert q.tolist() == [[0, 0, 0], [127, -127, 64], [127, 64, -32], [127, 0, -2]]   # ties to even: 63.5, 0.5, -1.5
    a = np.full((2, 64), -128, dtype=np.int8)
    one = np.ones(2, dtype=np.float32)
    assert np.all(oracle.int8.gemm_nt(a, one, a, one) == 128 * 128 * 64)
    rng = np.random.default_rng(7)
    a, b = rng.integers(-127, 128, (5, 48)), rng.integers(-127, 128, (7, 48))
    sa, sb = rng.random(5).astype(np.float32), rng.random(7).astype(np.float32)
    want = [[sum(int(x) * int(y) for x, y in zip(r, c)) * float(u) * float(v) for c, v in zip(b, sb)] for r, u in zip(a, sa)]
    np.testing.assert_allclose(oracle.int8.gemm_nt(a.astype(np.int8), sa, b.astype(np.int8), sb), want, rtol=1e-14)
