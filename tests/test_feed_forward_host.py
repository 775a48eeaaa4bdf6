"""Gated feed-forward operators and residual norms without a GPU: what the entry points refuse, the sizes they report, and
the plain implementations against torch's autograd and against differences."""

import ctypes

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
import oracle

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P, MIS = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1002)   # never dereferenced: the checks come first
MIS4 = ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def lib():
    return dg.lib()


# ---- what is refused ------------------------------------------------------------------------------

def test_gated_refusals(lib):
    base = dict(a=P, sa=P, ld=8, b=P, sb=P)
    out = dict(act=0, d=P, q=None, s=None, ld_s=0, pre=None, m=8, n=64, k=128)

    def nt(ws=None, nws=0, **kw):
        v = {**base, **out, **kw}
        return lib.dg_gemm_fp8_gated_nt(*v.values(), ws, nws, None)

    fp8 = dict(d=None, q=P, s=P, ld_s=8)
    common = (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(d=None), dict(q=P), dict(act=2), dict(act=-1),
              dict(m=-1), dict(n=-1), dict(k=0), dict(k=24), dict(ld=4), dict(ld=10), dict(a=MIS), dict(b=MIS), dict(d=MIS),
              dict(pre=MIS), {**fp8, "s": None}, {**fp8, "n": 72}, {**fp8, "ld_s": 4}, {**fp8, "ld_s": 9}, {**fp8, "s": MIS},
              {**fp8, "q": MIS})
    for bad in common + (dict(ws=MIS),):
        assert nt(**bad) == INVALID, bad
    assert nt(m=0, a=None, sa=None, d=None) == OK and nt(n=0) == OK
    assert lib.dg_set_num_cus(256) == OK     # (without a device, so that the plans can be made)
    assert nt(n=1 << 23, k=128) == UNSUPPORTED
    assert nt(m=1 << 21, k=1024, ld=1 << 21) == UNSUPPORTED

    def grouped(name, where=P, g=2, tail=(), **kw):
        v = {**base, **out, **kw}
        v = list(v.values())
        return getattr(lib, name)(*v[:5], where, g, *v[5:], *tail, None)

    for bad in common[:-1] + (dict(where=None), dict(where=MIS), dict(g=-1)):
        assert grouped("dg_gemm_fp8_gated_masked", tail=(None, 0), **bad) == INVALID, bad
        assert grouped("dg_gemm_fp8_gated_contiguous", **{"m": 128, "ld": 128, **({"ld_s": 128} if bad.get("q") else {}), **bad}) == INVALID, bad
    assert grouped("dg_gemm_fp8_gated_masked", tail=(None, 0), g=1025) == INVALID
    assert grouped("dg_gemm_fp8_gated_contiguous", m=100, ld=100) == INVALID
    assert grouped("dg_gemm_fp8_gated_contiguous", g=0) == OK and grouped("dg_gemm_fp8_gated_masked", g=0, tail=(None, 0)) == OK


def test_gated_plans(lib, monkeypatch):
    """Names and workspaces of the plans; forced ones; no plan for what is refused."""
    assert lib.dg_set_num_cus(256) == OK
    for m, n, k, groups in ((1, 2048, 7168, 1), (64, 128, 4096, 1), (100, 256, 2048, 1), (8192, 8192, 7168, 1), (5, 300, 640, 8)):
        name = dg.dg_gemm_fp8_gated_config_name(2 if groups > 1 else 0, m, n, k, groups)
        tile, splits = name.split("/")[0].removeprefix("stream"), int(name.rsplit("split", 1)[1])
        bn, bm = (int(v) for v in tile.split("x"))
        assert bn == 256 and bm in (16, 64, 128, 256)
        tiles = -(-n // 128) * -(-m // bm) * groups
        need = dg.dg_gemm_fp8_gated_workspace_size(m, n, k, groups)
        assert need == (65536 + tiles * splits * bn * bm * 4 if splits > 1 else 0)
    monkeypatch.setenv("DG_PLAN", "tile=256x128,splits=5")
    assert dg.dg_gemm_fp8_gated_config_name(0, 8, 128, 1280) == "256x128/8waves/split5"
    assert dg.dg_gemm_fp8_gated_config_name(1, 128, 128, 1280, 2) == "256x128/8waves/split1"
    monkeypatch.setenv("DG_PLAN", "stream=64")
    assert dg.dg_gemm_fp8_gated_config_name(0, 1000, 1280, 1280).startswith("stream256x64/8waves/")
    assert not dg.dg_gemm_fp8_gated_config_name(1, 128, 128, 1280, 2).startswith("stream")
    monkeypatch.delenv("DG_PLAN")
    for bad in ((3, 8, 128, 128, 1), (0, 0, 128, 128, 1), (0, 8, 0, 128, 1), (0, 8, 128, 100, 1), (2, 8, 128, 128, 0), (2, 8, 128, 128, 1025)):
        assert dg.dg_gemm_fp8_gated_config_name(*bad) == ""
    assert dg.dg_gemm_fp8_gated_workspace_size(8, 128, 100) == 0 and dg.dg_gemm_fp8_gated_workspace_size(8, 128, 128, 0) == 0


def test_gated_sizes_at_their_limits(lib):
    """Scales whose offsets leave 32 bits are refused; one expert's workspace is that of either form."""
    assert lib.dg_set_num_cus(256) == OK
    out = (0, P, None, None, 0, None, 8, 64)
    assert lib.dg_gemm_fp8_gated_nt(P, P, 1 << 29, P, P, *out, 128, None, 0, None) == UNSUPPORTED
    assert lib.dg_gemm_fp8_gated_nt(P, P, 1 << 28, P, P, *out, 256, None, 0, None) == UNSUPPORTED
    for m, n, k in ((8, 128, 4096), (40, 128, 4096), (100, 256, 2048), (256, 256, 7168)):
        for layout in (0, 2):
            name = dg.dg_gemm_fp8_gated_config_name(layout, m, n, k, 1)
            splits = int(name.rsplit("split", 1)[1])
            bn, bm = (int(v) for v in name.split("/")[0].removeprefix("stream").split("x"))
            need = 65536 + -(-n // 128) * -(-m // bm) * splits * bn * bm * 4 if splits > 1 else 0
            assert dg.dg_gemm_fp8_gated_workspace_size(m, n, k, 1) >= need


def test_gated_binding_refusals():
    a, sa = torch.zeros((8, 128), dtype=torch.uint8), torch.zeros((1, 8))
    b, sb = torch.zeros((2, 64, 128), dtype=torch.uint8), torch.zeros((2, 1, 1))
    mi = torch.zeros(8, dtype=torch.int32)
    for bad in (lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb),   # not on a device
                lambda: dg.dg_gemm_fp8_gated_nt(a[0], sa, b, sb), lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b[:, :, :64], sb),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b.view(128, 128), sb),   # stacked rows need N % 128 == 0
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb[:1]), lambda: dg.dg_gemm_fp8_gated_nt(a, sa[:, :4], b, sb),
                lambda: dg.dg_gemm_fp8_gated_nt(a.int(), sa, b, sb), lambda: dg.dg_gemm_fp8_gated_nt(a, sa.double(), b, sb),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, out="int8"), lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, q=a),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, out="fp8", d=torch.zeros((8, 64), dtype=torch.bfloat16)),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b[:, :40].contiguous(), sb, out="fp8"),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, pre=torch.zeros((8, 64), dtype=torch.bfloat16)),
                lambda: dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, d=torch.zeros((8, 64))),
                lambda: dg.dg_gemm_fp8_gated_contiguous(a, sa, b[None], sb[None], mi.long()),
                lambda: dg.dg_gemm_fp8_gated_contiguous(a, sa, b[None], sb[None], mi[:4]),
                lambda: dg.dg_gemm_fp8_gated_masked(a, sa, b[None], sb[None], mi[:1]),
                lambda: dg.dg_gemm_fp8_gated_masked(a[None], sa[None], b[None], sb[None], mi)):
        with pytest.raises(ValueError):
            bad()


def test_gated_scale_shapes():
    """Weight scales of another axis order have as many elements: refused, not read as if they were in order."""
    n, k, g = 384, 256, 3
    a, sa = torch.zeros((128, k), dtype=torch.uint8), torch.zeros((2, 128))
    mi, mm = torch.zeros(128, dtype=torch.int32), torch.zeros(g, dtype=torch.int32)
    b, stacked = torch.zeros((g, 2, n, k), dtype=torch.uint8), torch.zeros((g, 2 * n, k), dtype=torch.uint8)
    right, right_stacked = torch.zeros((g, 2, 3, 2)), torch.zeros((g, 6, 2))
    for sb in (right.transpose(2, 3), right.transpose(0, 1), right.transpose(2, 3).contiguous(), torch.zeros((2, g, 3, 2)),
               torch.zeros((g, 2, 6)), torch.zeros((6, g, 2)), torch.zeros((g, 3, 4))):
        assert sb.numel() == right.numel()
        for w in (b, stacked):
            with pytest.raises(ValueError, match="sb must be"):
                dg.dg_gemm_fp8_gated_contiguous(a, sa, w, sb, mi)
            with pytest.raises(ValueError, match="sb must be"):
                dg.dg_gemm_fp8_gated_masked(torch.zeros((g, 8, k), dtype=torch.uint8), torch.zeros((g, 2, 8)), w, sb, mm)
    for w in (b[0], stacked[0]):
        for sb in (torch.zeros((2, 2, 3)), torch.zeros((3, 2, 2)), torch.zeros((2, 6)), torch.zeros((1, 6, 2))):
            with pytest.raises(ValueError, match="sb must be"):
                dg.dg_gemm_fp8_gated_nt(a, sa, w, sb)
        for sb in (right[0], right_stacked[0]):   # in order, whichever the weights' shape: refused for the device alone
            with pytest.raises(ValueError, match="CUDA"):
                dg.dg_gemm_fp8_gated_nt(a, sa, w, sb)


def test_act_refusals(lib):
    def act(pre=P, dt=1, a=0, mi=None, mm=None, per=0, rows=32, n=64, h=P):
        return lib.dg_gated_act(pre, dt, a, mi, mm, per, rows, n, h, None)

    common = (dict(pre=None), dict(dt=3), dict(dt=-1), dict(a=2), dict(a=-1), dict(rows=-1), dict(n=0), dict(n=24),
              dict(mi=P, mm=P, per=8), dict(mm=P), dict(mm=P, per=5), dict(per=8), dict(pre=MIS), dict(mi=MIS), dict(mm=MIS, per=8),
              dict(n=1 << 28))
    for bad in common + (dict(h=None), dict(h=MIS4)):
        assert act(**bad) == INVALID, bad
    assert act(rows=0, pre=None, h=None) == OK

    def fp8(q=P, s=P, ld=32, **kw):
        a = dict(pre=P, dt=1, a=0, mi=None, mm=None, per=0, rows=32, n=64)
        a.update(kw)
        return lib.dg_gated_act_fp8(*a.values(), q, s, ld, None)

    for bad in common + (dict(q=None), dict(s=None), dict(ld=28), dict(ld=33), dict(s=MIS), dict(mm=P, per=16, ld=12)):
        assert fp8(**bad) == INVALID, bad

    def i8(q=P, s=P, **kw):
        a = dict(pre=P, dt=1, a=0, mi=None, mm=None, per=0, rows=32, n=64)
        a.update(kw)
        return lib.dg_gated_act_int8(*a.values(), q, s, None)

    for bad in common + (dict(q=None), dict(s=None), dict(q=MIS), dict(s=MIS)):
        assert i8(**bad) == INVALID, bad


def test_act_grad_refusals(lib):
    def grad(dh=P, pre=P, dt=1, a=0, rows=32, n=64, out=P):
        return lib.dg_gated_act_grad(dh, pre, dt, a, rows, n, out, None)

    for bad in (dict(dh=None), dict(pre=None), dict(out=None), dict(dt=4), dict(a=3), dict(rows=-1), dict(n=8), dict(dh=MIS),
                dict(out=MIS)):
        assert grad(**bad) == INVALID, bad
    assert grad(rows=0, dh=None, pre=None, out=None) == OK

    def fp8(dh=P, pre=P, dt=1, a=0, rows=32, n=128, q=P, s=P, ld=32, qt=P, st=P, ldt=256, ht=P, hst=P, ldh=128):
        return lib.dg_gated_act_grad_fp8(dh, pre, dt, a, rows, n, q, s, ld, qt, st, ldt, ht, hst, ldh, None)

    for bad in (dict(n=64), dict(n=144), dict(rows=24), dict(dh=None), dict(pre=None), dict(q=None), dict(s=None), dict(qt=None),
                dict(st=None), dict(ht=None), dict(hst=None), dict(ld=28), dict(ld=34), dict(ldt=252), dict(ldh=124),
                dict(q=None, s=None, qt=None, st=None, ht=None, hst=None), dict(s=MIS4), dict(qt=MIS), dict(hst=MIS4)):
        assert fp8(**bad) == INVALID, bad
    assert fp8(rows=0) == OK


def test_norm_refusals(lib):
    base = dict(x=P, r=P, dt=1, rdt=1, w=P, gate=None, gr=0, post=0, pw=None, scale=1.0, eps=1e-6, rows=8, h=64, sum=P)
    common = (dict(r=None), dict(dt=3), dict(rdt=2), dict(dt=0, rdt=1), dict(h=0), dict(h=40), dict(rows=-1), dict(gate=P),
              dict(gr=2), dict(gate=P, gr=3), dict(gate=P, gr=-1), dict(pw=P), dict(eps=-1.0), dict(eps=float("inf")),
              dict(eps=float("nan")), dict(x=None), dict(x=None, sum=None, gate=P, gr=1), dict(x=None, sum=None, post=1),
              dict(x=MIS), dict(r=MIS), dict(w=MIS4), dict(sum=MIS), dict(gate=MIS, gr=1), dict(post=1, pw=MIS4))

    def call(name, tail, **kw):
        a = dict(base)
        a.update(kw)
        return getattr(lib, name)(*a.values(), *tail, None)

    for name, tail, more in (("dg_residual_norm", (P,), ((None,), (MIS,))),
                             ("dg_residual_norm_fp8", (P, P, 8), ((None, P, 8), (P, None, 8), (P, P, 4), (P, P, 9), (P, MIS, 8))),
                             ("dg_residual_norm_int8", (P, P), ((None, P), (P, None), (P, MIS)))):
        for bad in common:
            assert call(name, tail, **bad) == INVALID, (name, bad)
        for bad in more:
            assert call(name, bad) == INVALID, (name, bad)
        assert call(name, tail, h=16400) == UNSUPPORTED and call(name, tail, rows=0, x=None, r=None, sum=None) == OK


def test_norm_grad_refusals(lib):
    def grad(dy=P, ds=P, x=P, s=P, dt=1, rdt=0, w=P, gate=P, gr=4, post=1, pw=P, eps=1e-6, rows=8, h=64, dx=P, dr=P, dw=P,
             dgate=P, dpw=P, ws=P, nws=1 << 40):
        return lib.dg_residual_norm_grad(dy, ds, x, s, dt, rdt, w, gate, gr, post, pw, 1.0, eps, rows, h, dx, dr, dw, dgate,
                                         dpw, ws, nws, None)

    for bad in (dict(dy=None), dict(s=None), dict(dr=None), dict(dx=None), dict(x=None), dict(x=None, dx=None), dict(w=None),
                dict(gate=None, gr=0), dict(pw=None), dict(post=0), dict(gr=3), dict(rdt=2), dict(h=24), dict(eps=-1.0),
                dict(ds=MIS), dict(dw=MIS4), dict(ws=MIS4), dict(dgate=MIS), dict(rows=-8)):
        assert grad(**bad) == INVALID, bad
    need = dg.dg_residual_norm_grad_workspace_size(8, 64)
    assert need > 0 and grad(ws=None) == WORKSPACE and grad(nws=need - 1) == WORKSPACE
    assert grad(h=16400) == UNSUPPORTED
    assert dg.dg_residual_norm_grad_workspace_size(0, 64) == 0 and dg.dg_residual_norm_grad_workspace_size(8, 60) == 0


def test_binding_refusals():
    """Shapes and types that the binding turns down before the library sees a pointer (no device is needed)."""
    pre = torch.zeros((4, 64))
    for bad in (lambda: dg.dg_gated_act(pre, act="relu"), lambda: dg.dg_gated_act(pre[:, :63]),
                lambda: dg.dg_gated_act(torch.zeros((2, 4, 64))),
                lambda: dg.dg_gated_act(pre, masked_m=torch.zeros(4, dtype=torch.int32)),
                lambda: dg.dg_gated_act(pre, m_indices=torch.zeros(3, dtype=torch.int32)),
                lambda: dg.dg_gated_act(pre, m_indices=torch.zeros(4, dtype=torch.int64)),
                lambda: dg.dg_gated_act(pre, h=torch.zeros((4, 64))), lambda: dg.dg_gated_act(pre.double()),
                lambda: dg.dg_gated_act(pre),   # not on a device
                lambda: dg.dg_gated_act_grad(torch.zeros((4, 31)), pre), lambda: dg.dg_gated_act_grad(pre[:, :32].half(), pre),
                lambda: dg.dg_gated_act_grad_fp8(torch.zeros((4, 32)), pre),
                lambda: dg.dg_gated_act_fp8(pre, s=torch.zeros((1, 2)))):
        with pytest.raises(ValueError):
            bad()
    x = torch.zeros((6, 32), dtype=torch.bfloat16)
    w = torch.ones(32)
    for bad in (lambda: dg.dg_residual_norm(x, x, w, dtype=torch.float16), lambda: dg.dg_residual_norm(x, x.half(), w), lambda: dg.dg_residual_norm(x, x[:5], w),
                lambda: dg.dg_residual_norm(x, x, w.bfloat16()), lambda: dg.dg_residual_norm(x, x, w[:16]),
                lambda: dg.dg_residual_norm(x, x, w, gate=torch.zeros((4, 32), dtype=torch.bfloat16)),
                lambda: dg.dg_residual_norm(x, x, w, gate=w), lambda: dg.dg_residual_norm(x, x, w, post_weight=w),
                lambda: dg.dg_residual_norm(None, x, w, gate=x), lambda: dg.dg_residual_norm(None, x, w, post_norm=True),
                lambda: dg.dg_residual_norm(None, x, w, sum=x), lambda: dg.dg_residual_norm(x, x, w),
                lambda: dg.dg_residual_norm_fp8(x, x, w, q=torch.zeros((6, 31), dtype=torch.uint8)),
                lambda: dg.dg_residual_norm_int8(x, x, w, s=torch.zeros(5)),
                lambda: dg.dg_residual_norm_grad(x, None, x, x[:5], w), lambda: dg.dg_residual_norm_grad(x, x.float(), x, x, w),
                lambda: dg.dg_residual_norm_grad(x, None, None, x, w, dx=x)):
        with pytest.raises(ValueError):
            bad()


# ---- the plain implementations --------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_oracle_gated(act):
    rng = np.random.default_rng(1)
    pre, dh = rng.standard_normal((5, 24)) * 3, rng.standard_normal((5, 12))
    t = torch.from_numpy(pre).requires_grad_(True)
    f = torch.nn.functional.silu if act == "silu" else lambda a: torch.nn.functional.gelu(a, approximate="tanh")
    h = f(t[:, :12]) * t[:, 12:]
    h.backward(torch.from_numpy(dh))
    np.testing.assert_allclose(oracle.feed_forward.gated(pre, act), h.detach().numpy(), rtol=1e-13, atol=1e-14)
    got = oracle.feed_forward.gated_grad(dh, pre, act)
    np.testing.assert_allclose(got, t.grad.numpy(), rtol=1e-12, atol=1e-13)
    # differences: an error of step^2 f''' / 6, below 1e-8 for these functions
    step = 1e-5
    for at in ((0, 0), (3, 7), (2, 15), (4, 23)):
        d = np.zeros_like(pre)
        d[at] = step
        diff = ((oracle.feed_forward.gated(pre + d, act) - oracle.feed_forward.gated(pre - d, act)) * dh).sum() / (2 * step)
        assert abs(diff - got[at]) < 1e-8


@pytest.mark.parametrize("post,weights", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("gates", [0, 1, 2, 6])
def test_oracle_norm(post, weights, gates):
    rng = np.random.default_rng(gates + 10 * post)
    rows, hidden, scale, eps = 6, 16, 0.7, 1e-3
    r = lambda *s: rng.standard_normal(s)   # noqa: E731
    x, res, dy, ds = r(rows, hidden), r(rows, hidden), r(rows, hidden), r(rows, hidden)
    w, v = (1 + r(hidden) / 4, 1 + r(hidden) / 4) if weights else (None, None)
    gate = r(gates, hidden) if gates else None
    kw = dict(gate=gate, post_norm=post, post_weight=v if post else None, scale=scale, eps=eps)
    s, y = oracle.feed_forward.residual_norm(x, res, w, **kw)
    got = oracle.feed_forward.residual_norm_grad(dy, ds, x, s, w, **kw)

    t = {k: torch.from_numpy(a).requires_grad_(True) for k, a in dict(x=x, res=res, w=w, v=v, gate=gate).items() if a is not None}
    rms = lambda a: torch.sqrt((a * a).mean(1, keepdim=True) + eps)   # noqa: E731
    z = t["x"] / rms(t["x"]) * t.get("v", 1.0) if post else t["x"]
    ts = t["res"] + scale * z * (t["gate"].repeat_interleave(rows // gates, 0) if gates else 1.0)
    ty = ts / rms(ts) * t.get("w", 1.0)
    np.testing.assert_allclose(y, ty.detach().numpy(), rtol=1e-12)
    ((ty * torch.from_numpy(dy)).sum() + (ts * torch.from_numpy(ds)).sum()).backward()
    for name, leaf in (("dx", "x"), ("dresidual", "res"), ("dweight", "w"), ("dpost_weight", "v"), ("dgate", "gate")):
        if leaf in t and t[leaf].grad is not None:
            np.testing.assert_allclose(got[name], t[leaf].grad.numpy(), rtol=1e-10, atol=1e-12, err_msg=name)
            assert np.all(np.abs(got[name]) <= got["size_" + name] * (1 + 1e-12))
    # differences of the formula itself
    step = 1e-6

    def value(x1, res1):
        s1, y1 = oracle.feed_forward.residual_norm(x1, res1, w, **kw)
        return (y1 * dy).sum() + (s1 * ds).sum()

    for at in ((0, 0), (5, 15), (2, 7)):
        d = np.zeros_like(x)
        d[at] = step
        assert abs((value(x + d, res) - value(x - d, res)) / (2 * step) - got["dx"][at]) < 1e-6
        assert abs((value(x, res + d) - value(x, res - d)) / (2 * step) - got["dresidual"][at]) < 1e-6
    alone = oracle.feed_forward.residual_norm(None, res, w, eps=eps)
    np.testing.assert_allclose(alone[1], res / np.sqrt((res ** 2).mean(1, keepdims=True) + eps) * (1 if w is None else w))
