"""The feed-forward operators where indexes and loops end: every length of K around the main loops' steps, more rows than a
launch holds workgroups of along x, offsets past 32 bits, calls at once on two streams.

Tolerances: those of the gated products' tests (64-bit arithmetic); elsewhere the same bits as the call on the rows alone.
Random codes (test_gated_product_of_many_rows) have products of all sizes, for which 2^-14 of their magnitudes is no bound:
a matrix instruction adds 8 neighbouring products at a time and keeps of each what reaches 2^-13 of the power of two below
the largest (measured: beside 2^16 the product 2^3 counts, 2^2 does not, at the seven places next to it and at no
other; 100 of them beside it lose 7).  So each loses less than min(|p|, 2^-13 max |p|), the largest nothing (8
bits); the groups' sums and the promotion add less than 2^-19 of the magnitudes (16 sums of 24 bits)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
from gpu_util import device, say
from test_gpu_gated_gemm import OF, alone, check_bf16, check_fp8, dequantized, operands, reference, same_bits

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("tile", ["stream=16", "stream=64", "tile=256x128", "tile=256x256"])
@pytest.mark.parametrize("k", [16, 128, 144, 384, 512, 528, 640, 768, 896, 1024, 1168])
def test_every_length_of_k(tile, k, monkeypatch):
    """One to ten K blocks, whole and partial, through rings of two, three, four and six blocks; several tiles a
    workgroup (few CUs), so that a tile's end meets the next one's start."""
    say("gated K", tile, k)
    monkeypatch.setenv("DG_PLAN", f"{tile},splits=1")
    rng = np.random.default_rng(k)
    a, sa, b, sb = operands(rng, (300,), 272, k)
    h, eh = reference(a, sa, 300, b, sb, "silu")[2::3]
    dg.dg_set_num_cus(8)
    try:
        d = dg.dg_gemm_fp8_gated_nt(a, sa, b, sb)
        q, s = dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, out="fp8")
    finally:
        dg.dg_set_num_cus(256)
    check_bf16(d, h, eh, "h")
    check_fp8(q, s[:, :300].t(), h, eh, "fp8")


@pytest.mark.parametrize("k", [128, 384, 512, 640, 896])
def test_lengths_of_k_in_groups(k, monkeypatch):
    """The same for the grouped forms on the 256x128 tile: contiguous, and masked with empty and full experts."""
    say("gated K in groups", k)
    monkeypatch.setenv("DG_PLAN", "tile=256x128")
    rng = np.random.default_rng(k + 1)
    a, sa, b, sb = operands(rng, (640,), 144, k, groups=3)
    experts = [2, 0, -1, 0, 1]
    mi = torch.tensor(experts, dtype=torch.int32, device=device()).repeat_interleave(128)
    counts = [200, 0, 130]
    masked = operands(rng, (3 * 256,), 144, k, groups=3)
    am = masked[0].view(3, 256, k)
    sm = masked[1][:, :768].view(-1, 3, 256).transpose(0, 1).contiguous()
    dg.dg_set_num_cus(8)
    try:
        d = dg.dg_gemm_fp8_gated_contiguous(a, sa, b, sb, mi, d=torch.full((640, 144), 7.0, dtype=BF16, device=device()))
        dm = dg.dg_gemm_fp8_gated_masked(am, sm, *masked[2:], torch.tensor(counts, dtype=torch.int32, device=device()),
                                         d=torch.full((3, 256, 144), 7.0, dtype=BF16, device=device()), use_workspace=False)
    finally:
        dg.dg_set_num_cus(256)
    for i, e in enumerate(experts):
        rows = slice(128 * i, 128 * i + 128)
        if e < 0:
            assert torch.all(d[rows] == 7)
        else:
            h, eh = reference(a[rows], sa[:, rows], 128, b[e], sb[e], "silu")[2::3]
            check_bf16(d[rows], h, eh, f"block {i}")
    for g, c in enumerate(counts):
        assert torch.all(dm[g, c:] == 7)
        if c:
            h, eh = reference(am[g, :c], sm[g, :, :c], c, masked[2][g], masked[3][g], "silu")[2::3]
            check_bf16(dm[g, :c], h, eh, f"expert {g}")


@pytest.mark.parametrize("n,k", [(16, 16), (128, 128), (112, 128), (128, 256), (64, 384), (128, 400)])
def test_one_column_block(n, k, monkeypatch):
    """One column block of one to four K blocks on the rings of two and three slots: the block scales are a few bytes, and
    the loads issued for K blocks behind the last one lie outside them (they would start 4 to 12 bytes past their end)."""
    say("gated one column block", n, k)
    rng = np.random.default_rng(n + k)
    a, sa, b, sb = operands(rng, (256,), n, k, groups=2)
    mi = torch.tensor([1, 0], dtype=torch.int32, device=device()).repeat_interleave(128)
    h = [reference(a[r], sa[:, r], 128, b[e], sb[e], "silu")[2::3] for r, e in ((slice(0, 128), 1), (slice(128, 256), 0))]
    h, eh = (np.concatenate(x) for x in zip(*h))
    for tile in ("256x128", "256x256"):
        monkeypatch.setenv("DG_PLAN", f"tile={tile},splits=1")
        pre = torch.full((256, 2 * n), 9.0, dtype=BF16, device=device())
        check_bf16(dg.dg_gemm_fp8_gated_contiguous(a, sa, b, sb, mi, pre=pre), h, eh, "contiguous")
        q, s = dg.dg_gemm_fp8_gated_contiguous(a, sa, b, sb, mi, out="fp8")
        check_fp8(q, s[:, :256].t(), h, eh, "contiguous fp8")
        for e, rows in ((1, slice(0, 128)), (0, slice(128, 256))):
            d = dg.dg_gemm_fp8_gated_nt(a[rows], sa[:, rows].contiguous(), alone(b[e]), alone(sb[e]))
            check_bf16(d, h[rows], eh[rows], "normal")
            for i in (0, 1):
                plain = dg.dg_gemm_fp8_nt(a[rows], sa[:, rows].contiguous(), alone(b[e, i]), alone(sb[e, i]))
                same_bits(pre[rows, i * n:(i + 1) * n], plain, f"projection {i}")


def wide_reference(a, sa, rows, b, sb):
    """(h, tolerance) for codes of any sizes, SiLU."""
    av, bv = dequantized(a, sa, rows, b, sb)
    g, u, e = av @ bv[0].T, av @ bv[1].T, []
    for w in bv:
        p = np.abs(av[:, None, :] * w[None]).reshape(rows, w.shape[0], -1, 8)
        cut = np.minimum(p, 2.0 ** -13 * p.max(-1, keepdims=True))
        e.append((cut.sum(-1) - cut.max(-1)).sum(-1) + 2.0 ** -19 * p.sum((-1, -2)))
    eg, eu = e
    f = OF.act_value(g, "silu")
    return f * u, 1.13 * eg * np.abs(u) + np.abs(f) * eu + 1.13 * eg * eu + (10 + 6 * np.abs(g)) * 2.0 ** -24 * np.abs(f * u)


def spots(rows):
    """Runs of rows at both ends and where 32-bit counts of elements and bytes would wrap."""
    at = sorted({0, 1 << 21, 1 << 22, 1 << 23, 1 << 24, 1 << 25, 1 << 26, rows - 40})
    return [slice(max(0, a - 24), a + 40) for a in at if a + 40 <= rows]


def test_gated_product_of_many_rows():
    """2^27 rows of 16: 2 GiB of activations, outputs past 2^32 bytes."""
    m, n, k = (1 << 27) - 100, 32, 16
    say("gated many rows", m, n, k)
    d = device()
    rng = np.random.default_rng(9)
    _, _, b, sb = operands(rng, (8,), n, k)
    gen = torch.Generator(device=d).manual_seed(11)
    a = torch.randint(0, 0x70, (m, k), dtype=torch.uint8, device=d, generator=gen)
    sa = torch.rand((1, m), device=d, generator=gen)
    out = dg.dg_gemm_fp8_gated_nt(a, sa, b, sb)
    for r in spots(m):
        h, eh = wide_reference(a[r], sa[:, r], r.stop - r.start, b, sb)
        check_bf16(out[r], h, eh, f"rows {r}")
    del out
    q, s = dg.dg_gemm_fp8_gated_nt(a, sa, b, sb, out="fp8")
    for r in spots(m):
        h, eh = wide_reference(a[r], sa[:, r], r.stop - r.start, b, sb)
        check_fp8(q[r], s[:, r].t(), h, eh, f"rows {r}")


def test_activation_of_many_rows():
    rows, n = (1 << 26) + 48, 32
    say("activation many rows", rows, n)
    d = device()
    pre = torch.randn((rows, 2 * n), device=d, dtype=BF16)
    h, (q, s), (q8, s8) = dg.dg_gated_act(pre), dg.dg_gated_act_fp8(pre), dg.dg_gated_act_int8(pre)
    for r in spots(rows):
        same_bits(h[r], dg.dg_gated_act(pre[r].clone()))
        want, ws = dg.dg_gated_act_fp8(pre[r].clone())
        same_bits(q[r], want)
        same_bits(s[:, r], ws[:, :want.shape[0]])
        want, ws = dg.dg_gated_act_int8(pre[r].clone())
        same_bits(q8[r].view(torch.uint8), want.view(torch.uint8))
        same_bits(s8[r], ws)
    del q, s, q8, s8
    got = dg.dg_gated_act_grad(h, pre)
    for r in spots(rows):
        same_bits(got[r], dg.dg_gated_act_grad(h[r].clone(), pre[r].clone()))


def test_norm_of_many_rows():
    rows, hidden = (1 << 26) + 48, 32
    say("norm many rows", rows, hidden)
    d = device()
    x, res = (torch.randn((rows, hidden), device=d, dtype=BF16) for _ in range(2))
    total, y = dg.dg_residual_norm(x, res)
    _, q, s = dg.dg_residual_norm_fp8(x, res)
    _, q8, s8 = dg.dg_residual_norm_int8(x, res)
    got = dg.dg_residual_norm_grad(y, res, x, total)
    for r in spots(rows):
        xr, rr = x[r].clone(), res[r].clone()
        same_bits(total[r], dg.dg_residual_norm(xr, rr)[0])
        same_bits(y[r], dg.dg_residual_norm(xr, rr)[1])
        want = dg.dg_residual_norm_fp8(xr, rr)
        same_bits(q[r], want[1])
        same_bits(s[:, r], want[2][:, :xr.shape[0]])
        want = dg.dg_residual_norm_int8(xr, rr)
        same_bits(q8[r].view(torch.uint8), want[1].view(torch.uint8))
        same_bits(s8[r], want[2])
        want = dg.dg_residual_norm_grad(y[r].clone(), rr, xr, total[r].clone())
        same_bits(got.dx[r], want.dx)
        same_bits(got.dresidual[r], want.dresidual)


def test_two_streams_at_once():
    """K splits of one shape from two streams at once, each with its own default workspace, the calls in flight together."""
    say("gated two streams")
    rng = np.random.default_rng(8)
    cases = [operands(rng, (m,), 256, 4096) for m in (1, 1, 60, 100)]
    want = [dg.dg_gemm_fp8_gated_nt(*c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append([dg.dg_gemm_fp8_gated_nt(*c) for c in (cases if i else cases[::-1])])
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            for x, y in zip(outs, want if i else want[::-1]):
                same_bits(x, y)


def test_one_expert():
    """The masked form of one expert gets the workspace that its plan asks for."""
    say("gated one expert")
    rng = np.random.default_rng(7)
    a, sa, b, sb = operands(rng, (40,), 128, 4096)
    need = dg.dg_gemm_fp8_gated_workspace_size(40, 128, 4096, 1)
    assert not dg.dg_gemm_fp8_gated_config_name(2, 40, 128, 4096, 1).endswith("split1")
    ws = torch.zeros(need, dtype=torch.uint8, device=device())
    count = torch.tensor([37], dtype=torch.int32, device=device())
    d = dg.dg_gemm_fp8_gated_masked(a[None], sa[None], b[None], sb[None], count, workspace=ws)
    h, eh = reference(a[:37], sa, 37, b, sb, "silu")[2::3]
    check_bf16(d[0, :37], h, eh, "h")
    assert torch.all(ws[:65536] == 0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("rows,n", [(1024, 2048), (1040, 2048), (1168, 1792)])
def test_act_grad_fp8_of_many_tiles(rows, n, act, dtype):
    """Both sides of the number of tiles up to which four workgroups share one: the bits of the fp32 gradient followed by the
    library's quantizers, with values whose scales lie far from 1 on both sides, and one that is infinite."""
    say("act grad fp8", rows, n, act, dtype)
    g = torch.Generator(device=device()).manual_seed(rows + n)
    pre = (torch.randn((rows, 2 * n), generator=g, device=device()) * 1.5).to(dtype)
    dh = torch.randn((rows, n), generator=g, device=device()).to(dtype)
    dh[7] *= 2.0 ** -70
    dh[:, 300:420] *= 2.0 ** -80
    dh[200:330, 130] *= 2.0 ** 100
    dh[900, 1000] = float("inf")
    wide = dg.dg_gated_act_grad(dh.float(), pre.float(), act=act)
    h = dg.dg_gated_act(pre.float(), act=act)
    got = dg.dg_gated_act_grad_fp8(dh, pre, act=act)
    want = (*dg.dg_quantize_per_token_group(wide), *dg.dg_quantize_per_channel_group(wide),
            *dg.dg_quantize_per_channel_group(h))
    for i, (a, b) in enumerate(zip(got, want)):
        b = b[..., :a.shape[-1]]
        assert torch.equal(torch.isnan(a.float()), torch.isnan(b.float()))
        a, b = a.clone(), b.clone()
        if a.dtype == torch.float32:   # (any NaN is one)
            a[torch.isnan(a)] = b[torch.isnan(b)] = 0.0
        same_bits(a, b, f"output {i}")


@pytest.mark.parametrize("power", [-140, -120, -100, -59, -52, 0, 40, 66, 70, 100, 118])
def test_scales_of_every_size(power):
    """Groups whose scales are subnormal, at the borders of the range that products serve, and next to fp32's largest."""
    say("scales", power)
    g = torch.Generator(device=device()).manual_seed(power + 200)
    x = torch.randn((64, 1024), generator=g, device=device())
    pre = torch.cat([torch.full((64, 1024), 30.0, device=device()), x * 2.0 ** (power / 2) * 2.0 ** (power / 2)], 1)
    pre[:, 2000:2040] = 0
    h = dg.dg_gated_act(pre)
    q, s = dg.dg_gated_act_fp8(pre)
    want, ws = dg.dg_quantize_per_token_group(h)
    same_bits(q, want)
    same_bits(s[:, :64], ws[:, :64])


# ---- the norm gradient's sums over many rows --------------------------------------------------------

MANY_ROWS = [(16384, 1024, 1), (16384, 1024, 4096), (24000, 64, 1), (24000, 64, 3), (24000, 64, 80), (24000, 64, 12000), (24000, 1008, 240),
             (9000, 2048, 9), (9000, 2048, 1500), (16384, 7168, 1), (16384, 7168, 64), (4100, 16384, 4), ((1 << 20) + 96, 64, 1),
             ((1 << 20) + 96, 64, 8), ((1 << 20) + 96, 64, 32771), (300000, 1040, 1), (300000, 1040, 750)]


@pytest.mark.parametrize("rows,hidden,gates", MANY_ROWS)
def test_norm_grad_sums_of_many_rows(rows, hidden, gates):
    """Many rows for every row group of a workgroup, gates shorter and longer than its rows: sums of small integers (rows of +-1
    have the norm 1), which fp32 holds exactly, so that each row counts once and in its gate only."""
    say("norm grad many rows", rows, hidden, gates)
    d = device()
    gen = torch.Generator(device=d).manual_seed(rows + hidden)
    ints = lambda n: torch.randint(-n, n + 1, (rows, hidden), generator=gen, device=d)   # noqa: E731
    s = 1.0 - 2.0 * torch.randint(0, 2, (rows, hidden), generator=gen, device=d)
    w = torch.ones(hidden, device=d)
    dy = ints(3).float()
    dy[-1], dy[0] = 50.0, -40.0
    got = dg.dg_residual_norm_grad(dy, None, None, s, w, eps=0.0)
    assert torch.equal(got.dweight.double(), (dy.double() * s).sum(0))
    del got
    # dz = dsum without dy; the gate's gradient of dsum x, the first norm's of dsum gate x
    for dtype in (torch.float32, BF16):
        dsum, zero = ints(2).float(), torch.zeros((rows, hidden), dtype=dtype, device=d)
        dsum[-1], dsum[rows // 2] = 30.0, -20.0
        x = (1.0 - 2.0 * torch.randint(0, 2, (rows, hidden), generator=gen, device=d)).to(dtype)
        gate = torch.randint(-2, 3, (gates, hidden), generator=gen, device=d).to(dtype)
        got = dg.dg_residual_norm_grad(zero, dsum, x, s, w, gate=gate, post_norm=True, post_weight=w, eps=0.0)
        each = (dsum * x).view(gates, rows // gates, hidden).sum(1, dtype=torch.float64)
        assert torch.equal(got.dgate.double(), each.to(dtype).double())
        assert torch.equal(got.dpost_weight.double(), (each * gate).sum(0))
        assert torch.equal(got.dweight, torch.zeros_like(w))


@pytest.mark.parametrize("rows,hidden", [(1 << 24, 32), (1 << 20, 1040)])
def test_norm_grad_chains(rows, hidden):
    """One term over and over, whose sum fp32 rounds to the same side every time: chains of at most 256 rows (2^24 rows of up to
    1024, 2^22 of longer ones) and of rows / (64 * 256 * row groups) partials, and 16 more additions."""
    say("norm grad chains", rows, hidden)
    d = device()
    term = 1.0 + 7 * 2.0 ** -16
    s, dy = torch.ones((rows, hidden), device=d), torch.full((rows, hidden), term, device=d)
    got = dg.dg_residual_norm_grad(dy, None, None, s, torch.ones(hidden, device=d), eps=0.0).dweight.double()
    groups = 4 if hidden <= 1024 else 1
    chains = 256 + rows / (64 * 256 * groups) + 16
    assert torch.all((got / (rows * term) - 1).abs() <= chains * 2.0 ** -24)


# ---- quantization by corrected products, against the library's divisions ---------------------------

def quantized_products(x):
    """(codes, scales) of dg_gated_act_fp8 for h = x exactly, and of the library's quantizer for x: 2^5 sigmoid(2^5) is 2^5."""
    pre = torch.cat((torch.full_like(x, 32.0), x * 2.0 ** -5), 1)
    got = dg.dg_gated_act_fp8(pre)
    del pre
    return got, dg.dg_quantize_per_token_group(x)


@pytest.mark.parametrize("power", [-52, 0, 8, 66])
def test_every_significand_of_a_scale(power):
    """All 2^23 significands of a group's largest value, so every scale and reciprocal of a power of two; with each the
    values around every border of two codes times that scale (the odd sixteenths above 1 and the odd ones of the subnormal
    codes, and their two neighbours on each side), where a quotient rounded otherwise would be another code."""
    say("significands", power)
    d = device()
    borders = torch.tensor([(16 + i) / 16.0 for i in range(1, 16, 2)] + [i / 1024.0 for i in range(1, 16, 2)], device=d, dtype=torch.float64)
    for start in range(0, 1 << 23, 1 << 20):
        bits = torch.arange(start, start + (1 << 20), device=d, dtype=torch.int32)
        amax = (bits + ((127 + power) << 23)).view(torch.float32)
        s = (amax / torch.full_like(amax, 448.0)).double()
        at = (s[:, None] * borders[None]).float()
        near = torch.cat([(at.view(torch.int32) + i).view(torch.float32) for i in range(-2, 3)], 1)   # 80 values
        near[:, ::2] *= -1.0
        x = torch.cat((amax[:, None], near, torch.zeros((1 << 20, 15), device=d)), 1).contiguous()
        (q, sq), (want, sw) = quantized_products(x)
        same_bits(q, want, f"codes from {start}")
        same_bits(sq, sw[:, :1 << 20], f"scales from {start}")


def test_every_value_at_scale_one():
    """Every fp32 number from 0 to 448, of both signs, in groups whose scale is 1: codes, signs of zeros among them."""
    say("every value")
    d = device()
    top = 0x43e00000   # 448
    step = 127 << 20
    for start in range(0, top + 1, step):
        bits = torch.arange(start, start + step, device=d, dtype=torch.int64).clamp_(max=top).to(torch.int32)
        for sign in (1.0, -1.0):
            v = (bits.view(torch.float32) * sign).view(-1, 127)
            x = torch.cat((torch.full((v.shape[0], 1), 448.0, device=d), v), 1).contiguous()
            # (numbers that x / 32 does not hold are as good a probe after the product as before it)
            x = x * 2.0 ** -5 * 2.0 ** 5
            (q, sq), (want, sw) = quantized_products(x)
            same_bits(q, want, f"from {start:#x} {sign}")
            assert torch.all(sq[:, :x.shape[0]] == 1)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_act_grad_fp8_of_nan(dtype):
    """Groups of nothing but NaN, of NaN beside numbers and beside infinities, by rows and by columns: the library's quantizers' bits."""
    say("act grad fp8 nan", dtype)
    g = torch.Generator(device=device()).manual_seed(5)
    rows, n, nan = 272, 256, float("nan")
    pre = torch.randn((rows, 2 * n), generator=g, device=device()).to(dtype)
    dh = torch.randn((rows, n), generator=g, device=device()).to(dtype)
    pre[:, n + 7] = nan           # columns of one projection
    pre[128:256, 9] = nan
    dh[3] = nan                   # a row
    dh[140:150, 40] = nan
    dh[200, 130] = float("inf")
    dh[201:205, 130] = nan
    dh[256:, 200] = nan           # a partial group of rows
    wide = dg.dg_gated_act_grad(dh.float(), pre.float())
    h = dg.dg_gated_act(pre.float())
    got = dg.dg_gated_act_grad_fp8(dh, pre)
    want = (*dg.dg_quantize_per_token_group(wide), *dg.dg_quantize_per_channel_group(wide), *dg.dg_quantize_per_channel_group(h))
    for i, (a, b) in enumerate(zip(got, want)):
        b = b[..., :a.shape[-1]]
        assert torch.equal(torch.isnan(a.float()), torch.isnan(b.float())), f"output {i}"
        if a.dtype == torch.float32:   # (any NaN is one)
            a, b = a.nan_to_num(nan=0.0, posinf=float("inf")), b.nan_to_num(nan=0.0, posinf=float("inf"))
        same_bits(a, b, f"output {i}")
