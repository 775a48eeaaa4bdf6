"""8-bit integer quantizer and GEMMs on the GPU against the plain 64-bit implementation.

Tolerance: the integer sum is exact, so a result is the sum's conversion to fp32, the product of the two
scales and the product with it - three roundings, 3 * 2^-24 of the value - and the rounding to the output's
type (2^-8 relative for bf16; 2^-11 for fp16, 2^-25 absolute near zero)."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
import oracle
from gpu_util import device, say

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
REL = {F32: 3 * 2.0 ** -24, BF16: 2.0 ** -8 + 4 * 2.0 ** -24, F16: 2.0 ** -11 + 4 * 2.0 ** -24}
ABS = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def host(t):
    return t.double().cpu().numpy()


def check(d, want):
    got = host(d)
    written = ~np.isnan(want)
    assert np.all(np.abs(got - want)[written] <= REL[d.dtype] * np.abs(want)[written] + ABS[d.dtype])
    assert np.all(np.isnan(got[~written])), "rows outside the problem were written"


def codes(rng, *shape):
    c = rng.integers(-128, 128, shape).astype(np.int8)
    return c, (rng.random(shape[:-1]) + 0.5).astype(np.float32) / 64


@pytest.mark.parametrize("rows,k", [(1, 16), (3, 48), (5, 128), (64, 1040), (7, 4096), (2, 4112), (9, 7168), (2, 40000)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_quantizer_is_exact(rows, k, dtype):
    rng = np.random.default_rng(rows * k)
    x = dev(rng.standard_normal((rows, k)).astype(np.float32) * 2).to(dtype)
    if rows > 2:
        x[0] = 0
        x[1] = torch.arange(k, device=device()) % 255 - 127.0   # codes hit .0 and, halved, .5 exactly
        x[2] = x[1] / 2
        x[2, 0] = 127
    say("int8 quantizer", rows, k, dtype)
    q, s = dg.dg_quantize_int8_per_token(x)
    wq, ws = oracle.int8.quantize(x.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(q.cpu().numpy(), wq)


def test_quantizer_of_values_that_are_not_finite():
    x = torch.ones((3, 64), device=device())
    x[0, 5] = float("nan")
    x[1, 9] = float("-inf")
    say("int8 quantizer, not finite")
    q, s = dg.dg_quantize_int8_per_token(x)
    assert torch.isnan(s[0]) and torch.isinf(s[1]) and s[2] == np.float32(1) / np.float32(127)
    w = torch.ones((8, 64), dtype=torch.int8, device=device())
    d = dg.dg_gemm_int8_nt(q, s, w, torch.ones(8, device=device()), out_dtype=F32)
    assert torch.isnan(d[:2]).all() and torch.isfinite(d[2]).all()
    q, s = dg.dg_quantize_int8_per_token(torch.empty((0, 64), device=device()))
    assert q.shape == (0, 64) and s.shape == (0,)


SHAPES = [  # m, n, k
    (1, 1, 16), (1, 7, 48), (1, 4096, 512), (2, 130, 1040), (3, 64, 7168), (5, 515, 144), (15, 257, 272), (16, 512, 2048),
    (17, 96, 528), (31, 1000, 256), (33, 129, 4112), (64, 2112, 7168), (65, 640, 112), (100, 31, 320), (127, 300, 128),
    (128, 128, 128), (129, 255, 384), (200, 1021, 176), (255, 512, 640), (257, 513, 2064), (384, 768, 512), (513, 1030, 400),
    (1024, 320, 1024), (1100, 1300, 272)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_gemm(m, n, k, dtype):
    rng = np.random.default_rng(m * 31 + n * 7 + k)
    (a, sa), (b, sb) = codes(rng, m, k), codes(rng, n, k)
    say("int8 gemm", m, n, k, dtype)
    want = oracle.int8.gemm_nt(a, sa, b, sb)
    da = [dev(v) for v in (a, sa, b, sb)]
    d = dg.dg_gemm_int8_nt(*da, out_dtype=dtype)
    check(d, want)
    # without a workspace, on a dirty output, and again: the same bits
    d2 = torch.full((m, n), float("nan"), dtype=dtype, device=device())
    dg.dg_gemm_int8_nt(*da, d=d2, use_workspace=False)
    assert torch.equal(d, d2) and torch.equal(d, dg.dg_gemm_int8_nt(*da, out_dtype=dtype))


def test_gemm_of_the_largest_sums():
    """K at its limit and every product at its largest: the sum stays inside int32."""
    k = 131056
    say("int8 gemm, largest sums")
    for m in (1, 40, 130):
        a = torch.full((m, k), -128, dtype=torch.int8, device=device())
        b = torch.full((150, k), -128, dtype=torch.int8, device=device())
        b[1] = 127
        d = dg.dg_gemm_int8_nt(a, torch.ones(m, device=device()), b, torch.ones(150, device=device()), out_dtype=F32)
        assert torch.all(d[:, 0] == float(128 * 128 * k)) and torch.all(d[:, 1] == float(np.float32(-128 * 127 * k)))
    with pytest.raises(dg.DGError):
        z = torch.zeros((2, 131072), dtype=torch.int8, device=device())
        dg.dg_gemm_int8_nt(z, torch.ones(2, device=device()), z, torch.ones(2, device=device()))


@pytest.mark.parametrize("m,n,k", [(1, 1, 16), (1, 2049, 7168), (2, 96, 1040), (4, 4096, 512), (5, 300, 2064), (8, 640, 16384),
                                   (16, 512, 400), (31, 257, 272), (64, 640, 4112), (200, 130, 528), (700, 1030, 1552)])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_in_call_quantization_is_the_two_calls(m, n, k, dtype):
    rng = np.random.default_rng(m + n + k)
    x = dev(rng.standard_normal((m, k)).astype(np.float32) * 3).to(dtype)
    if m > 3:
        x[2] = 0
        x[3, 1] = float("inf")
    b, sb = (dev(v) for v in codes(rng, n, k))
    say("int8 gemm with activation quantization", m, n, k, dtype)
    q, s = dg.dg_quantize_int8_per_token(x)
    for out in (F32, BF16, F16):
        want = dg.dg_gemm_int8_nt(q, s, b, sb, out_dtype=out)
        got = dg.dg_gemm_int8_nt_act_quant(x, b, sb, out_dtype=out)
        assert torch.equal(torch.nan_to_num(got.float(), nan=7e7), torch.nan_to_num(want.float(), nan=7e7))
    ws = torch.zeros(dg.dg_gemm_int8_nt_act_quant_workspace_size(m, n, k), dtype=torch.uint8, device=device())
    for _ in range(3):   # the counter prefix is left zero, and calls on one workspace follow each other
        got = dg.dg_gemm_int8_nt_act_quant(x, b, sb, out_dtype=out, workspace=ws)
        assert torch.equal(torch.nan_to_num(got.float(), nan=7e7), torch.nan_to_num(want.float(), nan=7e7))
        assert int(ws[:64 << 10].count_nonzero()) == 0
    if ws.numel() > 64 << 10:
        with pytest.raises(dg.DGError):
            dg.dg_gemm_int8_nt_act_quant(x, b, sb, workspace=ws[:64 << 10])


CONTIGUOUS = [  # experts of the 128-row blocks, n, k, groups
    ([0], 8, 16, 1), ([0, 0, 1, -1], 130, 272, 2), ([2, 0, 0, 7, -1, 1, 1], 257, 400, 3), ([0] * 6 + [1] * 5, 512, 1040, 2),
    ([-1, -1], 64, 64, 2), (list(range(9)), 300, 128, 9), ([3, -5, 2 ** 30, 1], 96, 528, 4)]


@pytest.mark.parametrize("blocks,n,k,groups", CONTIGUOUS)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_grouped_contiguous(blocks, n, k, groups, dtype):
    rng = np.random.default_rng(n + k)
    m = 128 * len(blocks)
    (a, sa), (b, sb) = codes(rng, m, k), codes(rng, groups, n, k)
    mi = np.repeat(np.array(blocks, dtype=np.int32), 128)
    say("int8 contiguous", blocks, n, k, dtype)
    d = torch.full((m, n), float("nan"), dtype=dtype, device=device())
    dg.dg_gemm_int8_grouped_contiguous(*(dev(v) for v in (a, sa, b, sb, mi)), d=d)
    check(d, oracle.int8.gemm_grouped_contiguous(a, sa, b, sb, mi))


MASKED = [  # m_max, counts, n, k
    (1, [1, 0, 1], 130, 272), (4, [4, -3, 9, 2], 64, 1040), (30, [0, 0, 17, 30, 1], 257, 528), (64, [64, 5], 512, 4112),
    (100, [33, 100, 0, 64], 96, 400), (130, [129, 130, 128, 1, 0], 300, 256), (256, [256, 0, 255, 1, 128, 129], 520, 640),
    (300, [299, 3], 129, 144)]


@pytest.mark.parametrize("m_max,counts,n,k", MASKED)
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_grouped_masked(m_max, counts, n, k, dtype):
    rng = np.random.default_rng(m_max + n + k)
    g = len(counts)
    (a, sa), (b, sb) = codes(rng, g, m_max, k), codes(rng, g, n, k)
    mm = np.array(counts, dtype=np.int32)
    say("int8 masked", m_max, counts, n, k, dtype)
    want = oracle.int8.gemm_grouped_masked(a, sa, b, sb, mm)
    args = [dev(v) for v in (a, sa, b, sb, mm)]
    for use in (True, False):
        d = torch.full((g, m_max, n), float("nan"), dtype=dtype, device=device())
        dg.dg_gemm_int8_grouped_masked(*args, d=d, use_workspace=use)
        check(d, want)


def test_under_a_cu_cap():
    """Plans for fewer compute units give the same bits."""
    rng = np.random.default_rng(3)
    cases = [(1, 700, 2064), (40, 300, 4112), (300, 520, 528), (513, 1030, 272)]
    ops = [[dev(v) for pair in (codes(rng, m, k), codes(rng, n, k)) for v in pair] for m, n, k in cases]
    want = [dg.dg_gemm_int8_nt(*o, out_dtype=F32) for o in ops]
    cus = dg.dg_get_num_cus()
    try:
        for cap in (1, 7, 64):
            say("int8 gemm under a CU cap", cap)
            dg.dg_set_num_cus(cap)
            for o, w in zip(ops, want):
                assert torch.equal(dg.dg_gemm_int8_nt(*o, out_dtype=F32), w)
    finally:
        dg.dg_set_num_cus(cus)


@pytest.mark.parametrize("m", [3, 16, 20, 32, 50, 64, 100, 128])
@pytest.mark.parametrize("n,k", [(1029, 2064), (390, 8336)])
def test_few_rows_on_every_strip_width(m, n, k):
    """The plans for fewer compute units take wider strips of the weights and other splits of K."""
    rng = np.random.default_rng(m + n)
    (a, sa), (b, sb) = codes(rng, m, k), codes(rng, n, k)
    want = oracle.int8.gemm_nt(a, sa, b, sb)
    args = [dev(v) for v in (a, sa, b, sb)]
    cus = dg.dg_get_num_cus()
    try:
        for cap in (1, 2, 4, 8, 11, 16, 32, cus):
            say("int8 gemm of few rows, strips under a CU cap", m, n, k, cap)
            dg.dg_set_num_cus(cap)
            for use in (True, False):
                d = torch.full((m, n), float("nan"), device=device())
                dg.dg_gemm_int8_nt(*args, d=d, use_workspace=use)
                check(d, want)
    finally:
        dg.dg_set_num_cus(cus)


def test_results_past_32_bit_offsets():
    m, n, k = 40000, 32768, 16
    say("int8 gemm, results past 32-bit offsets", m, n, k)
    gen = torch.Generator(device=device()).manual_seed(1)
    a = torch.randint(-127, 128, (m, k), generator=gen, device=device(), dtype=torch.int8)
    b = torch.randint(-127, 128, (n, k), generator=gen, device=device(), dtype=torch.int8)
    sa, sb = torch.rand(m, generator=gen, device=device()), torch.rand(n, generator=gen, device=device())
    d = dg.dg_gemm_int8_nt(a, sa, b, sb, out_dtype=F32)
    assert d.numel() * 4 > 2 ** 32
    for r in (0, m // 2 + 3, m - 1):
        check(d[r:r + 1], oracle.int8.gemm_nt(a[r:r + 1].cpu().numpy(), sa[r:r + 1].cpu().numpy(), b.cpu().numpy(),
                                             sb.cpu().numpy()))


def test_int8_graph_replays_match_eager():
    d = device()
    say("int8 graph")
    gen = torch.Generator(device=d).manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device=d)
    b, sb = dg.dg_quantize_int8_per_token(r(640, 4096))
    shapes = (1, 24, 300)
    xs = [r(m, 4096).to(BF16) for m in shapes]
    ws = [torch.zeros(dg.dg_gemm_int8_nt_act_quant_workspace_size(m, 640, 4096), dtype=torch.uint8, device=d) for m in shapes]
    outs = [torch.empty((m, 640), dtype=BF16, device=d) for m in shapes]
    step = lambda outs, ws: [dg.dg_gemm_int8_nt_act_quant(x, b, sb, d=o, workspace=w) for x, o, w in zip(xs, outs, ws)]
    step(outs, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs, ws)
    for seed in range(3):
        for x in xs:
            x.copy_(r(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        ref = [torch.empty_like(o) for o in outs]
        step(ref, [torch.zeros_like(w) for w in ws])
        torch.cuda.synchronize()
        for o, e in zip(outs, ref):
            assert torch.equal(o, e), seed
