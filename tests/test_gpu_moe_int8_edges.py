"""Expert rows and 8-bit integer GEMMs on the GPU where their arithmetic and their plans have edges: the
smallest rows and scales, values that are not finite, the longest rows, and every kernel that a plan can name.

Quantizers are compared byte for byte; a GEMM's tolerance is that of its arithmetic (the integer sum is
exact; its conversion and two products with the scales round in fp32, 3 * 2^-24, then the output's type:
2^-8 relative for bf16, 2^-11 for fp16 and 2^-25 absolute near zero, fp32 2^-149)."""

import os

import numpy as np
import pytest
import torch

import fp8_block_scaled_gemm_amd as dg
import oracle
from gpu_util import device, say

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = [F32, BF16, F16]
REL = {F32: 3 * 2.0 ** -24, BF16: 2.0 ** -8 + 4 * 2.0 ** -24, F16: 2.0 ** -11 + 4 * 2.0 ** -24}
ABS = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -24}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(device())


def host(t):
    return t.double().cpu().numpy()


def check(d, want):
    """Written values against `want` (64 bits); NaN in `want`: d has to be NaN there."""
    got, there = host(d), ~np.isnan(want)
    assert np.all(np.abs(got - want)[there] <= REL[d.dtype] * np.abs(want)[there] + ABS[d.dtype])
    assert np.all(np.isnan(got[~there]))


def codes(rng, *shape):
    c = rng.integers(-128, 128, shape).astype(np.int8)
    return c, (rng.random(shape[:-1]) + 0.5).astype(np.float32) / 64


# ---- the quantizer --------------------------------------------------------------------------------

TINY = np.float32(2.0 ** -149)
TINY_AMAX = [1, 2, 63, 64, 100, 127, 143, 178, 190, 191, 254, 1000, 16000, 16129, 127 << 16]   # in units of 2^-149


def tiny_rows(k):
    """Rows whose scale is zero or a subnormal of a few bits: amax of either sign, its halves and zeros."""
    x = np.zeros((2 * len(TINY_AMAX), k), dtype=np.float32)
    for i, units in enumerate(TINY_AMAX):
        a = np.float32(units) * TINY
        for row, sign in ((2 * i, 1), (2 * i + 1, -1)):
            x[row, 1::4] = sign * a
            x[row, 2::4] = -sign * np.float32(units // 2) * TINY
            x[row, 3] = -sign * a
    return x


@pytest.mark.parametrize("k", [48, 1040, 9232])
def test_codes_of_the_smallest_rows_saturate(k):
    x = tiny_rows(k)
    want, scale = oracle.int8.quantize(x)
    assert want.min() == -127 and want.max() == 127 and (scale == 0).any()
    say("int8 codes of the smallest rows", k)
    q, s = dg.dg_quantize_int8_per_token(dev(x))
    assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(q.cpu().numpy(), want)
    # the same codes from dispatch, and from the product that quantizes its one or two rows itself
    t = x.shape[0]
    lay = dg.dg_moe_layout(torch.zeros((t, 1), dtype=torch.int32, device=device()), 1)
    q2, s2 = dg.dg_moe_dispatch_int8(dev(x), lay)
    assert torch.equal(q2[:t], q) and torch.equal(s2[:t], s)
    b = torch.ones((16, k), dtype=torch.int8, device=device())
    sb = torch.full((16,), 2.0 ** 126, device=device())
    for r in range(0, t, 2):
        got = dg.dg_gemm_int8_nt_act_quant(dev(x[r:r + 2]), b, sb, out_dtype=F32)
        assert torch.equal(got, dg.dg_gemm_int8_nt(q[r:r + 2], s[r:r + 2], b, sb, out_dtype=F32)), r


def test_the_longest_rows():
    """A row of 2^31 - 16 elements: its last pieces lie where a 32-bit index is about to wrap."""
    k, d = 2 ** 31 - 16, device()
    say("int8 quantizer, longest row", k)
    x = torch.zeros((1, k), dtype=BF16, device=d)
    at = torch.tensor([0, 5, 16383, 16384, 2 ** 30 + 3, k - 4100, k - 4096, k - 9, k - 1], device=d)
    x[0, at] = torch.tensor([1.0, -3.0, 10.0, 127.0, -127.0, 0.4, 63.0, -2.0, 64.5], device=d).to(BF16)
    q, s = dg.dg_quantize_int8_per_token(x)
    assert s.item() == 1.0
    assert q[0, at].tolist() == [1, -3, 10, 127, -127, 0, 63, -2, 64]
    assert int(q.count_nonzero()) == 8


# ---- dispatch of values that are not finite -------------------------------------------------------

@pytest.mark.parametrize("tokens,top_k,hidden", [(20, 2, 400), (20, 2, 2064), (1300, 3, 2064 * 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_fp8_dispatch_of_values_that_are_not_finite_is_the_quantizer(tokens, top_k, hidden, dtype):
    """NaNs and infinities in a group, alone and together, in whole groups and in the partial last one."""
    rng = np.random.default_rng(hidden)
    x = rng.standard_normal((tokens, hidden)).astype(np.float32)
    nan, inf, last = np.nan, np.inf, hidden // 128 * 128
    x[0, 5] = nan
    x[1, [3, 77]] = nan, -nan
    x[2, 128:256] = nan                  # a group of NaNs alone
    x[3, last:] = nan                    # and the partial one
    x[4, 17], x[5, 200] = inf, -inf
    x[6, [1, 2, 300]] = nan, inf, nan
    x[7, 128:256] = 0
    x[7, 130] = nan                      # zeros and a NaN
    x[8, 0], x[8, hidden - 1] = nan, nan
    x[9, 384] = nan
    x[9, 385] = 3e38
    say("FP8 dispatch, not finite", tokens, top_k, hidden, dtype)
    d = dev(x).to(dtype)
    q, sa = dg.dg_quantize_per_token_group(d)
    ids = dev(np.argsort(rng.random((tokens, 5)), axis=1)[:, :top_k].astype(np.int32))
    for per in (0, 1 << 10):
        lay = dg.dg_moe_layout(ids, 5, rows_per_expert=per)
        gq, gs = dg.dg_moe_dispatch_fp8(d, lay)
        gq, gs = gq.view(-1, hidden), gs.view(-1, gs.shape[-2], gs.shape[-1])
        rows = lay.rows.long()
        token = torch.arange(tokens, device=device())[:, None].expand_as(rows)[rows >= 0]
        rows = rows[rows >= 0]
        assert torch.equal(gq[rows], q[token])
        got = gs[rows // per, :, rows % per] if per else gs[0][:, rows].t()
        want = sa[:, token].t()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, nan=-1.0), torch.nan_to_num(want, nan=-1.0))


# ---- layout ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("tokens,top_k,experts,per", [(1, 1, 1, 0), (3, 3, 5, 0), (7, 1, 6, 0), (5, 3, 7, 3), (1, 1, 1, 1),
                                                      (9, 5, 3, 33)])
def test_index_arrays_are_aligned(tokens, top_k, experts, per):
    """Every array of a layout starts at a multiple of 16 bytes, as the pointers that the GEMMs take."""
    say("alignment of a layout's arrays", tokens, top_k, experts, per)
    ids = np.random.default_rng(tokens).integers(0, experts, (tokens, top_k)).astype(np.int32)
    lay = dg.dg_moe_layout(dev(ids), experts, rows_per_expert=per)
    for name in ("rows", "sources", "counts") + (() if per else ("m_indices",)):
        assert getattr(lay, name).data_ptr() % 16 == 0, name
    rows, sources, m_indices, counts = oracle.moe.layout(ids, experts, per)
    assert np.array_equal(lay.rows.cpu().numpy(), rows) and np.array_equal(lay.counts.cpu().numpy(), counts)
    assert np.array_equal(lay.sources.cpu().numpy()[:len(sources)], sources)
    if not per:
        assert np.array_equal(lay.m_indices.cpu().numpy()[:len(m_indices)], m_indices)


# ---- scales far from one --------------------------------------------------------------------------

FAR = [1.0, 1e-34, 1e-6, 1e30, 1e-30, 1e10, 1e-10, 3e38, 1.2e-38, 0.0, 7 * 2.0 ** -149, 2.0 ** -133, 1e-20, 1e20, 1e-24]


def far_scales(rng, *shape):
    """Every pair of FAR meets where rows and columns count len(FAR) or more; some of them negative."""
    s = np.resize(np.array(FAR, dtype=np.float32), shape) * rng.choice([1, 1, -1], shape).astype(np.float32)
    return s.astype(np.float32)


def check_far(d, want):
    """As check, where a result past the type's range is the infinity of its sign."""
    got, top = host(d), float(torch.finfo(d.dtype).max)
    inside = np.abs(want) <= top * (1 - 2.0 ** -10)
    assert np.all(np.abs(got - want)[inside] <= (REL[d.dtype] * np.abs(want) + ABS[d.dtype])[inside])
    past = np.abs(want) >= top * (1 + 2.0 ** -7)
    assert np.array_equal(got[past], np.copysign(np.inf, want[past]))


@pytest.mark.parametrize("m,n,k", [(15, 64, 272), (33, 129, 2064), (128, 96, 400), (200, 130, 528), (513, 1030, 272)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_scales_far_from_one(m, n, k, dtype):
    """(sum * sa) * sb has a value where sa * sb does not: its product underflows, or overflows beside a small
    sum.  Rows of zero sums are 0 whatever the scales."""
    rng = np.random.default_rng(m + n)
    a, b = rng.integers(-128, 128, (m, k)).astype(np.int8), rng.integers(-128, 128, (n, k)).astype(np.int8)
    a[5] = 0
    a[6], b[7, 3] = 0, 1
    a[6, 3] = 1                          # sums of one code
    a[7] = a[6]
    sa, sb = far_scales(rng, m), far_scales(rng, n)
    sb = np.roll(sb, 4)
    sa[5], sa[7] = 3e38, 1e-38
    say("int8 scales far from one", m, n, k, dtype)
    args = [dev(v) for v in (a, sa, b, sb)]
    d = dg.dg_gemm_int8_nt(*args, out_dtype=dtype)
    check_far(d, oracle.int8.gemm_nt(a, sa, b, sb))
    assert torch.all(d[5] == 0)
    assert torch.equal(d, dg.dg_gemm_int8_nt(*args, out_dtype=dtype, use_workspace=False))
    # the grouped forms
    mi = np.repeat(np.array([1, 0, -1, 1], dtype=np.int32), 128)
    ga, gsa = rng.integers(-128, 128, (512, k)).astype(np.int8), far_scales(rng, 512)
    gb, gsb = rng.integers(-128, 128, (2, n, k)).astype(np.int8), np.roll(far_scales(rng, 2, n), 4, axis=1)
    d = torch.zeros((512, n), dtype=dtype, device=device())
    dg.dg_gemm_int8_grouped_contiguous(*(dev(v) for v in (ga, gsa, gb, gsb, mi)), d=d)
    check_far(d, np.nan_to_num(oracle.int8.gemm_grouped_contiguous(ga, gsa, gb, gsb, mi)))
    for m_max in (64, 256):
        ga, gsa = ga.reshape(-1)[:2 * m_max * k].reshape(2, m_max, k), gsa[:2 * m_max].reshape(2, m_max)
        mm = np.array([m_max, 17], dtype=np.int32)
        d = torch.zeros((2, m_max, n), dtype=dtype, device=device())
        dg.dg_gemm_int8_grouped_masked(*(dev(v) for v in (ga, gsa, gb, gsb, mm)), d=d)
        check_far(d, np.nan_to_num(oracle.int8.gemm_grouped_masked(ga, gsa, gb, gsb, mm)))
        ga, gsa = rng.integers(-128, 128, (512, k)).astype(np.int8), far_scales(rng, 512)


@pytest.mark.parametrize("rows", [1, 2, 5])
def test_scales_far_from_one_with_in_call_quantization(rows):
    rng = np.random.default_rng(rows)
    n, k = 300, 1040
    b, sb = rng.integers(-128, 128, (n, k)).astype(np.int8), np.roll(far_scales(rng, n), 4)
    for size in (1e-36, 1e-30, 1.0, 1e30, 3e37):
        x = (rng.standard_normal((rows, k)) * size).astype(np.float32)
        say("int8 scales far from one, in-call quantization", rows, size)
        a, sa = oracle.int8.quantize(x)
        want = oracle.int8.gemm_nt(a, sa, b, sb)
        for dtype in DTYPES:
            d = dg.dg_gemm_int8_nt_act_quant(dev(x), dev(b), dev(sb), out_dtype=dtype)
            check_far(d, want)
            assert torch.equal(d, dg.dg_gemm_int8_nt(dev(a), dev(sa), dev(b), dev(sb), out_dtype=dtype))


# ---- plans ----------------------------------------------------------------------------------------

class env:
    """Environment variables for the duration of a block (the library reads them per call); None: not set."""

    def __init__(self, **kv):
        self.kv = kv

    def _set(self, kv):
        for k, v in kv.items():
            if v is None:
                os.environ.pop(k, None)
            else:
                os.environ[k] = v

    def __enter__(self):
        self.old = {k: os.environ.get(k) for k in self.kv}
        self._set(self.kv)

    def __exit__(self, *exc):
        self._set(self.old)


def test_debug_log_of_int8_plans(capfd):
    """DG_DEBUG logs the plan of every form, the one that DG_PLAN asks for, and nothing without it."""
    rng = np.random.default_rng(1)
    say("int8 plan log")
    (a, sa), (b, sb) = codes(rng, 256, 512), codes(rng, 2, 300, 512)
    a, sa, b, sb = (dev(v) for v in (a, sa, b, sb))
    mi = torch.zeros(256, dtype=torch.int32, device=device())
    mm = torch.full((2,), 100, dtype=torch.int32, device=device())

    def run():
        dg.dg_gemm_int8_nt(a, sa, b[0], sb[0])
        dg.dg_gemm_int8_grouped_contiguous(a, sa, b, sb, mi)
        dg.dg_gemm_int8_grouped_masked(a.view(2, 128, 512), sa.view(2, 128), b, sb, mm)
        dg.dg_gemm_int8_nt_act_quant(a[:2].float(), b[0], sb[0])
        torch.cuda.synchronize()
        return capfd.readouterr().err

    with env(DG_DEBUG=None, DG_PLAN=None):
        capfd.readouterr()
        assert "int8 gemm" not in run()
    for plan in (None, "tile=256x256", "tile=128x128", "strip=64"):
        with env(DG_DEBUG="1", DG_PLAN=plan):
            err = run()
            for form, m, groups, layout in (("normal", 256, 1, 0), ("contiguous", 256, 2, 1), ("masked", 128, 2, 2)):
                name = dg.dg_gemm_int8_config_name(layout, m, 300, 512, groups)
                assert f"[dg] int8 gemm {form} m={m} n=300 k=512 groups={groups}: {name} " in err, (plan, err)
                if plan is not None and (plan != "strip=64" or layout != 1):
                    assert plan.split("=")[1] in name, (plan, name)
        assert "[dg] int8 gemm normal m=2 n=300 k=512 groups=1: direct16x16/4waves/split1 " in err, err


def test_debug_check_of_the_int8_contiguous_layout():
    """DG_DEBUG: a 128-row block of two experts and an expert out of range are reported; the rest is silent."""
    rng = np.random.default_rng(2)
    (a, sa), (b, sb) = codes(rng, 512, 272), codes(rng, 3, 130, 272)
    args = [dev(v) for v in (a, sa, b, sb)]
    valid = np.repeat(np.array([0, 1, -1, 2], np.int32), 128)
    mixed, far = valid.copy(), valid.copy()
    mixed[128 + 72] = 2
    far[384:] = 7
    say("int8 contiguous layout check")
    dg.dg_get_debug_status(clear=True)

    def status(m_indices):
        d = torch.full((512, 130), float("nan"), device=device())
        dg.dg_gemm_int8_grouped_contiguous(*args, dev(m_indices), d=d)
        return d, dg.dg_get_debug_status(clear=True)

    with env(DG_DEBUG="0"):
        assert status(mixed)[1] == (0, -1)
    with env(DG_DEBUG="1"):
        d, st = status(valid)
        assert st == (0, -1)
        check(d, oracle.int8.gemm_grouped_contiguous(a, sa, b, sb, valid))
        assert status(mixed)[1] == (dg.DG_DIAG_MIXED_BLOCK, 1)
        d, st = status(far)
        assert st == (dg.DG_DIAG_EXPERT_RANGE, 3)
        check(d, oracle.int8.gemm_grouped_contiguous(a, sa, b, sb, far))
    assert dg.dg_get_debug_status(clear=False) == (0, -1)


def test_one_or_two_rows_in_a_graph_without_a_workspace():
    d = device()
    say("int8 gemm of one and two rows, captured without a workspace")
    gen = torch.Generator(device=d).manual_seed(3)
    b, sb = dg.dg_quantize_int8_per_token(torch.randn((700, 2064), generator=gen, device=d))
    xs = [torch.randn((m, 2064), generator=gen, device=d).to(BF16) for m in (1, 2)]
    outs = [torch.empty((m, 700), dtype=BF16, device=d) for m in (1, 2)]
    step = lambda outs: [dg.dg_gemm_int8_nt_act_quant(x, b, sb, d=o) for x, o in zip(xs, outs)]
    step(outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(outs)
    for _ in range(3):
        for x in xs:
            x.copy_(torch.randn(x.shape, generator=gen, device=d))
        graph.replay()
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            q, s = dg.dg_quantize_int8_per_token(x)
            assert torch.equal(o, dg.dg_gemm_int8_nt(q, s, b, sb))


def test_few_rows_keep_to_the_cu_cap(capfd):
    """Under dg_set_num_cus no launch of the few-row kernels has more workgroups than the capped CUs hold (32 waves
    a CU), and the results stay the same bits."""
    rng = np.random.default_rng(4)
    shapes = [(1, 6200, 1040), (2, 3000, 7168), (16, 4096, 2064), (64, 4096, 4112), (100, 2050, 1040)]
    ops = [[dev(v) for pair in (codes(rng, m, k), codes(rng, n, k)) for v in pair] for m, n, k in shapes]
    masked = [dev(v) for pair in (codes(rng, 6, 40, 528), codes(rng, 6, 700, 528)) for v in pair]
    mm = dev(np.array([40, 0, 3, 17, 39, 33], np.int32))
    xs = [dev(rng.standard_normal((m, k)).astype(np.float32)) for m, _, k in shapes]

    def run():
        out = [dg.dg_gemm_int8_nt(*o, out_dtype=F32) for o in ops]
        out += [dg.dg_gemm_int8_nt_act_quant(x, o[2], o[3], out_dtype=F32) for x, o in zip(xs, ops)]
        d = torch.zeros((6, 40, 700), device=device())
        return out + [dg.dg_gemm_int8_grouped_masked(*masked, mm, d=d)]

    say("few-row int8 kernels under a CU cap")
    want = run()
    cus = dg.dg_get_num_cus()
    try:
        for cap in (1, 3, 8, 20, 100):
            dg.dg_set_num_cus(cap)
            with env(DG_DEBUG="1", DG_PLAN="strip=32"):
                capfd.readouterr()
                got = run()
                err = capfd.readouterr().err
            lines = [line for line in err.splitlines() if "int8 gemm" in line]
            assert len(lines) == len(want), err
            for line in lines:
                plan, workgroups = line.split(": ")[1].split()[0], int(line.split("workgroups=")[1].split()[0])
                waves = int(plan.split("/")[1][:-len("waves")])
                assert plan.startswith(("strip", "direct")), line
                assert workgroups <= cap * (32 // waves), line
            for a, b in zip(got, want):
                assert torch.equal(a, b), cap
    finally:
        dg.dg_set_num_cus(cus)


# ---- every kernel that a plan can name ------------------------------------------------------------

TILES = ["tile=256x256", "tile=128x128"]
# rows, columns, K: 1, 2, 3, 5, 8 and 9 blocks of 128 with a partial last one, edges on every side of a tile
TILE_SHAPES = [(1, 1, 16), (255, 257, 128), (300, 515, 256), (129, 250, 272), (256, 512, 640), (513, 300, 1024), (600, 259, 1040)]


@pytest.mark.parametrize("m,n,k", TILE_SHAPES)
@pytest.mark.parametrize("tile", TILES)
def test_tiles_and_their_splits(tile, m, n, k):
    rng = np.random.default_rng(m + n + k)
    (a, sa), (b, sb) = codes(rng, m, k), codes(rng, n, k)
    sa[::7] = far_scales(rng, m)[::7]     # some waves meet scales far from one, some do not
    want = oracle.int8.gemm_nt(a, sa, b, sb)
    args = [dev(v) for v in (a, sa, b, sb)]
    for dtype in DTYPES:
        first = None
        for splits in (1, 2, 3, 16):
            with env(DG_PLAN=f"{tile},splits={splits}"):
                kb = -(-k // 128)
                name = f"{tile[5:]}/8waves/split{-(-kb // -(-kb // splits))}"
                assert dg.dg_gemm_int8_config_name(0, m, n, k) == name
                say("int8 tiles", name, m, n, k, dtype)
                ws = torch.zeros(max(dg.dg_gemm_int8_workspace_size(m, n, k), 16), dtype=torch.uint8, device=device())
                for _ in range(2):        # the counters are left zero
                    d = torch.full((m, n), float("nan"), dtype=dtype, device=device())
                    dg.dg_gemm_int8_nt(*args, d=d, workspace=ws)
                    assert int(ws[:64 << 10].count_nonzero()) == 0
                    if first is None:
                        check_far(d, want)
                        first = d
                    assert torch.equal(d, first), (name, dtype)


# experts of the 128-row blocks of a call: both halves of a 256-row tile of one expert, of two, one or both
# unused, out of range, and a last tile of one block
TWO_EXPERTS = [[0, 1], [1, 1], [-1, 1], [1, -1], [-1, -1, 2], [0, 0, 1], [2, 0, 0, 7, -1, 1, 1], [0, 1, 2, 0, 1, 2, 2, 2],
               [-4, 2 ** 30, 0, 1, 1, 2, -1, 0, 0]]


@pytest.mark.parametrize("blocks", TWO_EXPERTS)
@pytest.mark.parametrize("tile", TILES)
def test_contiguous_tiles_of_two_experts(tile, blocks):
    rng = np.random.default_rng(len(blocks))
    m = 128 * len(blocks)
    mi = np.repeat(np.array(blocks, dtype=np.int32), 128)
    for n, k in ((257, 16), (300, 256), (512, 400), (130, 1040)):
        (a, sa), (b, sb) = codes(rng, m, k), codes(rng, 3, n, k)
        want = oracle.int8.gemm_grouped_contiguous(a, sa, b, sb, mi)
        args = [dev(v) for v in (a, sa, b, sb, mi)]
        with env(DG_PLAN=tile):
            assert dg.dg_gemm_int8_config_name(1, m, n, k, 3) == tile[5:] + "/8waves/split1"
            for dtype in DTYPES:
                say("int8 contiguous tiles", tile, blocks, n, k, dtype)
                d = torch.full((m, n), float("nan"), dtype=dtype, device=device())
                dg.dg_gemm_int8_grouped_contiguous(*args, d=d)
                check(d, want)


MASKED_COUNTS = [(300, [0, 1, 127, 128, 129, 255, 256, 257, 300, -3, 999]), (256, [256, 0, 255]), (60, [60, 0, 7, 33])]
STRIPS = ["strip=32", "strip=64", "strip=96", "strip=128"]   # 96 for at most 64 rows


@pytest.mark.parametrize("plan,m_max,counts", [(plan, m, c) for plan in TILES + STRIPS for m, c in MASKED_COUNTS
                                               if plan != "strip=96" or m <= 64])
def test_masked_on_every_plan(plan, m_max, counts):
    rng = np.random.default_rng(m_max)
    g, mm = len(counts), np.array(counts, dtype=np.int32)
    for n, k in ((257, 128), (300, 1040), (64, 2064)):
        (a, sa), (b, sb) = codes(rng, g, m_max, k), codes(rng, g, n, k)
        want = oracle.int8.gemm_grouped_masked(a, sa, b, sb, mm)
        args = [dev(v) for v in (a, sa, b, sb, mm)]
        for dtype in DTYPES:
            for splits in (1, 3):
                with env(DG_PLAN=f"{plan},splits={splits}"):
                    name = dg.dg_gemm_int8_config_name(2, m_max, n, k, g)
                    assert plan[5:] in name if plan in TILES else name.startswith("strip" + plan[6:] + "x"), name
                    say("int8 masked on", name, m_max, n, k, dtype)
                    d = torch.full((g, m_max, n), float("nan"), dtype=dtype, device=device())
                    dg.dg_gemm_int8_grouped_masked(*args, d=d)
                    check(d, want)


@pytest.mark.parametrize("strip,m", [(strip, m) for strip in (32, 64, 96, 128)
                                     for m in (1, 3, 16, 17, 32, 33, 64, 65, 128, 200) if strip != 96 or m <= 64])
def test_strips_and_their_splits(strip, m):
    rng = np.random.default_rng(m)
    for n, k in ((1, 16), (130, 400), (257, 2064), (100, 9232)):
        (a, sa), (b, sb) = codes(rng, m, k), codes(rng, n, k)
        want = oracle.int8.gemm_nt(a, sa, b, sb)
        args = [dev(v) for v in (a, sa, b, sb)]
        for splits, dtype in ((1, F32), (2, BF16), (5, F16), (16, F32)):
            with env(DG_PLAN=f"strip={strip},splits={splits}"):
                name = dg.dg_gemm_int8_config_name(0, m, n, k)
                assert name.startswith(f"strip{strip}x"), name
                say("int8 strips", name, m, n, k, dtype)
                d = torch.full((m, n), float("nan"), dtype=dtype, device=device())
                dg.dg_gemm_int8_nt(*args, d=d)
                check(d, want)


@pytest.mark.parametrize("m,n,k,name", [(1, 6200, 1040, "direct32x16/4waves"), (2, 6150, 7168, "direct32x16/8waves"),
                                        (1, 300, 16384, "direct16x16/16waves"), (2, 6150, 16384, "direct32x16/16waves"),
                                        (2, 129, 4096, "direct16x16/4waves"), (1, 515, 8192, "direct16x16/8waves"),
                                        (1, 6144, 4112, "direct32x16/8waves")])
@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_quantized_by_the_product_itself(m, n, k, name, dtype, capfd):
    rng = np.random.default_rng(n + k)
    x = dev(rng.standard_normal((m, k)).astype(np.float32) * 3).to(dtype)
    b, sb = (dev(v) for v in codes(rng, n, k))
    say("int8 gemm that quantizes its rows", name, m, n, k, dtype)
    a, sa = oracle.int8.quantize(x.float().cpu().numpy())
    want = oracle.int8.gemm_nt(a, sa, b.cpu().numpy(), sb.cpu().numpy())
    for out in DTYPES:
        capfd.readouterr()
        with env(DG_DEBUG="1"):
            d = dg.dg_gemm_int8_nt_act_quant(x, b, sb, out_dtype=out)
        if dg.dg_get_num_cus() == 256:
            assert f": {name}/split1 " in capfd.readouterr().err
        check(d, want)


# ---- rows that the last-level cache cannot hold ----------------------------------------------------

@pytest.mark.parametrize("tokens,top_k,hidden,dtype", [(70000, 2, 1024, BF16), (35000, 4, 1024, BF16),
                                                       (17000, 4, 2064, BF16), (9000, 8, 2064, F16), (35100, 1, 2064, F32)])
def test_combine_and_gradients_past_the_cache(tokens, top_k, hidden, dtype):
    """More than 256 MiB of rows: the nontemporal forms of combine and of its gradient.  Tolerances: a chain of
    top_k fused multiply-adds and one rounding; a sum of `hidden` products in lanes."""
    d = device()
    say("combine past the cache", tokens, top_k, hidden, dtype)
    gen = torch.Generator(device=d).manual_seed(tokens)
    ids = torch.argsort(torch.rand((tokens, 8), generator=gen, device=d), dim=1)[:, :top_k].int().contiguous()
    ids[5] = -1
    ids[11, 0] = -1
    lay = dg.dg_moe_layout(ids, 8)
    out = torch.randn((lay.rows_total, hidden), generator=gen, device=d).to(dtype)
    assert tokens * top_k * hidden * out.element_size() > 256 << 20
    w = torch.rand((tokens, top_k), generator=gen, device=d)
    dy = torch.randn((tokens, hidden), generator=gen, device=d).to(dtype)
    y = dg.dg_moe_combine(out, lay, weights=w)
    y1 = dg.dg_moe_combine(out, lay)
    dout, dw = dg.dg_moe_combine_grad(dy, out, lay, w, dout=torch.full_like(out, 9.0))
    rel = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}[dtype]
    chain = 2 * (top_k + 1) * 2.0 ** -24
    for t0 in range(0, tokens, 8192):
        t = slice(t0, min(t0 + 8192, tokens))
        rows = lay.rows[t].long()
        there = (rows >= 0).double().unsqueeze(-1)
        picked = out[rows.clamp_min(0)].double() * there
        for got, weight in ((y[t], w[t].double().unsqueeze(-1)), (y1[t], torch.ones_like(there))):
            want, size = (picked * weight).sum(1), (picked * weight).abs().sum(1)
            assert bool(((got.double() - want).abs() <= rel * want.abs() + ABS[dtype] + chain * size).all())
        products = picked * dy[t].double().unsqueeze(1)
        near = (hidden / 64 + 16) * 2.0 ** -24 * products.abs().sum(2) + 1e-37
        assert bool(((dw[t].double() - products.sum(2)).abs() <= near).all())
        want = dy[t].double().unsqueeze(1) * w[t].double().unsqueeze(-1) * there
        got = dout[rows.clamp_min(0)].double() * there
        assert bool(((got - want).abs() <= (rel + 2.0 ** -23) * want.abs() + ABS[dtype]).all())
    free = lay.sources < 0
    assert bool((dout[free & (lay.m_indices >= 0)] == 0).all()) and bool((dout[lay.m_indices < 0] == 9).all())


# ---- routing under masks of the type's lowest value ------------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_under_masks_of_the_lowest_value(score, dtype):
    """A mask that writes the type's lowest value leaves its expert available, last, and with no weight beside
    any other; a row of nothing else is shared evenly (softmax) or has no score left (sigmoid)."""
    rng = np.random.default_rng(8)
    low = torch.finfo(dtype).min
    x = dev(rng.standard_normal((40, 96)) * 2).to(dtype)
    x = torch.where(dev(rng.random((40, 96)) < 0.5), torch.full_like(x, low), x)
    x[3] = low
    x[4, 2:] = low
    x[5, 1:] = -np.inf
    x[5, 0] = low
    x[6, ::2], x[6, 1::2] = torch.finfo(dtype).max, low
    say("route under masks of the lowest value", score, dtype)
    for renorm in (True, False):
        ids, w = dg.dg_moe_route(x, 6, score=score, renormalize=renorm)
        want, _ = oracle.moe.route(host(x), 6, score=score, renormalize=renorm)
        if score == "softmax":            # compared by the logits, exactly
            assert np.array_equal(ids.cpu().numpy(), want)
        want = oracle.moe.weights_of(host(x), ids.cpu().numpy(), score, renorm, 1.0)
        np.testing.assert_allclose(host(w), want, rtol=80 * 2.0 ** -24, atol=1e-37)
        dx = dg.dg_moe_route_grad(torch.ones_like(w), x, ids, score=score, renormalize=renorm)
        want = oracle.moe.route_grad(np.ones(w.shape), host(x), ids.cpu().numpy(), score, renorm, 1.0)
        assert torch.isfinite(dx).all()
        assert np.all(np.abs(host(dx) - want) <= REL[dtype] * np.abs(want) + ABS[dtype] + 4 * 80 * 2.0 ** -24)


# ---- refusals of the binding ----------------------------------------------------------------------

def test_workspaces_and_layouts_that_the_kernels_cannot_read_are_refused():
    d = device()
    say("refused workspaces and layouts")
    rng = np.random.default_rng(6)
    (a, sa), (b, sb) = codes(rng, 40, 4112), codes(rng, 300, 4112)
    a, sa, b, sb = (dev(v) for v in (a, sa, b, sb))
    mm = torch.full((1,), 40, dtype=torch.int32, device=d)
    ids = torch.zeros((3000, 2), dtype=torch.int32, device=d)
    x = torch.ones((3000, 128), device=d)
    big = torch.zeros(1 << 22, dtype=torch.uint8, device=d)
    lay = dg.dg_moe_layout(ids, 4)
    for ws in (torch.zeros(1 << 21, dtype=torch.uint8), big[::2]):    # on the host; with gaps
        for call in (lambda: dg.dg_gemm_int8_nt(a, sa, b, sb, workspace=ws),
                     lambda: dg.dg_gemm_int8_nt_act_quant(x, b[:, :128].contiguous(), sb, workspace=ws),
                     lambda: dg.dg_gemm_int8_grouped_masked(a[None], sa[None], b[None], sb[None], mm, workspace=ws),
                     lambda: dg.dg_moe_layout(ids, 4, workspace=ws), lambda: dg.dg_moe_dispatch_fp8(x, lay, workspace=ws)):
            with pytest.raises(ValueError):
                call()
    # a layout made by hand: the same arrays are taken, others refused
    args = (lay.rows, lay.sources, lay.m_indices, lay.counts, lay.rows_total, 0, 4)
    mine = dg.MoeLayout(*args)
    assert torch.equal(dg.dg_moe_combine(dg.dg_moe_dispatch(x, mine), mine), 2 * x)
    for at, bad in ((0, lay.rows.long()), (0, lay.rows.cpu()), (0, lay.rows.view(-1)), (0, lay.rows.t()), (1, lay.sources[1:]),
                    (1, lay.sources.cpu()), (2, None), (2, lay.m_indices.long()), (3, lay.counts[:3]), (4, lay.rows_total - 1),
                    (5, 128), (5, -1)):
        with pytest.raises(ValueError):
            dg.MoeLayout(*(bad if i == at else v for i, v in enumerate(args)))
    masked = dg.dg_moe_layout(ids, 4, rows_per_expert=16)
    dg.MoeLayout(masked.rows, masked.sources, None, masked.counts, 64, 16, 4)
    with pytest.raises(ValueError):
        dg.MoeLayout(masked.rows, masked.sources, None, masked.counts, 64, 16, 5)
