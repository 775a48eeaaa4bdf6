"""Expert rows and 8-bit integer GEMMs on the GPU where their arithmetic and their plans have edges: the
smallest rows and scales, values that are not finite, the longest rows, and every kernel that a plan can name.

Quantizers are compared byte for byte; a GEMM's tolerance is that of its arithmetic (the integer sum is
exact; its conversion and two products with the scales round in fp32, 3 * 2^-24, then the output's type:
2^-8 relative for bf16, 2^-11 for fp16 and 2^-25 absolute near zero, fp32 2^-149)."""

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
