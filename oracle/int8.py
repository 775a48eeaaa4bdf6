"""Plain NumPy 8-bit integer product: per-row quantizer and the three forms of the GEMM.

s = fl32(amax / 127) over a row (1 when amax = 0), q = nearest even integer of fl32(x / s), saturated to
[-127, 127] (a subnormal s is rounded so far that quotients pass them, or become infinite), 0 where x / s is
not a number;
D = (A * B^T) * sa[row] * sb[col], the integer sum exact, the scales in 64 bits.
"""

import numpy as np


def quantize(x):
    """(q int8 like x, s float32 per row)."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(axis=-1)
    s = np.where(amax == 0, np.float32(1), amax / np.float32(127)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint(x / s[..., None])
    return np.where(np.isnan(q), np.float32(0), np.clip(q, -127, 127)).astype(np.int8), s


def gemm_nt(a, sa, b, sb):
    exact = a.astype(np.int64) @ b.astype(np.int64).T if a.size * b.shape[0] < 1 << 24 else \
        a.astype(np.float64) @ b.astype(np.float64).T   # exact as well: sums below 2^53
    return exact * (sa.astype(np.float64)[:, None] * sb.astype(np.float64)[None, :])


def gemm_grouped_contiguous(a, sa, b, sb, m_indices):
    """Rows of an expert outside [0, G) are left NaN."""
    d = np.full((a.shape[0], b.shape[1]), np.nan)
    for g in range(b.shape[0]):
        who = np.flatnonzero(m_indices == g)
        if who.size:
            d[who] = gemm_nt(a[who], sa[who], b[g], sb[g])
    return d


def gemm_grouped_masked(a, sa, b, sb, masked_m):
    """Rows at or past masked_m (clamped to the buffer) are left NaN."""
    d = np.full((a.shape[0], a.shape[1], b.shape[1]), np.nan)
    for g in range(b.shape[0]):
        m = min(max(int(masked_m[g]), 0), a.shape[1])
        if m:
            d[g, :m] = gemm_nt(a[g, :m], sa[g, :m], b[g], sb[g])
    return d
