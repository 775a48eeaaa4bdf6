"""Edges of expert rows and 8-bit integer GEMMs that need no GPU: the plain implementations at the smallest
values, sizes at the limits, and the plans."""

import ctypes

import numpy as np

import fp8_block_scaled_gemm_amd as dg
import oracle

UNSUPPORTED = -2


def test_plain_codes_of_the_smallest_rows_saturate():
    unit = np.float32(2.0 ** -149)
    rows = np.array([[190, -190, 95, 0], [143, 1, -142, 128], [63, -1, 0, 0], [64, -64, 32, 0], [127, -1, 2, 63]],
                    dtype=np.float32) * unit
    q, s = oracle.int8.quantize(rows)
    # amax / 127 in units of 2^-149, nearest even: 190/127 -> 1, 143/127 -> 1, 63/127 -> 0, 64/127 -> 1, 1
    assert (s / unit).tolist() == [1, 1, 0, 1, 1]
    assert q.tolist() == [[127, -127, 95, 0], [127, 1, -127, 127], [127, -127, 0, 0], [64, -64, 32, 0], [127, -1, 2, 63]]
    q, s = oracle.int8.quantize(np.array([[np.nan, 1], [np.inf, 1]], dtype=np.float32))
    assert q.tolist() == [[0, 0], [0, 0]] and np.isnan(s[0]) and np.isinf(s[1])


def test_quantizer_refuses_more_rows_than_a_grid_holds():
    """Checked before anything is launched, whatever the product of rows and threads wraps to."""
    lib, p = dg.lib(), ctypes.c_void_p(0x1000)
    for k, threads in ((64, 64), (4096, 256), (16384, 512)):
        for rows in (2 ** 32 // threads, (1 << 58) + 1, (1 << 62) + 1):
            assert lib.dg_quantize_int8_per_token(p, 1, rows, k, p, p, None) == UNSUPPORTED, (rows, k)
    assert lib.dg_quantize_int8_per_token(p, 1, 1, 1 << 31, p, p, None) == UNSUPPORTED
