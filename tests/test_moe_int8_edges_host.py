"""Edges of expert rows and 8-bit integer GEMMs that need no GPU: the plain implementations at the smallest
values, sizes at the limits, and the plans."""

import numpy as np

import oracle


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
