"""Edges of expert rows and 8-bit integer GEMMs that need no GPU: the plain implementations at the smallest
values, sizes at the limits, and the plans."""

import ctypes
import json
import os
import re
import subprocess
import sys

import numpy as np

import fp8_block_scaled_gemm_amd as dg
import oracle

UNSUPPORTED, WORKSPACE = -2, -3


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


# ---- plans of the 8-bit integer GEMMs --------------------------------------------------------------

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_QUERY = """
import json, sys
sys.path.insert(0, {root!r})
import fp8_block_scaled_gemm_amd as dg
dg.dg_set_num_cus({cus})
print(json.dumps([[c, dg.dg_gemm_int8_config_name(*c), dg.dg_gemm_int8_workspace_size(*c[1:]),
                   dg.dg_gemm_int8_nt_act_quant_workspace_size(*c[1:4])] for c in json.loads(sys.argv[1])]))
"""
NAME = re.compile(r"^(strip)?(\d+)x(\d+)/(\d+)waves/split(\d+)$")
COUNTERS = 64 * 1024


def plans(cases, cus=256, override=None):
    """{(layout, m, n, k, groups): (name, workspace, workspace with in-call quantization)}, in a process of its own:
    the cap that stands in for a device is process-wide."""
    env = {k: v for k, v in os.environ.items() if k != "DG_PLAN"}
    if override is not None:
        env["DG_PLAN"] = override
    r = subprocess.run([sys.executable, "-c", _QUERY.format(root=ROOT, cus=cus), json.dumps(cases)], capture_output=True,
                       text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr[-2000:]
    return {tuple(c): tuple(rest) for c, *rest in json.loads(r.stdout.strip().splitlines()[-1])}


def split_bytes(case, name):
    """Workspace of a plan: the counters and an int32 partial of every tile and split."""
    layout, m, n, _, groups = case
    _, bn, bm, _, splits = NAME.match(name).groups()
    bn, bm, splits = int(bn), int(bm), int(splits)
    tiles = -(-m // bm) * -(-n // bn) * (groups if layout == 2 else 1)
    return COUNTERS + tiles * splits * bn * bm * 4 if splits > 1 else 0


PLANS = {   # on 256 CUs
    (0, 1, 4096, 7168, 1): "strip32x16/8waves/split2", (0, 16, 7168, 16384, 1): "strip32x16/8waves/split1",
    (0, 64, 7168, 16384, 1): "strip128x64/8waves/split4", (0, 64, 24576, 7168, 1): "strip96x64/8waves/split1",
    (0, 128, 7168, 2048, 1): "strip32x128/4waves/split1", (0, 256, 4096, 7168, 1): "128x128/8waves/split4",
    (0, 4096, 4096, 7168, 1): "256x256/8waves/split1", (0, 16384, 7168, 16384, 1): "256x256/8waves/split1",
    (1, 65536, 4096, 7168, 32): "256x256/8waves/split1", (2, 256, 4096, 7168, 32): "256x256/8waves/split1",
    (2, 16, 7168, 2048, 8): "strip128x16/8waves/split1"}


def test_int8_plans_on_256_cus():
    got = plans([list(c) for c in PLANS])
    for case, name in PLANS.items():
        assert got[case][0] == name, (case, got[case])
        if case[0] != 1:
            assert got[case][1] == split_bytes(case, name), (case, got[case])
    assert dg.lib().dg_gemm_int8_config_name(3, 1, 1, 16, 1) == b"" == dg.lib().dg_gemm_int8_config_name(0, 1, 1, 24, 1)
    assert dg.lib().dg_gemm_int8_config_name(0, 1, 1, 131072, 1) == b""


def test_workspace_of_one_group_serves_the_masked_form():
    """The size asked for one group lets the masked form split K as well as the normal one."""
    nks = [(4096, 7168), (2112, 7168), (512, 4096), (7168, 2048)]
    cases = [[layout, m, n, k, 1] for layout in (0, 2) for m in (16, 64, 100, 300, 512, 1000) for n, k in nks]
    got = plans(cases)
    assert any(v[0].endswith("/split4") for c, v in got.items() if c[0] == 2)
    for case, (name, ws, _) in got.items():
        assert ws >= split_bytes(case, name), (case, name, ws)


def test_one_or_two_rows_need_no_workspace():
    cases = [[0, m, n, k, 1] for m in (1, 2, 3) for n in (1, 8, 24576) for k in (16, 7168, 16384, 16400)]
    for (_, m, n, k, _), (_, _, ws_quant) in plans(cases).items():
        assert (ws_quant == 0) == (m <= 2 and k <= 16384), (m, n, k, ws_quant)
    # and the call asks for none: it gets as far as the device, which is not there
    for m, status in ((3, WORKSPACE), (2, None), (1, None)):
        got = _act_quant_without_device(m)
        assert got != WORKSPACE if status is None else got == status, (m, got)


def _act_quant_without_device(m):
    """Status of the call without a workspace, in a process that sees no device."""
    code = f"""
import ctypes, sys
sys.path.insert(0, {ROOT!r})
import fp8_block_scaled_gemm_amd as dg
p = ctypes.c_void_p(0x1000)
dg.dg_set_num_cus(256)
print(dg.lib().dg_gemm_int8_nt_act_quant(p, 1, p, p, p, 1, {m}, 64, 128, None, 0, None))
"""
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120, env=env)
    assert r.returncode == 0, r.stderr[-2000:]
    return int(r.stdout.strip().splitlines()[-1])


def test_int8_plan_invariants():
    nks = [(1, 16), (128, 128), (512, 7168), (2112, 7168), (7168, 2048), (24576, 1536), (300, 16400), (2113, 131056)]
    cases = [[0, m, n, k, 1] for m in (1, 2, 17, 33, 64, 65, 128, 129, 300, 1000, 1025, 8192) for n, k in nks]
    cases += [[1, 512 * g, n, k, g] for g in (1, 4, 8) for n, k in nks]
    cases += [[2, m, n, k, g] for g in (1, 8, 32) for m in (5, 100, 256, 2000) for n, k in nks]
    for cus in (256, 64, 1):
        for case, (name, ws, ws_quant) in plans(cases, cus).items():
            layout, m, n, k, groups = case
            match = NAME.match(name)
            assert match, (case, name)
            strip, bn, bm, waves, splits = match.groups()
            bn, bm, waves, splits = int(bn), int(bm), int(waves), int(splits)
            if strip:
                assert layout != 1 and m <= 1024 and bn in (32, 64, 96, 128) and waves in (4, 8)
                assert bm == (16 if m <= 16 else 32 if m <= 32 else 64 if m <= 64 else 128) and (bn, bm) != (96, 128)
            else:
                assert (bn, bm, waves) in {(256, 256, 8), (128, 128, 8)} and (layout == 0 or splits == 1)
            assert 1 <= splits <= 16 and splits <= -(-k // 128)
            if layout == 0:
                codes = COUNTERS + -(-m * k // 256) * 256 + -(-m * 4 // 256) * 256
                assert m <= 2 and k <= 16384 or ws_quant >= codes + max(split_bytes(case, name) - COUNTERS, 0)
            if layout == 0 or groups > 1 and layout == 2:
                assert ws >= split_bytes(case, name), (case, name, ws)


def test_int8_plan_override():
    cases = [[0, 64, 2112, 7168, 1], [0, 4096, 2112, 7168, 1], [1, 4096, 2112, 7168, 4], [2, 100, 4096, 7168, 8]]
    dense, large, contiguous, masked = (tuple(c) for c in cases)
    base = plans(cases)
    got = plans(cases, override="strip=96,splits=3")
    assert got[dense][0] == "strip96x64/8waves/split3" and got[dense][1] == split_bytes(dense, got[dense][0])
    assert got[large][0].endswith("/split3") and not got[large][0].startswith("strip")    # more than 1024 rows
    assert got[contiguous][0] == base[contiguous][0]                                      # neither strips nor splits
    assert got[masked] == plans(cases, override="splits=3")[masked]                       # 96 is for at most 64 rows
    assert plans(cases, override="strip=64,splits=3")[masked][0] == "strip64x128/8waves/split3"
    got = plans(cases, override="tile=256x256")
    assert all(v[0].startswith("256x256/8waves/") for v in got.values())
    got = plans(cases, override="splits=5,tile=128x128")
    assert got[dense][0] == got[large][0] == "128x128/8waves/split5"                      # 56 K blocks in parts of 12
    assert got[contiguous][0] == got[masked][0] == "128x128/8waves/split1"
    assert plans(cases, override="splits=99")[dense][0].endswith("/split14")              # 16 at most, of 4 blocks each
    for junk in ("tile=64x64", "strip=48", "splits=0", "splits=-4", "nonsense", ",,", "tile="):
        assert plans(cases, override=junk) == base, junk
