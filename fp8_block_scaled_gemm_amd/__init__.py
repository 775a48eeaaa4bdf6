"""Python binding of libdg.so, the gfx950 FP8 block-scaled GEMM library.

Argument marshalling only: every step of the path runs in the HIP kernels of
libdg.so, called through its C ABI (``include/dg.h``).  PyTorch supplies
device memory and the current stream; nothing here computes.  If the library
is not built, every call raises - there is no fallback.

Functions carry the C names:

* ``dg_quantize_per_token_group(x)``  -> (q uint8 (M, K), sa float32 (ceil(K/128), ld_sa)); fp32 or
  bf16 x (the bf16 entry point is ``dg_quantize_per_token_group_bf16``)
* ``dg_quantize_per_block(w)``        -> (q uint8 like w, sb float32 ([G,] ceil(N/128), ceil(K/128)))
* ``dg_gemm_fp8_nt(a, sa, b, sb)``    -> d bf16 (M, N)
* ``dg_gemm_fp8_nt_act_quant(x, b, sb)`` -> d bf16 (M, N) from unquantized fp32 or bf16 x, its
  per-token-group quantization done inside the GEMM launch
* ``dg_gemm_fp8_grouped_contiguous(a, sa, b, sb, m_indices)``  -> d bf16 (M_total, N)
* ``dg_gemm_fp8_grouped_masked(a, sa, b, sb, masked_m)``       -> d bf16 (G, M_max, N)
* training-side layouts: ``dg_quantize_per_channel_group(x)`` -> (qt uint8 (K, M), st float32
  (ceil(M/128), ld_st)) in groups of 128 tokens per column, transposed (fp32 or bf16 x);
  ``dg_transpose_blocks(q, s)`` -> the block quantization of the transposed matrix;
  ``dg_gemm_fp8_nt_row_scaled(a, sa, b, sb)`` -> d bf16 (M, N) with per-row scales on both operands;
  ``dg_gemm_fp8_k_grouped_row_scaled(a, sa, b, sb, group_tokens)`` -> d bf16 (G, M, N), the MoE weight
  gradients over the contiguous layout
* expert routing and rows: ``dg_moe_route(logits, top_k)`` -> (ids, weights) and ``dg_moe_route_grad``;
  ``dg_moe_layout(ids, num_experts)`` -> the rows of the contiguous or masked layout (``MoeLayout``);
  ``dg_moe_dispatch`` / ``_fp8`` / ``_int8`` (x -> expert rows), ``dg_moe_combine`` (expert rows -> tokens)
  and ``dg_moe_combine_grad``
* 8-bit integer GEMMs (one scale per token, one per output channel): ``dg_quantize_int8_per_token(x)`` ->
  (q int8, s float32); ``dg_gemm_int8_nt``, ``dg_gemm_int8_nt_act_quant``,
  ``dg_gemm_int8_grouped_contiguous``, ``dg_gemm_int8_grouped_masked`` -> d bf16, fp16 or fp32
* utilities ``dg_get_num_cus``, ``dg_set_num_cus``,
  ``dg_get_m_alignment_for_contiguous_layout``, ``dg_get_scale_ld``,
  ``dg_gemm_workspace_size``.

Activation scales use the K-group-major layout of the library: ``sa[kb, row]``
(for the masked form ``sa[g, kb, row]``), row stride ``ld_sa = sa.shape[-1]``.
"""

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")

_lib = None
_lock = threading.Lock()

_c_int64 = ctypes.c_int64
_c_int = ctypes.c_int
_vp = ctypes.c_void_p

_SIGNATURES = {
    "dg_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "dg_last_error_message": (ctypes.c_char_p, []),
    "dg_quantize_per_token_group": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _c_int64, _vp]),
    "dg_quantize_per_token_group_bf16": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _c_int64,
                                                        _vp]),
    "dg_quantize_per_block": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _vp]),
    "dg_gemm_fp8_nt": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64,
                                      _vp, ctypes.c_size_t, _vp]),
    "dg_gemm_fp8_nt_no_alloc": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64,
                                               _vp]),
    "dg_gemm_fp8_nt_act_quant": (ctypes.c_int, [_vp, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _vp,
                                                ctypes.c_size_t, _vp]),
    "dg_gemm_fp8_nt_act_quant_bf16": (ctypes.c_int, [_vp, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _vp,
                                                     ctypes.c_size_t, _vp]),
    "dg_gemm_fp8_nt_act_quant_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64]),
    "dg_gemm_fp8_grouped_contiguous": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _vp, _c_int64, _vp,
                                                      _c_int64, _c_int64, _c_int64, _vp]),
    "dg_gemm_fp8_grouped_masked": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _vp, _vp, _c_int64,
                                                  _c_int64, _c_int64, _c_int64, _vp, ctypes.c_size_t, _vp]),
    "dg_gemm_fp8_nt_row_scaled": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _c_int64, _vp, _c_int64, _c_int64,
                                                 _c_int64, _vp, ctypes.c_size_t, _vp]),
    "dg_gemm_fp8_k_grouped_row_scaled": (ctypes.c_int, [_vp, _vp, _c_int64, _vp, _vp, _c_int64, _vp, _vp,
                                                        _c_int64, _c_int64, _c_int64, _c_int64, _vp, ctypes.c_size_t,
                                                        _vp]),
    "dg_quantize_per_channel_group": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _c_int64, _vp]),
    "dg_quantize_per_channel_group_bf16": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _c_int64,
                                                          _vp]),
    "dg_transpose_blocks": (ctypes.c_int, [_vp, _vp, _c_int64, _c_int64, _c_int64, _vp, _vp, _vp]),
    "dg_moe_route": (ctypes.c_int, [_vp, _c_int, _c_int64, _vp, _c_int64, _c_int64, _c_int64, _c_int64, _c_int64, _c_int,
                                    _c_int, _c_int, ctypes.c_float, _vp, _vp, _vp]),
    "dg_moe_route_grad": (ctypes.c_int, [_vp, _vp, _c_int, _c_int64, _vp, _c_int64, _c_int64, _c_int64, _c_int, _c_int,
                                         ctypes.c_float, _vp, _c_int64, _vp]),
    "dg_moe_layout_rows": (_c_int64, [_c_int64, _c_int64, _c_int64]),
    "dg_moe_layout_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64]),
    "dg_moe_layout": (ctypes.c_int, [_vp, _c_int64, _c_int64, _c_int64, _c_int64, _c_int64, _vp, _vp, _vp, _vp, _vp,
                                     ctypes.c_size_t, _vp]),
    "dg_moe_dispatch": (ctypes.c_int, [_vp, _c_int, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _c_int64, _c_int64, _vp,
                                       _vp]),
    "dg_moe_dispatch_fp8": (ctypes.c_int, [_vp, _c_int, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _c_int64, _c_int64,
                                           _vp, _vp, _c_int64, _vp, ctypes.c_size_t, _vp]),
    "dg_moe_dispatch_fp8_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64]),
    "dg_moe_dispatch_int8": (ctypes.c_int, [_vp, _c_int, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _c_int64, _c_int64,
                                            _vp, _vp, _vp]),
    "dg_moe_combine": (ctypes.c_int, [_vp, _c_int, _vp, _vp, _c_int64, _c_int64, _c_int64, _c_int64, _vp, _vp]),
    "dg_moe_combine_grad": (ctypes.c_int, [_vp, _vp, _c_int, _vp, _vp, _vp, _vp, _c_int64, _c_int64, _c_int64, _c_int64,
                                           _vp, _vp, _vp]),
    "dg_quantize_int8_per_token": (ctypes.c_int, [_vp, _c_int, _c_int64, _c_int64, _vp, _vp, _vp]),
    "dg_gemm_int8_nt": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int64, _c_int64, _c_int64, _vp,
                                       ctypes.c_size_t, _vp]),
    "dg_gemm_int8_nt_act_quant": (ctypes.c_int, [_vp, _c_int, _vp, _vp, _vp, _c_int, _c_int64, _c_int64, _c_int64, _vp,
                                                 ctypes.c_size_t, _vp]),
    "dg_gemm_int8_nt_act_quant_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64]),
    "dg_gemm_int8_grouped_contiguous": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _c_int64, _vp, _c_int, _c_int64, _c_int64,
                                                       _c_int64, _vp]),
    "dg_gemm_int8_grouped_masked": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _vp, _c_int64, _c_int64, _c_int64,
                                                   _c_int64, _vp, ctypes.c_size_t, _vp]),
    "dg_gemm_int8_config_name": (ctypes.c_char_p, [ctypes.c_int, _c_int64, _c_int64, _c_int64, _c_int64]),
    "dg_gemm_int8_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64, _c_int64]),
    "dg_get_num_cus": (ctypes.c_int, []),
    "dg_set_num_cus": (ctypes.c_int, [ctypes.c_int]),
    "dg_get_m_alignment_for_contiguous_layout": (ctypes.c_int, []),
    "dg_get_scale_ld": (_c_int64, [_c_int64]),
    "dg_gemm_workspace_size": (ctypes.c_size_t, [_c_int64, _c_int64, _c_int64, _c_int64]),
    "dg_gemm_config_name": (ctypes.c_char_p, [ctypes.c_int, _c_int64, _c_int64, _c_int64, _c_int64]),
    "dg_get_debug_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(_c_int64), ctypes.c_int]),
}

DG_DIAG_MIXED_BLOCK = 1
DG_DIAG_EXPERT_RANGE = 2
DG_DIAG_FQ_TIMEOUT = 4


def lib():
    """Load libdg.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"libdg.so is not built ({LIB_PATH}); run "
                                       "`python -m fp8_block_scaled_gemm_amd._build` first")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in _SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


class DGError(RuntimeError):
    def __init__(self, fn, status):
        L = lib()
        super().__init__(f"{fn}: {L.dg_status_string(status).decode()} "
                         f"({L.dg_last_error_message().decode()})")
        self.status = status


def _check(fn, status):
    if status != 0:
        raise DGError(fn, status)


# torch's own query of the current stream's handle (0.1 us; building a Stream object for it takes 2 us,
# a sixth of a small call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(device):
    if _raw_stream is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _stream(t):
    return _stream_handle(t.device)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _bytes(t):
    """View an FP8 tensor (uint8 or float8_e4m3fn) as uint8."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _require(cond, msg):
    if not cond:
        raise ValueError(msg)


def _dev(*ts):
    for t in ts:
        _require(t.is_cuda and t.is_contiguous(), "tensors must be contiguous CUDA (HIP) tensors")
    return ts[0].device


# ---------------------------------------------------------------------------
# utilities
# ---------------------------------------------------------------------------

def dg_get_num_cus():
    r = lib().dg_get_num_cus()
    _check("dg_get_num_cus", r if r < 0 else 0)
    return r


def dg_set_num_cus(n):
    _check("dg_set_num_cus", lib().dg_set_num_cus(int(n)))


def dg_get_m_alignment_for_contiguous_layout():
    return lib().dg_get_m_alignment_for_contiguous_layout()


def dg_get_scale_ld(rows):
    return lib().dg_get_scale_ld(int(rows))


def dg_gemm_workspace_size(m, n, k, num_groups=1):
    return lib().dg_gemm_workspace_size(int(m), int(n), int(k), int(num_groups))


def dg_gemm_config_name(layout, m, n, k, num_groups=1):
    """Tile configuration / K split the GEMM picks (layout 0 normal, 1 contiguous, 2 masked,
    3 row-scaled normal)."""
    return lib().dg_gemm_config_name(int(layout), int(m), int(n), int(k), int(num_groups)).decode()


def dg_get_debug_status(clear=True):
    """(flags, block): the sticky device diagnostics (DG_DIAG_* bits) of the current device and the
    first 128-row block a contiguous-layout check found wrong (-1 if none).  Synchronises."""
    flags, block = ctypes.c_uint32(0), _c_int64(-1)
    _check("dg_get_debug_status", lib().dg_get_debug_status(ctypes.byref(flags), ctypes.byref(block), int(clear)))
    return int(flags.value), int(block.value)


_ws_cache = {}
_ws_retired = []


def default_workspace(device, nbytes):
    """A zero-filled workspace for the current stream of `device`, grown on demand (the kernels
    leave its counters zeroed).  Calls that share a workspace must be ordered on one stream, so
    every (device, stream) pair gets its own.  A buffer that a larger request supersedes is kept
    alive until the process ends, never freed: a graph captured with it, or a kernel still queued
    on it, may use it later.  Inside graph capture there is no default workspace (a buffer made
    there would be zero-filled only when the graph runs): pass one created before the capture."""
    if nbytes == 0:
        return None
    dev = device if isinstance(device, torch.device) else torch.device(device)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if torch.cuda.is_current_stream_capturing():
        raise ValueError("no default workspace during graph capture: pass workspace= (a zero-filled uint8 "
                         "tensor of dg_gemm_workspace_size(...) bytes created before the capture)")
    key = (dev.index, _stream_handle(dev))
    ws = _ws_cache.get(key)
    if ws is None or ws.numel() < nbytes:
        if ws is not None:
            _ws_retired.append(ws)
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _ws_cache[key] = ws
    return ws


# ---------------------------------------------------------------------------
# quantizers
# ---------------------------------------------------------------------------

def dg_quantize_per_token_group(x, q=None, sa=None):
    """x float32 or bfloat16 (M, K) -> (q uint8 (M, K), sa float32 (K/128, ld_sa)); or x (G, M, K)
    -> (q (G, M, K), sa (G, K/128, ld_sa)) for the per-expert masked layout.  Runs on x's stream.
    bfloat16 input goes to dg_quantize_per_token_group_bf16 (same result as the widened fp32)."""
    _require(x.dtype in (torch.float32, torch.bfloat16) and x.dim() in (2, 3),
             "x must be float32 or bfloat16, (M, K) or (G, M, K)")
    grouped = x.dim() == 3
    g, m, k = (x.shape if grouped else (1,) + tuple(x.shape))
    kb = -(-k // 128)   # a last K group of k % 128 elements is partial
    if q is None:
        q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.empty(((g,) if grouped else ()) + (max(kb, 1), dg_get_scale_ld(m)),
                         dtype=torch.float32, device=x.device)
    q = _bytes(q)
    _dev(x, q, sa)
    name = "dg_quantize_per_token_group" + ("_bf16" if x.dtype == torch.bfloat16 else "")
    _check(name, getattr(lib(), name)(_ptr(x), g, m, k, _ptr(q), _ptr(sa), sa.shape[-1], _stream(x)))
    return q, sa


def dg_quantize_per_token_group_bf16(x, q=None, sa=None):
    """bfloat16 x (M, K) or (G, M, K) -> (q, sa): dg_quantize_per_token_group_bf16."""
    _require(x.dtype == torch.bfloat16, "x must be bfloat16")
    return dg_quantize_per_token_group(x, q=q, sa=sa)


def dg_quantize_per_block(w, q=None, sb=None):
    """w float32 (N, K) or (G, N, K) -> (q uint8, sb float32 ([G,] ceil(N/128), K/128))."""
    _require(w.dtype == torch.float32 and w.dim() in (2, 3), "w must be float32 (N, K) or (G, N, K)")
    grouped = w.dim() == 3
    g, n, k = (w.shape if grouped else (1,) + tuple(w.shape))
    nb, kb = -(-n // 128), max(-(-k // 128), 1)
    if q is None:
        q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    if sb is None:
        sb = torch.empty(((g,) if grouped else ()) + (nb, kb), dtype=torch.float32, device=w.device)
    q = _bytes(q)
    _dev(w, q, sb)
    _check("dg_quantize_per_block",
           lib().dg_quantize_per_block(_ptr(w), g, n, k, _ptr(q), _ptr(sb), _stream(w)))
    return q, sb


def dg_quantize_per_channel_group(x, qt=None, st=None):
    """x float32 or bfloat16 (M, K) -> (qt uint8 (K, M), st float32 (ceil(M/128), ld_st)): groups of 128
    consecutive tokens of one column, codes transposed (qt[col, tok] encodes x[tok, col]), scales in
    the activation-scale layout of x^T.  x (G, M, K) -> (qt (G, K, M), st (G, ceil(M/128), ld_st))."""
    _require(x.dtype in (torch.float32, torch.bfloat16) and x.dim() in (2, 3),
             "x must be float32 or bfloat16, (M, K) or (G, M, K)")
    grouped = x.dim() == 3
    g, m, k = (x.shape if grouped else (1,) + tuple(x.shape))
    mb = max(-(-m // 128), 1)
    if qt is None:
        qt = torch.empty(((g,) if grouped else ()) + (k, m), dtype=torch.uint8, device=x.device)
    if st is None:
        st = torch.empty(((g,) if grouped else ()) + (mb, dg_get_scale_ld(k)), dtype=torch.float32, device=x.device)
    qt = _bytes(qt)
    _dev(x, qt, st)
    name = "dg_quantize_per_channel_group" + ("_bf16" if x.dtype == torch.bfloat16 else "")
    _check(name, getattr(lib(), name)(_ptr(x), g, m, k, _ptr(qt), _ptr(st), st.shape[-1], _stream(x)))
    return qt, st


def dg_quantize_per_channel_group_bf16(x, qt=None, st=None):
    """bfloat16 x (M, K) or (G, M, K) -> (qt, st): dg_quantize_per_channel_group_bf16."""
    _require(x.dtype == torch.bfloat16, "x must be bfloat16")
    return dg_quantize_per_channel_group(x, qt=qt, st=st)


def dg_transpose_blocks(q, s, qt=None, st=None):
    """Block-quantized (q uint8 ([G,] R, C), s ([G,] ceil(R/128), ceil(C/128))) -> the same for the
    transposed matrix: (qt ([G,] C, R), st ([G,] ceil(C/128), ceil(R/128)))."""
    q = _bytes(q)
    _require(q.dim() in (2, 3) and s.dim() == q.dim() and s.dtype == torch.float32, "q (R, C) or (G, R, C), s float32")
    grouped = q.dim() == 3
    g, r, c = (q.shape if grouped else (1,) + tuple(q.shape))
    lead = (g,) if grouped else ()
    if qt is None:
        qt = torch.empty(lead + (c, r), dtype=torch.uint8, device=q.device)
    if st is None:
        st = torch.empty(lead + (s.shape[-1], s.shape[-2]), dtype=torch.float32, device=q.device)
    qt = _bytes(qt)
    _dev(q, s, qt, st)
    _check("dg_transpose_blocks", lib().dg_transpose_blocks(_ptr(q), _ptr(s), g, r, c, _ptr(qt), _ptr(st), _stream(q)))
    return qt, st


# ---------------------------------------------------------------------------
# GEMMs
# ---------------------------------------------------------------------------

def dg_gemm_fp8_nt(a, sa, b, sb, d=None, workspace=None, use_workspace=True):
    """D (M, N) bf16 = A (M, K) * B (N, K)^T with fine-grained scales and promoted accumulation."""
    a, b = _bytes(a), _bytes(b)
    m, k = a.shape
    n = b.shape[0]
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _dev(a, sa, b, sb, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, dg_gemm_workspace_size(m, n, k, 1))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("dg_gemm_fp8_nt",
           lib().dg_gemm_fp8_nt(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb), _ptr(d), m, n, k,
                                _ptr(workspace), ws_bytes, _stream(a)))
    return d


def dg_gemm_fp8_nt_no_alloc(a, sa, b, sb, d):
    """dg_gemm_fp8_nt with the split-K scratch held by the library (no workspace argument; the
    output d (M, N) bf16 must be given: this call allocates nothing)."""
    a, b = _bytes(a), _bytes(b)
    m, k = a.shape
    n = b.shape[0]
    _dev(a, sa, b, sb, d)
    _require(d.dtype == torch.bfloat16 and tuple(d.shape) == (m, n), "d must be bfloat16 (M, N)")
    _check("dg_gemm_fp8_nt_no_alloc",
           lib().dg_gemm_fp8_nt_no_alloc(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb), _ptr(d), m, n, k,
                                         _stream(a)))
    return d


def dg_gemm_fp8_nt_act_quant_workspace_size(m, n, k):
    return int(lib().dg_gemm_fp8_nt_act_quant_workspace_size(int(m), int(n), int(k)))


def dg_gemm_fp8_nt_act_quant(x, b, sb, d=None, workspace=None):
    """D (M, N) bf16 = A (M, K) * B (N, K)^T where (A, sa) is the per-token-group quantization of
    x (float32 or bfloat16 (M, K)), done inside the GEMM launch.  The workspace is required (by
    default a zero-filled one per device); the result is bit-identical to
    dg_quantize_per_token_group(x) followed by dg_gemm_fp8_nt."""
    _require(x.dtype in (torch.float32, torch.bfloat16) and x.dim() == 2, "x must be float32 or bfloat16 (M, K)")
    b = _bytes(b)
    m, k = x.shape
    n = b.shape[0]
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=x.device)
    _dev(x, b, sb, d)
    if workspace is None:
        workspace = default_workspace(x.device, dg_gemm_fp8_nt_act_quant_workspace_size(m, n, k))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    name = "dg_gemm_fp8_nt_act_quant" + ("_bf16" if x.dtype == torch.bfloat16 else "")
    _check(name, getattr(lib(), name)(_ptr(x), _ptr(b), _ptr(sb), _ptr(d), m, n, k, _ptr(workspace), ws_bytes,
                                      _stream(x)))
    return d


def dg_gemm_fp8_nt_act_quant_bf16(x, b, sb, d=None, workspace=None):
    """bfloat16 x (M, K): dg_gemm_fp8_nt_act_quant_bf16."""
    _require(x.dtype == torch.bfloat16, "x must be bfloat16")
    return dg_gemm_fp8_nt_act_quant(x, b, sb, d=d, workspace=workspace)


def dg_gemm_fp8_nt_row_scaled(a, sa, b, sb, d=None, workspace=None, use_workspace=True):
    """D (M, N) bf16 = A (M, K) * B (N, K)^T where both operands carry per-row group scales:
    sa (ceil(K/128), ld_sa >= M), sb (ceil(K/128), ld_sb >= N) - e.g. the weight gradient
    dW = dY^T X from dg_quantize_per_channel_group(dY) and dg_quantize_per_channel_group(X)."""
    a, b = _bytes(a), _bytes(b)
    m, k = a.shape
    n = b.shape[0]
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _dev(a, sa, b, sb, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, dg_gemm_workspace_size(m, n, k, 1))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("dg_gemm_fp8_nt_row_scaled",
           lib().dg_gemm_fp8_nt_row_scaled(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb), sb.shape[-1], _ptr(d),
                                           m, n, k, _ptr(workspace), ws_bytes, _stream(a)))
    return d


def dg_gemm_fp8_k_grouped_row_scaled(a, sa, b, sb, group_tokens, d=None, workspace=None, use_workspace=True):
    """MoE weight gradients: a (M, T) and b (N, T) per-channel-quantized over T tokens in the contiguous
    layout, group_tokens (host sequence of G counts, multiples of 128) -> d bf16 (G, M, N) with
    d[g] = a[:, seg_g] * b[:, seg_g]^T (zeros for an empty expert)."""
    a, b = _bytes(a), _bytes(b)
    m, t = a.shape
    n = b.shape[0]
    counts = [int(c) for c in group_tokens]
    g = len(counts)
    if d is None:
        d = torch.empty((g, m, n), dtype=torch.bfloat16, device=a.device)
    _dev(a, sa, b, sb, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, max([dg_gemm_workspace_size(m, n, c, 1) for c in counts if c] or [0]))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    arr = (ctypes.c_int64 * max(g, 1))(*counts)
    _check("dg_gemm_fp8_k_grouped_row_scaled",
           lib().dg_gemm_fp8_k_grouped_row_scaled(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb), sb.shape[-1],
                                                  _ptr(d), arr, g, m, n, t, _ptr(workspace), ws_bytes, _stream(a)))
    return d


def dg_gemm_fp8_grouped_contiguous(a, sa, b, sb, m_indices, d=None):
    """D (M_total, N): row r uses expert m_indices[r] of B (G, N, K)."""
    a, b = _bytes(a), _bytes(b)
    m, k = a.shape
    g, n, _ = b.shape
    if d is None:
        d = torch.empty((m, n), dtype=torch.bfloat16, device=a.device)
    _require(m_indices.dtype == torch.int32, "m_indices must be int32")
    _dev(a, sa, b, sb, m_indices, d)
    _check("dg_gemm_fp8_grouped_contiguous",
           lib().dg_gemm_fp8_grouped_contiguous(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb),
                                                _ptr(m_indices), g, _ptr(d), m, n, k, _stream(a)))
    return d


def dg_gemm_fp8_grouped_masked(a, sa, b, sb, masked_m, d=None, workspace=None, use_workspace=True):
    """D (G, M_max, N): expert g computes only its first masked_m[g] rows; the rest stay untouched."""
    a, b = _bytes(a), _bytes(b)
    g, m_max, k = a.shape
    n = b.shape[1]
    if d is None:
        d = torch.empty((g, m_max, n), dtype=torch.bfloat16, device=a.device)
    _require(masked_m.dtype == torch.int32, "masked_m must be int32")
    _dev(a, sa, b, sb, masked_m, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, dg_gemm_workspace_size(m_max, n, k, g))
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("dg_gemm_fp8_grouped_masked",
           lib().dg_gemm_fp8_grouped_masked(_ptr(a), _ptr(sa), sa.shape[-1], _ptr(b), _ptr(sb), _ptr(d),
                                            _ptr(masked_m), g, m_max, n, k, _ptr(workspace), ws_bytes,
                                            _stream(a)))
    return d


# ---------------------------------------------------------------------------
# expert routing and the expert row layout
# ---------------------------------------------------------------------------

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_SCORES = {"softmax": 0, "sigmoid": 1}


def _dtype(t, what):
    code = _DTYPES.get(t if isinstance(t, torch.dtype) else t.dtype)
    _require(code is not None, f"{what} must be float32, bfloat16 or float16")
    return code


def _logit_rows(logits):
    """(tokens, experts, row stride) of a 2-D tensor whose rows are contiguous, whatever their distance."""
    _require(logits.dim() == 2 and logits.is_cuda, "logits must be a CUDA (HIP) tensor (tokens, experts)")
    t, e = logits.shape
    _require(e > 0 and (logits.stride(1) == 1 or e == 1), "the logits of a token must be contiguous")
    ld = logits.stride(0) if t > 1 else e
    _require(ld >= e, "the rows of logits must not overlap")
    return t, e, ld


def dg_moe_route(logits, top_k, bias=None, num_groups=1, topk_groups=1, group_top=1, score="softmax", renormalize=True,
                 scale=1.0, ids=None, weights=None):
    """Expert choice from logits (T, E) float32 / bfloat16 / float16 (rows may be strided) ->
    (ids int32 (T, top_k), weights float32 (T, top_k)).  `bias` float32 (E,) decides the choice only;
    with num_groups > 1 the topk_groups best groups (by their group_top best experts) stay.  -inf
    switches an expert off; id -1 and weight 0 where fewer than top_k are available."""
    t, e, ld = _logit_rows(logits)
    _require(score in _SCORES, "score must be 'softmax' or 'sigmoid'")
    if ids is None:
        ids = torch.empty((t, top_k), dtype=torch.int32, device=logits.device)
    else:
        _dev(ids)
        _require(ids.dtype == torch.int32 and tuple(ids.shape) == (t, top_k), "ids must be int32 (tokens, top_k)")
    if weights is None:
        weights = torch.empty((t, top_k), dtype=torch.float32, device=logits.device)
    else:
        _dev(weights)
        _require(weights.dtype == torch.float32 and tuple(weights.shape) == (t, top_k),
                 "weights must be float32 (tokens, top_k)")
    if bias is not None:
        _dev(bias)
        _require(bias.dtype == torch.float32 and tuple(bias.shape) == (e,), "bias must be float32 (experts,)")
    _check("dg_moe_route",
           lib().dg_moe_route(_ptr(logits), _dtype(logits, "logits"), ld, _ptr(bias), t, e, top_k, num_groups, topk_groups,
                              group_top, _SCORES[score], int(renormalize), scale, _ptr(ids), _ptr(weights),
                              _stream(logits)))
    return ids, weights


def dg_moe_route_grad(dweights, logits, ids, score="softmax", renormalize=True, scale=1.0, dlogits=None):
    """Gradient of dg_moe_route's weights with respect to its logits (the choice ids held fixed):
    dweights float32 (T, top_k) -> dlogits (T, E) in the logits' type."""
    t, e, ld = _logit_rows(logits)
    _require(score in _SCORES, "score must be 'softmax' or 'sigmoid'")
    _dev(dweights, ids)
    _require(ids.dtype == torch.int32 and ids.dim() == 2 and ids.shape[0] == t, "ids must be int32 (tokens, top_k)")
    _require(dweights.dtype == torch.float32 and dweights.shape == ids.shape, "dweights must be float32 (tokens, top_k)")
    if dlogits is None:
        dlogits = torch.empty((t, e), dtype=logits.dtype, device=logits.device)
    _require(dlogits.dtype == logits.dtype and tuple(dlogits.shape) == (t, e), "dlogits must be like logits")
    ld_out = _logit_rows(dlogits)[2]
    _check("dg_moe_route_grad",
           lib().dg_moe_route_grad(_ptr(dweights), _ptr(logits), _dtype(logits, "logits"), ld, _ptr(ids), t, e, ids.shape[1],
                                   _SCORES[score], int(renormalize), scale, _ptr(dlogits), ld_out, _stream(logits)))
    return dlogits


def dg_moe_layout_rows(tokens, top_k, experts):
    """Rows that the contiguous layout of any choice of experts fits in."""
    return lib().dg_moe_layout_rows(int(tokens), int(top_k), int(experts))


def dg_moe_layout_workspace_size(tokens, top_k, experts):
    return lib().dg_moe_layout_workspace_size(int(tokens), int(top_k), int(experts))


class MoeLayout:
    """Rows of the (token, k) entries of a batch: rows int32 (T, top_k) (-1: none), sources int32
    (rows_total,) (the inverse), m_indices int32 (rows_total,) for the contiguous grouped GEMMs (None in
    the masked layout), counts int32 (experts,) (masked_m of the masked ones).  rows_per_expert is 0 in
    the contiguous layout.  Made by dg_moe_layout, or by hand from arrays of those kinds."""

    __slots__ = ("rows", "sources", "m_indices", "counts", "rows_total", "rows_per_expert", "num_experts")

    def __init__(self, rows, sources, m_indices, counts, rows_total, rows_per_expert, num_experts, _check=True):
        if _check:
            arrays = [rows, sources, counts] + ([] if m_indices is None else [m_indices])
            _dev(*arrays)
            _require(all(a.dtype == torch.int32 and a.device == rows.device for a in arrays),
                     "the arrays of a layout must be int32, on one device")
            _require(rows_per_expert >= 0 and (m_indices is None) == (rows_per_expert > 0) and
                     (not rows_per_expert or rows_total == num_experts * rows_per_expert),
                     "m_indices for the contiguous layout, num_experts * rows_per_expert rows for the masked one")
            _require(rows.dim() == 2 and sources.numel() == rows_total and counts.numel() == num_experts and
                     (m_indices is None or m_indices.numel() == rows_total),
                     "rows (tokens, top_k), sources and m_indices (rows_total,), counts (num_experts,)")
        self.rows, self.sources, self.m_indices, self.counts = rows, sources, m_indices, counts
        self.rows_total, self.rows_per_expert, self.num_experts = rows_total, rows_per_expert, num_experts

    def lead(self):
        """Leading dimensions of this layout's row data."""
        return (self.num_experts, self.rows_per_expert) if self.rows_per_expert else (self.rows_total,)


def dg_moe_layout(ids, num_experts, rows_per_expert=0, rows_total=None, workspace=None):
    """ids int32 (T, top_k) -> MoeLayout: the contiguous layout (rows_per_expert = 0; rows_total rows,
    by default what any choice fits in) or the masked one (rows_per_expert rows per expert, entries
    past them dropped).  Runs on the device without a host synchronisation."""
    _require(ids.dim() == 2 and ids.dtype == torch.int32, "ids must be int32 (tokens, top_k)")
    _dev(ids)
    t, k = ids.shape
    dev, L = ids.device, lib()
    if rows_total is None:
        rows_total = num_experts * rows_per_expert if rows_per_expert else L.dg_moe_layout_rows(t, k, num_experts)
    # one allocation for the index arrays, each at a multiple of 16 bytes (as every pointer of the GEMMs)
    n, contiguous = t * k, not rows_per_expert
    _require(n >= 0 and rows_total >= 0 and num_experts >= 1, "sizes must not be negative")
    e4, r4 = num_experts + -num_experts % 4, rows_total + -rows_total % 4
    if contiguous:
        buf = torch.empty(2 * r4 + e4 + n, dtype=torch.int32, device=dev)
        sources, m_indices, counts, rows = buf.split((r4, r4, e4, n))
    else:
        buf = torch.empty(r4 + e4 + n, dtype=torch.int32, device=dev)
        (sources, counts, rows), m_indices = buf.split((r4, e4, n)), None
    if e4 != num_experts:
        counts = counts[:num_experts]
    if r4 != rows_total:   # (the masked layout's; the other's rows are a multiple of 128, or refused)
        sources = sources[:rows_total]
    rows = rows.view(t, k)
    if workspace is None:
        need = L.dg_moe_layout_workspace_size(t, k, num_experts)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check("dg_moe_layout",
           L.dg_moe_layout(_ptr(ids), t, k, num_experts, rows_per_expert, rows_total, _ptr(rows), _ptr(sources),
                           _ptr(m_indices), _ptr(counts), *_ws(workspace), _stream(ids)))
    return MoeLayout(rows, sources, m_indices, counts, rows_total, rows_per_expert, num_experts, _check=False)


def _dispatch_args(x, layout):
    _require(x.dim() == 2 and x.shape[0] == layout.rows.shape[0], "x must be (tokens, hidden) for the layout's tokens")
    t, h = x.shape
    return (_ptr(x), _dtype(x, "x"), _ptr(layout.rows), _ptr(layout.sources), _ptr(layout.m_indices), t,
            layout.rows.shape[1], h, layout.rows_total, layout.rows_per_expert)


def dg_moe_dispatch(x, layout, out=None):
    """x (T, H) -> the layout's rows (rows_total, H) or (experts, rows_per_expert, H), in x's type; the
    contiguous layout's padding rows are zeros.  Gradient with respect to x: dg_moe_combine(dout, layout)."""
    if out is None:
        out = torch.empty((*layout.lead(), x.shape[-1]), dtype=x.dtype, device=x.device)
    _dev(x, out)
    _require(out.dtype == x.dtype and out.numel() == layout.rows_total * x.shape[-1], "out must hold the layout's rows")
    _check("dg_moe_dispatch", lib().dg_moe_dispatch(*_dispatch_args(x, layout), _ptr(out), _stream(x)))
    return out


def dg_moe_dispatch_fp8_workspace_size(tokens, top_k, hidden):
    return lib().dg_moe_dispatch_fp8_workspace_size(int(tokens), int(top_k), int(hidden))


def dg_moe_dispatch_fp8(x, layout, q=None, sa=None, workspace=None):
    """x (T, H) -> (q uint8 rows, sa float32 (ceil(H/128), ld_sa) per matrix): the layout's rows as
    dg_quantize_per_token_group would quantize them, ready for the grouped FP8 GEMMs."""
    h, lead = x.shape[-1], layout.lead()
    if q is None:
        q = torch.empty((*lead, h), dtype=torch.uint8, device=x.device)
    if sa is None:
        sa = torch.empty((*lead[:-1], -(-h // 128), dg_get_scale_ld(lead[-1])), dtype=torch.float32, device=x.device)
    q = _bytes(q)
    _dev(x, q, sa)
    _require(q.dtype == torch.uint8 and q.numel() == layout.rows_total * h, "q must be uint8 and hold the layout's rows")
    _require(sa.dtype == torch.float32 and tuple(sa.shape[:-1]) == (*lead[:-1], -(-h // 128)), "sa must be float32, K-group-major")
    if workspace is None:
        need = lib().dg_moe_dispatch_fp8_workspace_size(x.shape[0], layout.rows.shape[1], h)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _check("dg_moe_dispatch_fp8",
           lib().dg_moe_dispatch_fp8(*_dispatch_args(x, layout), _ptr(q), _ptr(sa), sa.shape[-1], *_ws(workspace),
                                     _stream(x)))
    return q, sa


def dg_moe_dispatch_int8(x, layout, q=None, s=None):
    """x (T, H) -> (q int8 rows, s float32 per row): the layout's rows as dg_quantize_int8_per_token would
    quantize them, ready for the grouped int8 GEMMs."""
    h, lead = x.shape[-1], layout.lead()
    if q is None:
        q = torch.empty((*lead, h), dtype=torch.int8, device=x.device)
    if s is None:
        s = torch.empty(lead, dtype=torch.float32, device=x.device)
    _dev(x, q, s)
    _require(q.dtype == torch.int8 and q.numel() == layout.rows_total * h, "q must be int8 and hold the layout's rows")
    _require(s.dtype == torch.float32 and s.numel() == layout.rows_total, "s must be float32, one per row")
    _check("dg_moe_dispatch_int8", lib().dg_moe_dispatch_int8(*_dispatch_args(x, layout), _ptr(q), _ptr(s), _stream(x)))
    return q, s


def _check_weights(weights, layout):
    _dev(weights)
    _require(weights.dtype == torch.float32 and weights.shape == layout.rows.shape, "weights must be float32 (tokens, top_k)")


def dg_moe_combine(out, layout, weights=None, y=None):
    """y (T, H) = sum over k of weights[t, k] * out[row(t, k)], out holding the layout's rows (weights
    None: 1, the gradient of dg_moe_dispatch)."""
    t, k = layout.rows.shape
    h = out.shape[-1]
    _require(out.numel() == layout.rows_total * h, "out must hold the layout's rows")
    if y is None:
        y = torch.empty((t, h), dtype=out.dtype, device=out.device)
    _dev(out, y)
    _require(y.dtype == out.dtype and tuple(y.shape) == (t, h), "y must be (tokens, hidden) in out's type")
    if weights is not None:
        _check_weights(weights, layout)
    _check("dg_moe_combine",
           lib().dg_moe_combine(_ptr(out), _dtype(out, "out"), _ptr(layout.rows), _ptr(weights), t, k, h, layout.rows_total,
                                _ptr(y), _stream(out)))
    return y


def dg_moe_combine_grad(dy, out, layout, weights, dout=None, dweights=None):
    """Gradients of dg_moe_combine(out, layout, weights) from dy (T, H) -> (dout like out, dweights
    float32 (T, top_k)); the contiguous layout's padding rows of dout are zeros, rows that belong to no
    token otherwise untouched."""
    t, k = layout.rows.shape
    h = out.shape[-1]
    _require(out.numel() == layout.rows_total * h and tuple(dy.shape) == (t, h) and dy.dtype == out.dtype,
             "dy must be (tokens, hidden) and out hold the layout's rows, in one type")
    if dout is None:
        dout = torch.empty_like(out)
    if dweights is None:
        dweights = torch.empty((t, k), dtype=torch.float32, device=out.device)
    _dev(dy, out, dout)
    _require(dout.dtype == out.dtype and dout.numel() == out.numel(), "dout must be like out")
    _check_weights(weights, layout)
    _check_weights(dweights, layout)
    _check("dg_moe_combine_grad",
           lib().dg_moe_combine_grad(_ptr(dy), _ptr(out), _dtype(out, "out"), _ptr(layout.rows), _ptr(layout.sources),
                                     _ptr(layout.m_indices), _ptr(weights), t, k, h, layout.rows_total, _ptr(dout),
                                     _ptr(dweights), _stream(out)))
    return dout, dweights


# ---------------------------------------------------------------------------
# 8-bit integer GEMMs
# ---------------------------------------------------------------------------

def dg_gemm_int8_workspace_size(m, n, k, num_groups=1):
    return lib().dg_gemm_int8_workspace_size(int(m), int(n), int(k), int(num_groups))


def dg_gemm_int8_config_name(layout, m, n, k, num_groups=1):
    """Tile or strip and K split that the int8 GEMM picks (layout 0 normal, 1 contiguous, 2 masked)."""
    return lib().dg_gemm_int8_config_name(int(layout), int(m), int(n), int(k), int(num_groups)).decode()


def dg_gemm_int8_nt_act_quant_workspace_size(m, n, k):
    return lib().dg_gemm_int8_nt_act_quant_workspace_size(int(m), int(n), int(k))


def dg_quantize_int8_per_token(x, q=None, s=None):
    """x float32 / bfloat16 / float16 (..., K) -> (q int8 like x, s float32 (...)): one scale per row, for
    activations (per token) and weights (N, K) or (G, N, K) (per output channel)."""
    _require(x.dim() >= 1, "x must have rows")
    k = x.shape[-1]
    if q is None:
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    if s is None:
        s = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _dev(x, q, s)
    _require(q.dtype == torch.int8 and q.shape == x.shape, "q must be int8 like x")
    _require(s.dtype == torch.float32 and s.shape == x.shape[:-1], "s must be float32, one per row")
    _check("dg_quantize_int8_per_token",
           lib().dg_quantize_int8_per_token(_ptr(x), _dtype(x, "x"), s.numel(), k, _ptr(q), _ptr(s), _stream(x)))
    return q, s


def _check_int8(a, sa, b, sb):
    _require(a.dtype == torch.int8 and b.dtype == torch.int8, "a and b must be int8")
    _require(sa.dtype == torch.float32 and sb.dtype == torch.float32, "sa and sb must be float32")
    _require(sa.shape == a.shape[:-1] and sb.shape == b.shape[:-1] and a.shape[-1] == b.shape[-1],
             "sa: one scale per row of a, sb: one per row of b, the same K")


def _int8_out(d, shape, out_dtype, device):
    if d is None:
        return torch.empty(shape, dtype=out_dtype, device=device)
    _require(tuple(d.shape) == shape, f"d must be {shape}")
    return d


def _ws(workspace):
    """(pointer, bytes) of a caller's workspace, or of none."""
    if workspace is None:
        return None, 0
    _dev(workspace)
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def dg_gemm_int8_nt(a, sa, b, sb, d=None, out_dtype=torch.bfloat16, workspace=None, use_workspace=True):
    """D (M, N) = (A (M, K) * B (N, K)^T) * sa[m] * sb[n] from int8 codes, in d's or out_dtype's type
    (bfloat16, float16 or float32)."""
    _require(a.dim() == 2 and b.dim() == 2, "a (M, K), b (N, K)")
    _check_int8(a, sa, b, sb)
    m, k = a.shape
    n = b.shape[0]
    d = _int8_out(d, (m, n), out_dtype, a.device)
    _dev(a, sa, b, sb, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, lib().dg_gemm_int8_workspace_size(m, n, k, 1))
    _check("dg_gemm_int8_nt",
           lib().dg_gemm_int8_nt(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), _dtype(d, "d"), m, n, k, *_ws(workspace),
                                 _stream(a)))
    return d


def dg_gemm_int8_nt_act_quant(x, b, sb, d=None, out_dtype=torch.bfloat16, workspace=None):
    """D (M, N) from unquantized x (M, K) float32 / bfloat16 / float16: dg_quantize_int8_per_token(x) and
    dg_gemm_int8_nt in one call, the same bits.  The workspace is required (by default one per device
    and stream) for more than two rows or 16384 elements a row."""
    _require(x.dim() == 2 and b.dim() == 2 and b.dtype == torch.int8 and x.shape[1] == b.shape[1], "x (M, K), b int8 (N, K)")
    _require(sb.dtype == torch.float32 and sb.shape == b.shape[:1], "sb must be float32, one per row of b")
    m, k = x.shape
    n = b.shape[0]
    d = _int8_out(d, (m, n), out_dtype, x.device)
    _dev(x, b, sb, d)
    if workspace is None:
        workspace = default_workspace(x.device, lib().dg_gemm_int8_nt_act_quant_workspace_size(m, n, k))
    _check("dg_gemm_int8_nt_act_quant",
           lib().dg_gemm_int8_nt_act_quant(_ptr(x), _dtype(x, "x"), _ptr(b), _ptr(sb), _ptr(d), _dtype(d, "d"), m, n, k,
                                           *_ws(workspace), _stream(x)))
    return d


def dg_gemm_int8_grouped_contiguous(a, sa, b, sb, m_indices, d=None, out_dtype=torch.bfloat16):
    """D (M_total, N): row r uses expert m_indices[r] of B (G, N, K); blocks of -1 are skipped."""
    _require(a.dim() == 2 and b.dim() == 3, "a (M_total, K), b (G, N, K)")
    _check_int8(a, sa, b, sb)
    m, k = a.shape
    g, n, _ = b.shape
    d = _int8_out(d, (m, n), out_dtype, a.device)
    _require(m_indices.dtype == torch.int32 and m_indices.numel() == m, "m_indices must be int32, one per row")
    _dev(a, sa, b, sb, m_indices, d)
    _check("dg_gemm_int8_grouped_contiguous",
           lib().dg_gemm_int8_grouped_contiguous(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(m_indices), g, _ptr(d),
                                                 _dtype(d, "d"), m, n, k, _stream(a)))
    return d


def dg_gemm_int8_grouped_masked(a, sa, b, sb, masked_m, d=None, out_dtype=torch.bfloat16, workspace=None,
                                use_workspace=True):
    """D (G, M_max, N): expert g computes only its first masked_m[g] rows; the rest stay untouched."""
    _require(a.dim() == 3 and b.dim() == 3 and a.shape[0] == b.shape[0], "a (G, M_max, K), b (G, N, K)")
    _check_int8(a, sa, b, sb)
    g, m_max, k = a.shape
    n = b.shape[1]
    d = _int8_out(d, (g, m_max, n), out_dtype, a.device)
    _require(masked_m.dtype == torch.int32 and masked_m.numel() == g, "masked_m must be int32, one per expert")
    _dev(a, sa, b, sb, masked_m, d)
    if workspace is None and use_workspace:
        workspace = default_workspace(a.device, lib().dg_gemm_int8_workspace_size(m_max, n, k, g))
    _check("dg_gemm_int8_grouped_masked",
           lib().dg_gemm_int8_grouped_masked(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(d), _dtype(d, "d"), _ptr(masked_m),
                                             g, m_max, n, k, *_ws(workspace), _stream(a)))
    return d
