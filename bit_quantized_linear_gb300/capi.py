"""Thin Python binding of libqlin (include/qlin.h): argument marshalling only.

Each ``qlin_*`` function takes torch tensors (device tensors for the data,
caller-allocated outputs), passes their device pointers, sizes and the current
CUDA stream to the C entry point of the same name, and raises QlinError on a
non-OK status.  No computation happens here; if the shared library is missing
the import fails loudly.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlin.so")

QLIN_OK, QLIN_ERR_INVALID_ARG, QLIN_ERR_UNSUPPORTED, QLIN_ERR_WORKSPACE, QLIN_ERR_CUDA, QLIN_ERR_TIMEOUT = range(6)
QLIN_INT8, QLIN_E4M3 = 0, 1
(QLIN_OP_QUANTIZE_WEIGHT, QLIN_OP_ACT_SCALE, QLIN_OP_QUANTIZE_ACT, QLIN_OP_W8A16_LINEAR,
 QLIN_OP_W8A8_LINEAR, QLIN_OP_I8_GEMM_S32, QLIN_OP_W8A8_DYNAMIC_LINEAR, QLIN_OP_KV_STORE_MIXED,
 QLIN_OP_KV_LOAD_MIXED, QLIN_OP_W8A16_GATE_UP_SILU, QLIN_OP_W8A8_GATE_UP_SILU, QLIN_OP_RMSNORM,
 QLIN_OP_RMSNORM_QUANT, QLIN_OP_W8A8_LINEAR_CODES, QLIN_OP_ROPE, QLIN_OP_ROPE_KV_STORE_MIXED,
 QLIN_OP_QK_NORM_ROPE, QLIN_OP_QK_NORM_ROPE_KV_STORE_INT4) = range(18)

QTYPES = {"int8": QLIN_INT8, "e4m3": QLIN_E4M3}
ROPE_LAYOUTS = {"half": 0, "pairs": 1}
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "by_parts": 3}

# Every symbol the header declares (checked by the not-gpu ABI test).
EXPORTS = ["qlin_quantize_weight", "qlin_act_scale_from_calib", "qlin_quantize_act_static",
           "qlin_w8a16_linear", "qlin_w8a8_linear", "qlin_i8_gemm_s32", "qlin_workspace_bytes",
           "qlin_get_device_status", "qlin_status_string", "qlin_version", "qlin_debug_wait_flag",
           "qlin_kernel_name", "qlin_launch_count", "qlin_w8a8_linear_noalloc",
           "qlin_quantize_act_dynamic", "qlin_w8a8_dynamic_linear", "qlin_kv_store_mixed",
           "qlin_kv_load_mixed", "qlin_w8a16_gate_up_silu", "qlin_w8a8_gate_up_silu",
           "qlin_rmsnorm", "qlin_rmsnorm_quant", "qlin_w8a8_linear_codes", "qlin_rope_table", "qlin_rope",
           "qlin_rope_kv_store_mixed", "qlin_attn_mixed", "qlin_attn_mixed_workspace_bytes",
           "qlin_attn_mixed_kernel_name", "qlin_qk_norm_rope", "qlin_qk_norm_rope_kv_store_int4", "qlin_attn_int4",
           "qlin_attn_int4_workspace_bytes", "qlin_attn_int4_kernel_name"]

# Size of the library-owned scratch of qlin_w8a8_linear_noalloc (QLIN_W8A8_NOALLOC_SCRATCH_BYTES).
W8A8_NOALLOC_SCRATCH_BYTES = 64 << 20


class QlinError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libqlin.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    F, F64 = ctypes.c_float, ctypes.c_double
    sig = {
        "qlin_quantize_weight": [I, I64, I64, P, P, P, P],
        "qlin_act_scale_from_calib": [I, I64, I64, P, P, P, SZ, P],
        "qlin_quantize_act_static": [I, I64, I64, P, P, P, P],
        "qlin_w8a16_linear": [I, I64, I64, I64, P, P, P, P, P, P, SZ, P],
        "qlin_w8a8_linear": [I, I64, I64, I64, P, P, P, P, P, P, P, SZ, P],
        "qlin_i8_gemm_s32": [I64, I64, I64, P, P, P, P, SZ, P],
        "qlin_workspace_bytes": [I, I, I64, I64, I64],
        "qlin_get_device_status": [P],
        "qlin_status_string": [I],
        "qlin_version": [],
        "qlin_debug_wait_flag": [P, ctypes.c_uint64, P],
        "qlin_kernel_name": [I, I, I64, I64, I64],
        "qlin_launch_count": [],
        "qlin_w8a8_linear_noalloc": [I, I64, I64, I64, P, P, P, P, P, P, P],
        "qlin_quantize_act_dynamic": [I, I64, I64, P, P, P, P],
        "qlin_w8a8_dynamic_linear": [I, I64, I64, I64, P, P, P, P, P, P, SZ, P],
        "qlin_kv_store_mixed": [I64, I64, I64, P, I64, P, I64, P, I64, P, P, P, P, P],
        "qlin_kv_load_mixed": [I64, I64, I64, P, I64, P, P, P, P, P, P, P],
        "qlin_w8a16_gate_up_silu": [I, I64, I64, I64, P, P, P, P, P, P, SZ, P],
        "qlin_w8a8_gate_up_silu": [I, I64, I64, I64, P, P, P, P, P, P, P, SZ, P],
        "qlin_rmsnorm": [I64, I64, P, I64, P, I64, P, F, P, P, P],
        "qlin_rmsnorm_quant": [I, I64, I64, P, I64, P, I64, P, F, P, P, P, P, P],
        "qlin_w8a8_linear_codes": [I, I64, I64, I64, P, P, I, P, P, P, P, P, SZ, P],
        "qlin_rope_table": [I64, I64, F64, I, F64, F64, F64, F64, F64, P, P],
        "qlin_rope": [I, I64, I64, I64, I64, I64, P, I64, P, P, I64, P, I64, P, I64, P, I64, P],
        "qlin_rope_kv_store_mixed": [I, I64, I64, I64, I64, I64, P, I64, P, P, I64, P, I64, P, I64, P, I64, P, I64,
                                     P, P, P, P, P],
        "qlin_attn_mixed": [I64, I64, I64, I64, I64, P, I64, P, I64, P, I64, P, I64, I64, I64, P, P, P, P, F, I, I64,
                            P, I64, P, SZ, P],
        "qlin_attn_mixed_workspace_bytes": [I64] * 7,
        "qlin_attn_mixed_kernel_name": [I64] * 7,
        "qlin_qk_norm_rope": [I, I64, I64, I64, I64, I64, I64, ctypes.c_char_p, P, I64, P, P, I64, P, P, I64, P, F, P,
                              I64, P, I64, P],
        "qlin_qk_norm_rope_kv_store_int4": [I, I64, I64, I64, I64, I64, I64, ctypes.c_char_p, P, I64, P, P, I64, P, P,
                                            I64, P, F, P, I64, P, I64, P, I64, I64, P, P, P, P, P],
        "qlin_attn_int4": [I64, I64, I64, I64, I64, P, I64, P, I64, P, I64, P, I64, I64, I64, P, P, P, P, F, I, I64,
                           P, I64, P, SZ, P],
        "qlin_attn_int4_workspace_bytes": [I64] * 7,
        "qlin_attn_int4_kernel_name": [I64] * 7,
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = I
    L.qlin_workspace_bytes.restype = SZ
    L.qlin_status_string.restype = ctypes.c_char_p
    L.qlin_kernel_name.restype = ctypes.c_char_p
    L.qlin_launch_count.restype = ctypes.c_uint64
    L.qlin_attn_mixed_workspace_bytes.restype = SZ
    L.qlin_attn_mixed_kernel_name.restype = ctypes.c_char_p
    L.qlin_attn_int4_workspace_bytes.restype = SZ
    L.qlin_attn_int4_kernel_name.restype = ctypes.c_char_p
    return L


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def status_string(s: int) -> str:
    return _lib.qlin_status_string(int(s)).decode()


def _check(status: int, where: str):
    if status != QLIN_OK:
        raise QlinError(status, where)


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    # the handle of torch.cuda.current_stream(), without the 3 us that the Stream object costs
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _qt(qtype):
    return QTYPES[qtype] if isinstance(qtype, str) else int(qtype)


def qlin_workspace_bytes(op: int, qtype, M: int, K: int, N: int) -> int:
    return int(_lib.qlin_workspace_bytes(op, _qt(qtype), M, K, N))


def qlin_quantize_weight(qtype, w, qw, w_scale, stream=None):
    N, K = w.shape
    _check(_lib.qlin_quantize_weight(_qt(qtype), N, K, _p(w), _p(qw), _p(w_scale), _stream(stream)),
           "qlin_quantize_weight")


def qlin_act_scale_from_calib(qtype, x_cal, input_scale, ws, stream=None):
    rows, K = x_cal.shape
    _check(_lib.qlin_act_scale_from_calib(_qt(qtype), rows, K, _p(x_cal), _p(input_scale), _p(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(),
                                          _stream(stream)), "qlin_act_scale_from_calib")


def qlin_quantize_act_static(qtype, x, input_scale, qx, stream=None):
    M, K = x.shape
    _check(_lib.qlin_quantize_act_static(_qt(qtype), M, K, _p(x), _p(input_scale), _p(qx), _stream(stream)),
           "qlin_quantize_act_static")


def _ws(ws):
    return (None, 0) if ws is None else (_p(ws), ws.numel() * ws.element_size())


def qlin_w8a16_linear(qtype, x, qw, w_scale, bias, y, ws=None, stream=None):
    M, K = x.shape
    N = qw.shape[0]
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a16_linear(_qt(qtype), M, K, N, _p(x), _p(qw), _p(w_scale), _p(bias), _p(y),
                                  wp, wb, _stream(stream)), "qlin_w8a16_linear")


def qlin_w8a8_linear(qtype, x, input_scale, qw, w_scale, bias, y, ws, stream=None):
    M, K = x.shape
    N = qw.shape[0]
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a8_linear(_qt(qtype), M, K, N, _p(x), _p(input_scale), _p(qw), _p(w_scale),
                                 _p(bias), _p(y), wp, wb, _stream(stream)), "qlin_w8a8_linear")


def qlin_w8a8_linear_noalloc(qtype, x, input_scale, qw, w_scale, bias, y, stream=None):
    """W8A8 static linear without a workspace (see qlin_w8a8_linear_noalloc in
    include/qlin.h): for callers that cannot allocate device memory."""
    M, K = x.shape
    N = qw.shape[0]
    _check(_lib.qlin_w8a8_linear_noalloc(_qt(qtype), M, K, N, _p(x), _p(input_scale), _p(qw), _p(w_scale),
                                         _p(bias), _p(y), _stream(stream)), "qlin_w8a8_linear_noalloc")


def qlin_quantize_act_dynamic(qtype, x, qx, x_scale, stream=None):
    M, K = x.shape
    _check(_lib.qlin_quantize_act_dynamic(_qt(qtype), M, K, _p(x), _p(qx), _p(x_scale), _stream(stream)),
           "qlin_quantize_act_dynamic")


def qlin_w8a8_dynamic_linear(qtype, x, qw, w_scale, bias, y, ws, stream=None):
    M, K = x.shape
    N = qw.shape[0]
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a8_dynamic_linear(_qt(qtype), M, K, N, _p(x), _p(qw), _p(w_scale), _p(bias), _p(y),
                                         wp, wb, _stream(stream)), "qlin_w8a8_dynamic_linear")


def qlin_i8_gemm_s32(qx, qw, acc, ws=None, stream=None):
    M, K = qx.shape
    N = qw.shape[0]
    wp, wb = _ws(ws)
    _check(_lib.qlin_i8_gemm_s32(M, K, N, _p(qx), _p(qw), _p(acc), wp, wb, _stream(stream)),
           "qlin_i8_gemm_s32")


def qlin_w8a16_gate_up_silu(qtype, x, qw, w_scale, bias, y, ws=None, stream=None):
    """qw [2I, K] (gate rows first), y [M, I]."""
    M, K = x.shape
    I = qw.shape[0] // 2
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a16_gate_up_silu(_qt(qtype), M, K, I, _p(x), _p(qw), _p(w_scale), _p(bias), _p(y), wp, wb,
                                        _stream(stream)), "qlin_w8a16_gate_up_silu")


def qlin_w8a8_gate_up_silu(qtype, x, input_scale, qw, w_scale, bias, y, ws, stream=None):
    M, K = x.shape
    I = qw.shape[0] // 2
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a8_gate_up_silu(_qt(qtype), M, K, I, _p(x), _p(input_scale), _p(qw), _p(w_scale), _p(bias),
                                       _p(y), wp, wb, _stream(stream)), "qlin_w8a8_gate_up_silu")


def qlin_kv_store_mixed(k, v, slots, k_cache, k_scale, v_cache, v_scale, stream=None):
    """k, v: BF16 [T, ld] (row stride ld elements, last dim contiguous); slots int64 [T];
    caches as allocated by kv_cache_alloc()."""
    S, H, D = k_cache.shape
    T = slots.shape[0]
    assert k.stride(-1) == 1 and v.stride(-1) == 1
    ldk = k.stride(0) if T > 0 else H * D
    ldv = v.stride(0) if T > 0 else H * D
    _check(_lib.qlin_kv_store_mixed(T, H, D, _p(k), ldk, _p(v), ldv, _p(slots), S, _p(k_cache), _p(k_scale),
                                    _p(v_cache), _p(v_scale), _stream(stream)), "qlin_kv_store_mixed")


def qlin_kv_load_mixed(slots, k_cache, k_scale, v_cache, v_scale, k_out, v_out, stream=None):
    S, H, D = k_cache.shape
    T = slots.shape[0]
    _check(_lib.qlin_kv_load_mixed(T, H, D, _p(slots), S, _p(k_cache), _p(k_scale), _p(v_cache), _p(v_scale),
                                   _p(k_out), _p(v_out), _stream(stream)), "qlin_kv_load_mixed")


# The C entry points see addresses: what a tensor's type, size or strides would make them misread, the functions
# below refuse.  (An index array of another type, or a slice of a wider table, is read as other numbers.)  Arrays that
# are read whole are told by their bytes, a cheaper question than type and count.
_BF16 = torch.bfloat16


def _refuse(**arrays):
    """What an array (tensor, bytes) should have been."""
    said = "; ".join(f"{k}: {n} contiguous bytes, not {t.dtype} {tuple(t.shape)} with strides {t.stride()}"
                     for k, (t, n) in arrays.items() if t.nbytes != n or not t.is_contiguous())
    raise ValueError(said or ", ".join(f"{k}: BF16, not {t.dtype}" for k, (t, _) in arrays.items()))


def _rows(t, rows: int, least: int, what: str) -> int:
    """Row stride (elements) of BF16 rows of `least` elements or more."""
    if t.dtype is _BF16:
        (m, n), (row, one) = t.shape, t.stride()
        if m == rows and n >= least and one == 1:
            return row if row >= least or m > 1 else least  # a single row's is whatever its tensor says
    raise ValueError(f"{what}: {rows} BF16 rows of at least {least} contiguous elements, not {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()}")


def _mixed_cache(k_cache, k_scale, v_cache, v_scale):
    """Slots, heads and head size of the four arrays of kv_cache_alloc()."""
    S, H, D = k_cache.shape
    n = S * H
    if (k_cache.nbytes != n * D or k_scale.nbytes != D // 32 * 2 * n or v_cache.nbytes != n * D
            or v_scale.nbytes != 2 * n or not (k_cache.is_contiguous() and k_scale.is_contiguous()
                                               and v_cache.is_contiguous() and v_scale.is_contiguous())):
        _refuse(k_cache=(k_cache, n * D), k_scale=(k_scale, D // 32 * 2 * n), v_cache=(v_cache, n * D),
                v_scale=(v_scale, 2 * n))
    return S, H, D


def _norm_arrays(M: int, K: int, weight, h_out):
    if weight.dtype is not _BF16 or weight.nbytes != 2 * K or not weight.is_contiguous():
        _refuse(weight=(weight, 2 * K))
    if h_out is not None and (h_out.dtype is not _BF16 or h_out.nbytes != 2 * M * K or not h_out.is_contiguous()):
        _refuse(h_out=(h_out, 2 * M * K))


def qlin_rmsnorm(x, residual, weight, eps: float, h_out, y_out, stream=None):
    """x, residual (or None) BF16 [M, K] rows; h_out (with a residual) and y_out BF16 [M, K]."""
    M, K = x.shape
    _norm_arrays(M, K, weight, h_out)
    if y_out.dtype is not _BF16 or y_out.nbytes != 2 * M * K or not y_out.is_contiguous():
        _refuse(y_out=(y_out, 2 * M * K))
    _check(_lib.qlin_rmsnorm(M, K, _p(x), _rows(x, M, K, "x"), _p(residual),
                             0 if residual is None else _rows(residual, M, K, "residual"), _p(weight), eps, _p(h_out),
                             _p(y_out), _stream(stream)), "qlin_rmsnorm")


def qlin_rmsnorm_quant(qtype, x, residual, weight, eps: float, input_scale, h_out, qx, x_scale, stream=None):
    """As qlin_rmsnorm with 1-byte codes qx [M, K]: under input_scale [1] (x_scale None), or per-token
    scales written to x_scale [M] (input_scale None)."""
    M, K = x.shape
    _norm_arrays(M, K, weight, h_out)
    if qx.nbytes != M * K or not qx.is_contiguous():
        _refuse(qx=(qx, M * K))
    if input_scale is not None and input_scale.nbytes != 4:
        _refuse(input_scale=(input_scale, 4))
    if x_scale is not None and (x_scale.nbytes != 4 * M or not x_scale.is_contiguous()):
        _refuse(x_scale=(x_scale, 4 * M))
    _check(_lib.qlin_rmsnorm_quant(_qt(qtype), M, K, _p(x), _rows(x, M, K, "x"), _p(residual),
                                   0 if residual is None else _rows(residual, M, K, "residual"), _p(weight), eps,
                                   _p(input_scale), _p(h_out), _p(qx), _p(x_scale), _stream(stream)),
           "qlin_rmsnorm_quant")


def qlin_w8a8_linear_codes(qtype, qx, x_scale, qw, w_scale, bias, y, ws=None, stream=None):
    """qx [M, K] codes; x_scale one value (per tensor) or [M] (per token, told apart by its size: a single
    row's one scale is both)."""
    M, K = qx.shape
    N = qw.shape[0]
    scales = x_scale.numel()  # one value, or one a row
    if (x_scale.nbytes != 4 * (1 if scales == 1 else M) or qx.nbytes != M * K or qw.nbytes != N * K
            or w_scale.nbytes != 4 * N or y.dtype is not _BF16 or y.nbytes != 2 * M * N
            or not (x_scale.is_contiguous() and qx.is_contiguous() and qw.is_contiguous() and w_scale.is_contiguous()
                    and y.is_contiguous())):
        _refuse(x_scale=(x_scale, 4 * M), qx=(qx, M * K), qw=(qw, N * K), w_scale=(w_scale, 4 * N), y=(y, 2 * M * N))
    if bias is not None and (bias.dtype is not _BF16 or bias.nbytes != 2 * N or not bias.is_contiguous()):
        _refuse(bias=(bias, 2 * N))
    wp, wb = _ws(ws)
    _check(_lib.qlin_w8a8_linear_codes(_qt(qtype), M, K, N, _p(qx), _p(x_scale), int(scales > 1), _p(qw),
                                       _p(w_scale), _p(bias), _p(y), wp, wb, _stream(stream)),
           "qlin_w8a8_linear_codes")


def qlin_rope_table(table, theta: float, scaling="plain", factor: float = 1.0, original_context: float = 0.0,
                    beta_fast: float = 32.0, beta_slow: float = 1.0, amplitude: float = 1.0, stream=None):
    """Fills table, fp32 [max_pos, rot]."""
    max_pos, rot = table.shape
    if table.nbytes != 4 * max_pos * rot or not table.is_contiguous():
        _refuse(table=(table, 4 * max_pos * rot))
    _check(_lib.qlin_rope_table(max_pos, rot, theta, ROPE_SCALINGS[scaling], factor, original_context, beta_fast,
                                beta_slow, amplitude, _p(table), _stream(stream)), "qlin_rope_table")


def _turns(table, rot: int, positions):
    """Tokens and rows of the table."""
    max_pos, turned = table.shape
    if turned != rot:
        raise ValueError(f"the table turns {turned} dimensions, not {rot}")
    T = positions.shape[0]
    if (table.nbytes != 4 * max_pos * rot or positions.nbytes != 8 * T
            or not (table.is_contiguous() and positions.is_contiguous())):
        _refuse(table=(table, 4 * max_pos * rot), positions=(positions, 8 * T))
    return T, max_pos


def qlin_rope(layout, Hq: int, Hk: int, D: int, rot: int, table, positions, q, k, q_out, k_out, stream=None):
    """q [T, >= Hq*D] and k [T, >= Hk*D] BF16 rows (k and k_out None when Hk is 0); table of qlin_rope_table."""
    T, max_pos = _turns(table, rot, positions)
    n, m = Hq * D, Hk * D
    _check(_lib.qlin_rope(ROPE_LAYOUTS[layout], T, Hq, Hk, D, rot, _p(table), max_pos, _p(positions), _p(q),
                          _rows(q, T, n, "q"), _p(k), 0 if k is None else _rows(k, T, m, "k"), _p(q_out),
                          _rows(q_out, T, n, "q_out"), _p(k_out), 0 if k_out is None else _rows(k_out, T, m, "k_out"),
                          _stream(stream)), "qlin_rope")


def qlin_rope_kv_store_mixed(layout, Hq: int, rot: int, table, positions, q, k, v, q_out, slots, k_cache, k_scale,
                             v_cache, v_scale, stream=None):
    """q turned into q_out; k (turned) and v quantized into their slots of the caches of kv_cache_alloc()."""
    T, max_pos = _turns(table, rot, positions)
    S, H, D = _mixed_cache(k_cache, k_scale, v_cache, v_scale)
    n, m = Hq * D, H * D
    if slots.nbytes != 8 * T or not slots.is_contiguous():
        _refuse(slots=(slots, 8 * T))
    _check(_lib.qlin_rope_kv_store_mixed(ROPE_LAYOUTS[layout], T, Hq, H, D, rot, _p(table), max_pos, _p(positions),
                                         _p(q), _rows(q, T, n, "q"), _p(k), _rows(k, T, m, "k"), _p(v),
                                         _rows(v, T, m, "v"), _p(q_out), _rows(q_out, T, n, "q_out"), _p(slots), S,
                                         _p(k_cache), _p(k_scale), _p(v_cache), _p(v_scale), _stream(stream)),
           "qlin_rope_kv_store_mixed")


def qlin_attn_mixed(q, q_start, kv_len, block_table, block_size: int, k_cache, k_scale, v_cache, v_scale, max_q: int,
                    max_kv: int, scale: float, causal: bool, window: int, out, ws=None, stream=None):
    """q, out BF16 [T, Hq*D] rows; q_start int32 [B+1]; kv_len int32 [B]; block_table int32 [B, max_blocks]."""
    S, H, D = _mixed_cache(k_cache, k_scale, v_cache, v_scale)
    (T, n), (B, blocks) = q.shape, block_table.shape
    if n % D:
        raise ValueError(f"rows of q hold {n} elements, not heads of {D}")
    if (q_start.nbytes != 4 * (B + 1) or kv_len.nbytes != 4 * B or block_table.nbytes != 4 * B * blocks
            or not (q_start.is_contiguous() and kv_len.is_contiguous() and block_table.is_contiguous())):
        _refuse(q_start=(q_start, 4 * (B + 1)), kv_len=(kv_len, 4 * B), block_table=(block_table, 4 * B * blocks))
    wp, wb = _ws(ws)
    _check(_lib.qlin_attn_mixed(B, T, n // D, H, D, _p(q), _rows(q, T, n, "q"), _p(q_start), max_q, _p(kv_len), max_kv,
                                _p(block_table), blocks, block_size, S, _p(k_cache), _p(k_scale), _p(v_cache),
                                _p(v_scale), scale, int(causal), window, _p(out), _rows(out, T, n, "out"), wp, wb,
                                _stream(stream)), "qlin_attn_mixed")


def qlin_attn_mixed_workspace_bytes(B: int, Hq: int, H: int, D: int, max_q: int, max_kv: int, window: int = 0) -> int:
    return int(_lib.qlin_attn_mixed_workspace_bytes(B, Hq, H, D, max_q, max_kv, window))


def qlin_attn_mixed_kernel_name(B: int, Hq: int, H: int, D: int, max_q: int, max_kv: int, window: int = 0) -> str:
    return _lib.qlin_attn_mixed_kernel_name(B, Hq, H, D, max_q, max_kv, window).decode()


def rope_axes(sections, interleaved: bool = False) -> bytes:
    """The axis of each pair of dimensions, for the `axes` of the functions below: sections[a] pairs turn by
    axis a's positions; one section after the other, or, interleaved, the axes in turn until their sections are used up."""
    if not interleaved:
        return bytes(a for a, n in enumerate(sections) for _ in range(n))
    left, out = list(sections), []
    while any(left):
        for a, n in enumerate(left):
            if n:
                out.append(a)
                left[a] -= 1
    return bytes(out)


def _angles(table, rot: int, positions, axes):
    """Tokens, rows of the table, number of axes."""
    if positions.dim() == 2:
        A, T = positions.shape
    else:
        A, T = 1, positions.shape[0]
    if not rot:
        return T, 0, 1
    max_pos, turned = table.shape
    if turned != rot:
        raise ValueError(f"the table turns {turned} dimensions, not {rot}")
    if axes is not None and len(axes) != rot // 2:
        raise ValueError(f"axes: one for each of {rot // 2} pairs, not {len(axes)}")
    if (table.nbytes != 4 * max_pos * rot or positions.nbytes != 8 * A * T
            or not (table.is_contiguous() and positions.is_contiguous())):
        _refuse(table=(table, 4 * max_pos * rot), positions=(positions, 8 * A * T))
    return T, max_pos, A


def _head_weights(D: int, q_weight, k_weight):
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and (w.dtype is not _BF16 or w.nbytes != 2 * D or not w.is_contiguous()):
            _refuse(**{name: (w, 2 * D)})


def qlin_qk_norm_rope(layout, Hq: int, Hk: int, D: int, rot: int, table, positions, q, k, q_weight, k_weight,
                      eps: float, q_out, k_out, axes=None, stream=None):
    """Norms of q's and k's heads (weights [D] or None) and their rotation.  positions int64 [T], or [A, T] with
    `axes` (bytes, see rope_axes); rot 0: no rotation (table None, positions only counts the tokens).  q, k as for qlin_rope."""
    T, max_pos, A = _angles(table, rot, positions, axes)
    n, m = Hq * D, Hk * D
    _head_weights(D, q_weight, k_weight)
    _check(_lib.qlin_qk_norm_rope(ROPE_LAYOUTS[layout], T, Hq, Hk, D, rot, A, axes, _p(table), max_pos,
                                  _p(positions), _p(q), _rows(q, T, n, "q"), _p(q_weight), _p(k),
                                  0 if k is None else _rows(k, T, m, "k"), _p(k_weight), eps, _p(q_out),
                                  _rows(q_out, T, n, "q_out"), _p(k_out),
                                  0 if k_out is None else _rows(k_out, T, m, "k_out"), _stream(stream)),
           "qlin_qk_norm_rope")


def _int4_cache(k_cache, k_scale, v_cache, v_scale):
    """Pages, heads, positions of a page and head size of the four arrays of kv_int4_alloc()."""
    N, H, block, half = k_cache.shape
    n = N * H * block
    if (k_cache.nbytes != n * half or k_scale.nbytes != half // 16 * 2 * n or v_cache.nbytes != n * half
            or v_scale.nbytes != half // 16 * 2 * n or not (k_cache.is_contiguous() and k_scale.is_contiguous()
                                                            and v_cache.is_contiguous() and v_scale.is_contiguous())):
        _refuse(k_cache=(k_cache, n * half), k_scale=(k_scale, half // 16 * 2 * n), v_cache=(v_cache, n * half),
                v_scale=(v_scale, half // 16 * 2 * n))
    return N, H, block, 2 * half


def qlin_qk_norm_rope_kv_store_int4(layout, Hq: int, rot: int, table, positions, q, k, v, q_weight, k_weight,
                                    eps: float, q_out, slots, k_cache, k_scale, v_cache, v_scale, axes=None,
                                    stream=None):
    """As qlin_qk_norm_rope into q_out (q and q_out None when Hq is 0), k (so treated) and v quantized into their
    slots of the caches of kv_int4_alloc()."""
    T, max_pos, A = _angles(table, rot, positions, axes)
    N, H, block, D = _int4_cache(k_cache, k_scale, v_cache, v_scale)
    n, m = Hq * D, H * D
    _head_weights(D, q_weight, k_weight)
    if slots.nbytes != 8 * T or not slots.is_contiguous():
        _refuse(slots=(slots, 8 * T))
    _check(_lib.qlin_qk_norm_rope_kv_store_int4(
        ROPE_LAYOUTS[layout], T, Hq, H, D, rot, A, axes, _p(table), max_pos, _p(positions), _p(q),
        _rows(q, T, n, "q") if Hq else 0, _p(q_weight), _p(k), _rows(k, T, m, "k"), _p(k_weight), eps, _p(v),
        _rows(v, T, m, "v"), _p(q_out), _rows(q_out, T, n, "q_out") if Hq else 0, _p(slots), N, block, _p(k_cache),
        _p(k_scale), _p(v_cache), _p(v_scale), _stream(stream)), "qlin_qk_norm_rope_kv_store_int4")


def qlin_attn_int4(q, q_start, kv_len, block_table, k_cache, k_scale, v_cache, v_scale, max_q: int, max_kv: int,
                   scale: float, causal: bool, window: int, out, ws=None, stream=None):
    """As qlin_attn_mixed over the caches of kv_int4_alloc()."""
    N, H, block, D = _int4_cache(k_cache, k_scale, v_cache, v_scale)
    (T, n), (B, blocks) = q.shape, block_table.shape
    if n % D:
        raise ValueError(f"rows of q hold {n} elements, not heads of {D}")
    if (q_start.nbytes != 4 * (B + 1) or kv_len.nbytes != 4 * B or block_table.nbytes != 4 * B * blocks
            or not (q_start.is_contiguous() and kv_len.is_contiguous() and block_table.is_contiguous())):
        _refuse(q_start=(q_start, 4 * (B + 1)), kv_len=(kv_len, 4 * B), block_table=(block_table, 4 * B * blocks))
    wp, wb = _ws(ws)
    _check(_lib.qlin_attn_int4(B, T, n // D, H, D, _p(q), _rows(q, T, n, "q"), _p(q_start), max_q, _p(kv_len), max_kv,
                               _p(block_table), blocks, block, N, _p(k_cache), _p(k_scale), _p(v_cache), _p(v_scale),
                               scale, int(causal), window, _p(out), _rows(out, T, n, "out"), wp, wb, _stream(stream)),
           "qlin_attn_int4")


def qlin_attn_int4_workspace_bytes(B: int, Hq: int, H: int, D: int, max_q: int, max_kv: int, window: int = 0) -> int:
    return int(_lib.qlin_attn_int4_workspace_bytes(B, Hq, H, D, max_q, max_kv, window))


def qlin_attn_int4_kernel_name(B: int, Hq: int, H: int, D: int, max_q: int, max_kv: int, window: int = 0) -> str:
    return _lib.qlin_attn_int4_kernel_name(B, Hq, H, D, max_q, max_kv, window).decode()


def qlin_kernel_name(op: int, qtype, M: int, K: int, N: int) -> str:
    return _lib.qlin_kernel_name(op, _qt(qtype), M, K, N).decode()


def qlin_launch_count() -> int:
    return int(_lib.qlin_launch_count())


def qlin_get_device_status(stream=None) -> int:
    return int(_lib.qlin_get_device_status(_stream(stream)))


def qlin_debug_wait_flag(flag, timeout_ns: int, stream=None):
    _check(_lib.qlin_debug_wait_flag(_p(flag), int(timeout_ns), _stream(stream)), "qlin_debug_wait_flag")


# ---------------------------------------------------------------------------
# Convenience wrappers that allocate outputs / workspaces with torch (device
# memory only) and call the entry points above.
# ---------------------------------------------------------------------------
def workspace(op: int, qtype, M: int, K: int, N: int, device=None):
    n = qlin_workspace_bytes(op, qtype, M, K, N)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def quantize_weight(qtype, w):
    N, K = w.shape
    qw = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    s = torch.empty((N,), dtype=torch.float32, device=w.device)
    qlin_quantize_weight(qtype, w, qw, s)
    return qw, s


def act_scale_from_calib(qtype, x_cal):
    s = torch.empty((1,), dtype=torch.float32, device=x_cal.device)
    ws = workspace(QLIN_OP_ACT_SCALE, qtype, *x_cal.shape, 0, device=x_cal.device)
    qlin_act_scale_from_calib(qtype, x_cal, s, ws)
    return s


def quantize_act_static(qtype, x, input_scale):
    qx = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    qlin_quantize_act_static(qtype, x, input_scale, qx)
    return qx


def w8a16_linear(qtype, x, qw, w_scale, bias=None):
    M, K = x.shape
    N = qw.shape[0]
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws = workspace(QLIN_OP_W8A16_LINEAR, qtype, M, K, N, device=x.device)
    qlin_w8a16_linear(qtype, x, qw, w_scale, bias, y, ws)
    return y


def w8a8_linear(qtype, x, input_scale, qw, w_scale, bias=None):
    M, K = x.shape
    N = qw.shape[0]
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws = workspace(QLIN_OP_W8A8_LINEAR, qtype, M, K, N, device=x.device)
    qlin_w8a8_linear(qtype, x, input_scale, qw, w_scale, bias, y, ws)
    return y


def quantize_act_dynamic(qtype, x):
    qx = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((x.shape[0],), dtype=torch.float32, device=x.device)
    qlin_quantize_act_dynamic(qtype, x, qx, s)
    return qx, s


def w8a8_dynamic_linear(qtype, x, qw, w_scale, bias=None):
    M, K = x.shape
    N = qw.shape[0]
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ws = workspace(QLIN_OP_W8A8_DYNAMIC_LINEAR, qtype, M, K, N, device=x.device)
    qlin_w8a8_dynamic_linear(qtype, x, qw, w_scale, bias, y, ws)
    return y


def i8_gemm_s32(qx, qw):
    M, K = qx.shape
    N = qw.shape[0]
    acc = torch.empty((M, N), dtype=torch.int32, device=qx.device)
    ws = workspace(QLIN_OP_I8_GEMM_S32, QLIN_INT8, M, K, N, device=qx.device)
    qlin_i8_gemm_s32(qx, qw, acc, ws)
    return acc


def kv_cache_alloc(num_slots: int, H: int, D: int, device=None):
    """Device arrays of a mixed KV cache: k_cache int8 [S,H,D], k_scale float16 bits
    [S,H,D/32] (int16 storage), v_cache E4M3 codes [S,H,D] (uint8), v_scale float16
    bits [S,H] (int16 storage)."""
    dev = device or "cuda"
    return (torch.empty((num_slots, H, D), dtype=torch.int8, device=dev),
            torch.empty((num_slots, H, D // 32), dtype=torch.int16, device=dev),
            torch.empty((num_slots, H, D), dtype=torch.uint8, device=dev),
            torch.empty((num_slots, H), dtype=torch.int16, device=dev))


def kv_load_mixed(slots, cache):
    S, H, D = cache[0].shape
    T = slots.shape[0]
    k = torch.empty((T, H, D), dtype=torch.bfloat16, device=slots.device)
    v = torch.empty((T, H, D), dtype=torch.bfloat16, device=slots.device)
    qlin_kv_load_mixed(slots, *cache, k, v)
    return k, v


def w8a16_gate_up_silu(qtype, x, qw, w_scale, bias=None):
    M, K = x.shape
    I = qw.shape[0] // 2
    y = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    ws = workspace(QLIN_OP_W8A16_GATE_UP_SILU, qtype, M, K, I, device=x.device)
    qlin_w8a16_gate_up_silu(qtype, x, qw, w_scale, bias, y, ws)
    return y


def w8a8_gate_up_silu(qtype, x, input_scale, qw, w_scale, bias=None):
    M, K = x.shape
    I = qw.shape[0] // 2
    y = torch.empty((M, I), dtype=torch.bfloat16, device=x.device)
    ws = workspace(QLIN_OP_W8A8_GATE_UP_SILU, qtype, M, K, I, device=x.device)
    qlin_w8a8_gate_up_silu(qtype, x, input_scale, qw, w_scale, bias, y, ws)
    return y


def rmsnorm(x, weight, eps: float, residual=None):
    """BF16 norm; returns (h, y) with h = x when there is no residual."""
    h = None if residual is None else torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    qlin_rmsnorm(x, residual, weight, eps, h, y)
    return (x if h is None else h), y


def rmsnorm_quant(qtype, x, weight, eps: float, residual=None, input_scale=None):
    """8-bit norm; returns (h, codes, scale): scale is input_scale, or the per-token scales made here."""
    h = None if residual is None else torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    qx = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    s = torch.empty((x.shape[0],), dtype=torch.float32, device=x.device) if input_scale is None else None
    qlin_rmsnorm_quant(qtype, x, residual, weight, eps, input_scale, h, qx, s)
    return (x if h is None else h), qx, (s if input_scale is None else input_scale)


def w8a8_linear_codes(qtype, qx, x_scale, qw, w_scale, bias=None):
    M, K = qx.shape
    N = qw.shape[0]
    y = torch.empty((M, N), dtype=torch.bfloat16, device=qx.device)
    ws = workspace(QLIN_OP_W8A8_LINEAR_CODES, qtype, M, K, N, device=qx.device)
    qlin_w8a8_linear_codes(qtype, qx, x_scale, qw, w_scale, bias, y, ws)
    return y


def rope_table(max_pos: int, rot: int, theta: float = 10000.0, device=None, **scaling):
    """The table qlin_rope reads, fp32 [max_pos, rot]; scaling as the arguments of qlin_rope_table."""
    table = torch.empty((max_pos, rot), dtype=torch.float32, device=device or "cuda")
    qlin_rope_table(table, theta, **scaling)
    return table


def attn_mixed(q, q_start, kv_len, block_table, block_size: int, cache, max_q: int, max_kv: int, scale=None,
               causal: bool = True, window: int = 0, out=None, ws=None):
    """Attention of q over a mixed cache (the four arrays of kv_cache_alloc()); scale defaults to D^-1/2."""
    _, H, D = cache[0].shape
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if ws is None:
        n = qlin_attn_mixed_workspace_bytes(kv_len.shape[0], q.shape[1] // D, H, D, max_q, max_kv, window)
        if 0 < n < 2 ** 63:  # invalid sizes are the call's to report
            ws = torch.empty(n, dtype=torch.uint8, device=q.device)
    qlin_attn_mixed(q, q_start, kv_len, block_table, block_size, *cache, max_q, max_kv,
                    D ** -0.5 if scale is None else scale, causal, window, out, ws)
    return out


def kv_int4_alloc(num_blocks: int, block_size: int, H: int, D: int, device=None):
    """Device arrays of a 4-bit KV cache: k_cache uint8 [num_blocks, H, block_size, D/2], k_scale float16 bits
    [num_blocks, H, block_size, D/32] (int16 storage), v_cache and v_scale likewise."""
    dev = device or "cuda"
    codes, scales = (num_blocks, H, block_size, D // 2), (num_blocks, H, block_size, D // 32)
    return (torch.empty(codes, dtype=torch.uint8, device=dev), torch.empty(scales, dtype=torch.int16, device=dev),
            torch.empty(codes, dtype=torch.uint8, device=dev), torch.empty(scales, dtype=torch.int16, device=dev))


def kv_store_int4(k, v, slots, cache):
    """Quantizes rows k, v [T, >= H*D] as they are into their slots of a 4-bit cache."""
    qlin_qk_norm_rope_kv_store_int4("half", 0, 0, None, slots, None, k, v, None, None, 0.0, None, slots, *cache)


class _Scratch:
    """Workspace of one call on the device of `like`: a tensor's memory without the tensor (16.2 and 18.8 us of host time
    a call of attn_int4 with them)."""
    __slots__ = ("n", "memory")

    def __init__(self, n: int, like):
        self.n = n
        self.memory = torch.UntypedStorage(n, device=like.device)

    def data_ptr(self):
        return self.memory.data_ptr()

    def numel(self):
        return self.n

    def element_size(self):
        return 1


def attn_int4(q, q_start, kv_len, block_table, cache, max_q: int, max_kv: int, scale=None, causal: bool = True,
              window: int = 0, out=None, ws=None):
    """Attention of q over a 4-bit cache (the four arrays of kv_int4_alloc()); scale defaults to D^-1/2."""
    _, H, _, half = cache[0].shape
    D = 2 * half
    if out is None:
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if ws is None:
        n = qlin_attn_int4_workspace_bytes(kv_len.shape[0], q.shape[1] // D, H, D, max_q, max_kv, window)
        if 0 < n < 2 ** 63:  # invalid sizes are the call's to report
            ws = _Scratch(n, q)
    qlin_attn_int4(q, q_start, kv_len, block_table, *cache, max_q, max_kv, D ** -0.5 if scale is None else scale,
                   causal, window, out, ws)
    return out
