"""Packed low-bit weight-quantized matmul for AMD Instinct MI355X (gfx950).

Thin ctypes binding over libbqmm.so (C ABI in include/bqmm.h).  The binding
only marshals arguments: every step runs in the library's HIP kernels.  torch
is used for device memory and the current stream; tensors must be contiguous
CUDA (HIP) tensors.  bf16 data travels as torch.bfloat16 (or int16/uint16
views), packed weights and q8_1 buffers as torch.uint8.

The library must be built first (python -m bit_quantized_matmul_quantize_amd.build);
there is no fallback implementation: a missing library raises ImportError on
first use.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# BQMM_SANITIZE=1 selects the host-sanitized build of the same library (see
# build.py); it is for the CPU test suite only.
LIB_PATH = os.path.join(_HERE, "libbqmm_san.so" if os.environ.get("BQMM_SANITIZE") == "1" else "libbqmm.so")

BQ_OK, BQ_EINVAL, BQ_EUNSUPPORTED, BQ_EALIGN, BQ_EHIP = 0, -1, -2, -3, -4

# name -> (restype, argtypes); P = pointer, U32/U64 = unsigned ints, I = int, F/D = float/double
_P, _U32, _U64, _I = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int
_F, _D = ctypes.c_float, ctypes.c_double
EXPORTS = {
    "bq_last_error": (ctypes.c_char_p, []),
    "bq_status_string": (ctypes.c_char_p, [_I]),
    "q8_1_act_bytes": (_U64, [_U32, _U32]),
    "q2_0_weight_bytes": (_U64, [_U32, _U32, _U32]),
    "q4k_weight_bytes": (_U64, [_U32, _U32]),
    "quantize_act_q8_1": (_I, [_P, _P, _U32, _U32, _P]),
    "silu_mul_quantize_q8_1": (_I, [_P, _P, _P, _U32, _U32, _P]),
    "q2_0_mmq_gemm": (_I, [_P, _P, _P, _U32, _U32, _U32, _P]),
    "q2_0_mmq_gemm_ldc": (_I, [_P, _P, _P, _U32, _U32, _U32, _U32, _P]),
    "q4k_mmq_gemm_ldc": (_I, [_P, _P, _P, _U32, _U32, _U32, _U32, _P]),
    "q2_0_gemv_vec": (_I, [_P, _P, _P, _U32, _U32, _P]),
    "q2_0_gemv_vec_batchm": (_I, [_P, _P, _P, _U32, _U32, _U32, _P]),
    "q2_0_gemv_gate_up_silu": (_I, [_P, _P, _P, _P, _U32, _U32, _U32, _P]),
    "dequant_q2_0_to_bf16": (_I, [_P, _P, _U32, _U32, _U32, _P]),
    "dense_gemm_bf16": (_I, [_P, _P, _P, _U32, _U32, _U32, _P]),
    "q2_0_prefill_gemm": (_I, [_P, _P, _P, _P, _P, _U32, _U32, _U32, _U32, _I, _P]),
    "q2_0_prefill_gemm_noalloc": (_I, [_P, _P, _P, _U32, _U32, _U32, _U32, _I, _P]),
    "q4k_mmq_gemm": (_I, [_P, _P, _P, _U32, _U32, _U32, _P]),
    "q4k_gemv_vec": (_I, [_P, _P, _P, _U32, _U32, _P]),
    "quantize_weight_q4k": (_I, [_P, _P, _U32, _U32, _P]),
    "silu_mul_bf16": (_I, [_P, _P, _P, _U64, _P]),
    "int8_rows_bytes": (_U64, [_U32, _U32]),
    "gated_delta_rule_workspace_bytes": (_U64, [_U32] * 6),
    "add_rms_norm_bf16": (_I, [_P, _P, _P, _P, _U32, _U32, _D, _P]),
    "add_rms_norm_quantize_q8_1": (_I, [_P, _P, _P, _P, _U32, _U32, _D, _P]),
    "add_rms_norm_quantize_int8": (_I, [_P, _P, _P, _P, _U32, _U32, _D, _P]),
    "quantize_rows_int8": (_I, [_P, _P, _U32, _U32, _P]),
    "w8a8_gemm_form": (_I, [_U32] * 4),
    "w8a8_gemm": (_I, [_P, _P, _P, _P, _U32, _U32, _U32, _P]),
    "gated_delta_rule_recurrent": (_I, [_P] * 10 + [_U32] * 7 + [_U64] * 6 + [_F, _I, _P]),
    "gated_delta_rule_chunked": (_I, [_P] * 11 + [_U64] + [_U32] * 7 + [_U64] * 6 + [_F, _I, _P]),
    "kv_cache_page_bytes": (_U64, [_U32] * 4),
    "paged_attention_workspace_bytes": (_U64, [_U32] * 5),
    "rope_write_kv_cache": (_I, [_P] * 14 + [_U32] * 12 + [_U64] * 6 + [_F, _P]),
    "read_kv_cache": (_I, [_P] * 7 + [_U32] * 8 + [_P]),
    "paged_attention_decode": (_I, [_P] * 8 + [_U64] + [_U32] * 9 + [_U64] * 2 + [_U32, _F, _F, _P]),
    "paged_attention_prefill": (_I, [_P] * 7 + [_U32] * 9 + [_U64] * 2 + [_U32, _F, _F, _P]),
    "q2_0_mmq_blockdots": (_I, [_P, _P, _P, _U32, _U32, _U32, _U32, _U32, _U32, _U32, _P]),
    "q4k_mmq_blockdots": (_I, [_P, _P, _P, _U32, _U32, _U32, _U32, _U32, _U32, _U32, _P]),
}

_lib = None


class BqmmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


def lib():
    """Load libbqmm.so (raises ImportError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m bit_quantized_matmul_quantize_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(status: int):
    if status != BQ_OK:
        raise BqmmError(status, lib().bq_last_error().decode())


_current_stream = None


def _stream(stream):
    """The given stream, or torch's current one, as an address."""
    global _current_stream
    if stream is not None:
        return int(stream)
    if _current_stream is None:
        import torch
        # the address alone: a torch.cuda.Stream object costs 2 us per call, as much as the launch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _current_stream = ((lambda: raw(torch.cuda.current_device())) if raw
                           else (lambda: torch.cuda.current_stream().cuda_stream))
    return _current_stream()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


_BF16, _U8 = ("torch.bfloat16", "torch.int16", "torch.uint16"), ("torch.uint8",)
_kinds = {}  # dtype -> its name (str() of a dtype builds it anew)


def _kind(t):
    d = t.dtype
    return _kinds.get(d) or _kinds.setdefault(d, str(d))


def _bf16(t, what):
    if _kind(t) not in _BF16:
        raise TypeError(f"{what}: expected bfloat16 data, got {t.dtype}")
    return t


def _u8(t, what):
    if _kind(t) not in _U8:
        raise TypeError(f"{what}: expected uint8 bytes, got {t.dtype}")
    return t


# ---- sizes ------------------------------------------------------------------

def q8_1_act_bytes(m: int, k: int) -> int:
    return int(lib().q8_1_act_bytes(m, k))


def q2_0_weight_bytes(n: int, k: int, group: int = 128) -> int:
    return int(lib().q2_0_weight_bytes(n, k, group))


def q4k_weight_bytes(n: int, k: int) -> int:
    return int(lib().q4k_weight_bytes(n, k))


# ---- calls (same names as the C ABI) -----------------------------------------
#
# Each wrapper checks, before anything reaches the library: dtypes, that every
# tensor holds at least the bytes its shape arguments address (the C ABI sees
# plain pointers and cannot), and that all tensors are contiguous device
# tensors on one device.

def _nbytes(t) -> int:
    return t.nbytes


def _need(t, nbytes: int, what: str):
    if t is not None and _nbytes(t) < nbytes:
        raise ValueError(f"{what}: {_nbytes(t)} bytes, the shape arguments address {nbytes}")
    return t


def _same_device(*tensors):
    devs = {t.get_device() for t in tensors if t is not None and t.is_cuda}
    if len(devs) > 1:
        raise ValueError(f"tensors on different devices: {['cuda:%d' % d for d in sorted(devs)]}")


def _ptrs(*tensors):
    """Device pointers of the given contiguous tensors (None passes through), all on one device."""
    ptrs, dev = [], None
    for t in tensors:
        if t is None:
            ptrs.append(None)
            continue
        d = t.get_device()  # -1: not on a device
        if (d != dev and (d < 0 or dev is not None)) or not t.is_contiguous():
            _same_device(*tensors)  # one of these says what is wrong
            return [_ptr(t) for t in tensors]
        dev = d
        ptrs.append(t.data_ptr())
    return ptrs


def _bf(m: int, k: int) -> int:
    return 2 * m * k


def quantize_act_q8_1(act, out_q8, m: int, k: int, stream=None):
    _need(_bf16(act, "act"), _bf(m, k), "act")
    _need(_u8(out_q8, "out_q8"), q8_1_act_bytes(m, k), "out_q8")
    _check(lib().quantize_act_q8_1(*_ptrs(act, out_q8), m, k, _stream(stream)))


def silu_mul_quantize_q8_1(gate, up, out_q8, m: int, k: int, stream=None):
    _need(_bf16(gate, "gate"), _bf(m, k), "gate")
    _need(_bf16(up, "up"), _bf(m, k), "up")
    _need(_u8(out_q8, "out_q8"), q8_1_act_bytes(m, k), "out_q8")
    _check(lib().silu_mul_quantize_q8_1(*_ptrs(gate, up, out_q8), m, k, _stream(stream)))


def q2_0_mmq_gemm(act_q8, w_q2, out, m: int, n: int, k: int, stream=None):
    _need(_u8(act_q8, "act_q8"), q8_1_act_bytes(m, k), "act_q8")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k), "w_q2")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().q2_0_mmq_gemm(*_ptrs(act_q8, w_q2, out), m, n, k, _stream(stream)))


def _ptr_rows(t, m: int, n: int, ldc: int, what):
    """A [m, n] bf16 view whose rows are ldc elements apart (a column range of a wider buffer)."""
    _bf16(t, what)
    if tuple(t.shape) != (m, n) or (m > 1 and t.stride(0) != ldc) or (n > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: expected an [{m}, {n}] view with row stride {ldc}")
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    return ctypes.c_void_p(t.data_ptr())


def q2_0_mmq_gemm_ldc(act_q8, w_q2, out, m: int, n: int, k: int, ldc: int, stream=None):
    _need(_u8(act_q8, "act_q8"), q8_1_act_bytes(m, k), "act_q8")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k), "w_q2")
    out_p = _ptr_rows(out, m, n, ldc, "out")
    _same_device(act_q8, w_q2, out)
    a_p, w_p = _ptrs(act_q8, w_q2)
    _check(lib().q2_0_mmq_gemm_ldc(a_p, w_p, out_p, m, n, k, ldc, _stream(stream)))


def q4k_mmq_gemm_ldc(act_q8, w_q4k, out, m: int, n: int, k: int, ldc: int, stream=None):
    _need(_u8(act_q8, "act_q8"), q8_1_act_bytes(m, k), "act_q8")
    _need(_u8(w_q4k, "w_q4k"), q4k_weight_bytes(n, k), "w_q4k")
    out_p = _ptr_rows(out, m, n, ldc, "out")
    _same_device(act_q8, w_q4k, out)
    a_p, w_p = _ptrs(act_q8, w_q4k)
    _check(lib().q4k_mmq_gemm_ldc(a_p, w_p, out_p, m, n, k, ldc, _stream(stream)))


def q2_0_gemv_vec(act, w_q2, out, n: int, k: int, stream=None):
    _need(_bf16(act, "act"), _bf(1, k), "act")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k), "w_q2")
    _need(_bf16(out, "out"), _bf(1, n), "out")
    _check(lib().q2_0_gemv_vec(*_ptrs(act, w_q2, out), n, k, _stream(stream)))


def q2_0_gemv_vec_batchm(act, w_q2, out, m: int, n: int, k: int, stream=None):
    _need(_bf16(act, "act"), _bf(m, k), "act")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k), "w_q2")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().q2_0_gemv_vec_batchm(*_ptrs(act, w_q2, out), m, n, k, _stream(stream)))


def q2_0_gemv_gate_up_silu(act, w_gate, w_up, out, m: int, n: int, k: int, stream=None):
    _need(_bf16(act, "act"), _bf(m, k), "act")
    _need(_u8(w_gate, "w_gate"), q2_0_weight_bytes(n, k), "w_gate")
    _need(_u8(w_up, "w_up"), q2_0_weight_bytes(n, k), "w_up")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().q2_0_gemv_gate_up_silu(*_ptrs(act, w_gate, w_up, out), m, n, k, _stream(stream)))


def dequant_q2_0_to_bf16(w_q2, out, n: int, k: int, group: int = 128, stream=None):
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k, group), "w_q2")
    _need(_bf16(out, "out"), _bf(n, k), "out")
    _check(lib().dequant_q2_0_to_bf16(*_ptrs(w_q2, out), n, k, group, _stream(stream)))


def dense_gemm_bf16(a, w, out, m: int, n: int, k: int, stream=None):
    _need(_bf16(a, "a"), _bf(m, k), "a")
    _need(_bf16(w, "w"), _bf(n, k), "w")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().dense_gemm_bf16(*_ptrs(a, w, out), m, n, k, _stream(stream)))


def q2_0_prefill_gemm(act, w_q2, out, scratch, act_q8, m: int, n: int, k: int, group: int = 128,
                      use_mmq: bool = True, stream=None):
    _need(_bf16(act, "act"), _bf(m, k), "act")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k, group), "w_q2")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    if use_mmq and group == 128:  # the MMQ branch writes act_q8, the dequant branch scratch
        _need(act_q8, q8_1_act_bytes(m, k), "act_q8")
    else:
        _need(scratch, _bf(n, k), "scratch")
    _check(lib().q2_0_prefill_gemm(*_ptrs(act, w_q2, out, scratch, act_q8), m, n, k, group,
                                   int(bool(use_mmq)), _stream(stream)))


def q2_0_prefill_gemm_noalloc(act, w_q2, out, m: int, n: int, k: int, group: int = 128,
                              use_mmq: bool = True, stream=None):
    _need(_bf16(act, "act"), _bf(m, k), "act")
    _need(_u8(w_q2, "w_q2"), q2_0_weight_bytes(n, k, group), "w_q2")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().q2_0_prefill_gemm_noalloc(*_ptrs(act, w_q2, out), m, n, k, group, int(bool(use_mmq)),
                                           _stream(stream)))


def q4k_mmq_gemm(act_q8, w_q4k, out, m: int, n: int, k: int, stream=None):
    _need(_u8(act_q8, "act_q8"), q8_1_act_bytes(m, k), "act_q8")
    _need(_u8(w_q4k, "w_q4k"), q4k_weight_bytes(n, k), "w_q4k")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    _check(lib().q4k_mmq_gemm(*_ptrs(act_q8, w_q4k, out), m, n, k, _stream(stream)))


def q4k_gemv_vec(act, w_q4k, out, n: int, k: int, stream=None):
    _need(_bf16(act, "act"), _bf(1, k), "act")
    _need(_u8(w_q4k, "w_q4k"), q4k_weight_bytes(n, k), "w_q4k")
    _need(_bf16(out, "out"), _bf(1, n), "out")
    _check(lib().q4k_gemv_vec(*_ptrs(act, w_q4k, out), n, k, _stream(stream)))


def quantize_weight_q4k(w, out_q4k, n: int, k: int, stream=None):
    _need(_bf16(w, "w"), _bf(n, k), "w")
    _need(_u8(out_q4k, "out_q4k"), q4k_weight_bytes(n, k), "out_q4k")
    _check(lib().quantize_weight_q4k(*_ptrs(w, out_q4k), n, k, _stream(stream)))


def silu_mul_bf16(gate, up, out, count: int | None = None, stream=None):
    count = gate.numel() if count is None else count
    for t, what in ((gate, "gate"), (up, "up"), (out, "out")):
        _need(_bf16(t, what), 2 * count, what)
    _check(lib().silu_mul_bf16(*_ptrs(gate, up, out), count, _stream(stream)))


def int8_rows_bytes(rows: int, k: int) -> int:
    return rows * ((k + 127) // 128 * 128 + 4) if k <= 1 << 30 else 0


def gated_delta_rule_workspace_bytes(tokens: int, count: int, hk: int, hv: int, dk: int, dv: int) -> int:
    """Enough for every chunked call of at most these tokens and sequences."""
    return int(lib().gated_delta_rule_workspace_bytes(tokens, count, hk, hv, dk, dv))


def _norm(fn, x, residual, weight, out, m, k, eps, stream):
    _need(_bf16(x, "x"), _bf(m, k), "x")
    if residual is not None:
        _need(_bf16(residual, "residual"), _bf(m, k), "residual")
    _need(_bf16(weight, "weight"), _bf(1, k), "weight")
    _check(fn(*_ptrs(x, residual, weight, out), m, k, eps, _stream(stream)))


def add_rms_norm_bf16(x, residual, weight, out, m: int, k: int, eps: float = 1e-6, stream=None):
    """residual is updated in place; None: a plain norm of x."""
    _need(_bf16(out, "out"), _bf(m, k), "out")
    _norm(lib().add_rms_norm_bf16, x, residual, weight, out, m, k, eps, stream)


def add_rms_norm_quantize_q8_1(x, residual, weight, out_q8, m: int, k: int, eps: float = 1e-6, stream=None):
    _need(_u8(out_q8, "out_q8"), q8_1_act_bytes(m, k), "out_q8")
    _norm(lib().add_rms_norm_quantize_q8_1, x, residual, weight, out_q8, m, k, eps, stream)


def add_rms_norm_quantize_int8(x, residual, weight, out_i8, m: int, k: int, eps: float = 1e-6, stream=None):
    _need(_u8(out_i8, "out_i8"), int8_rows_bytes(m, k), "out_i8")
    _norm(lib().add_rms_norm_quantize_int8, x, residual, weight, out_i8, m, k, eps, stream)


def quantize_rows_int8(x, out_i8, rows: int, k: int, stream=None):
    _need(_bf16(x, "x"), _bf(rows, k), "x")
    _need(_u8(out_i8, "out_i8"), int8_rows_bytes(rows, k), "out_i8")
    _check(lib().quantize_rows_int8(*_ptrs(x, out_i8), rows, k, _stream(stream)))


def w8a8_gemm(act_i8, w_i8, out, m: int, n: int, k: int, bias=None, stream=None):
    _need(_u8(act_i8, "act_i8"), int8_rows_bytes(m, k), "act_i8")
    _need(_u8(w_i8, "w_i8"), int8_rows_bytes(n, k), "w_i8")
    _need(_bf16(out, "out"), _bf(m, n), "out")
    if bias is not None:
        _need(_bf16(bias, "bias"), _bf(1, n), "bias")
    _check(lib().w8a8_gemm(*_ptrs(act_i8, w_i8, bias, out), m, n, k, _stream(stream)))


def w8a8_gemm_form(m: int, n: int, k: int, cus: int) -> int:
    """The number of the kernel that w8a8_gemm takes on a device of so many compute units (a test hook)."""
    form = lib().w8a8_gemm_form(m, n, k, cus)
    if form < 0:
        _check(form)
    return form


def _typed(t, kind, shape, what):
    """Refuses a tensor that is not of this type and shape."""
    if _kinds.get(t.dtype) != kind and _kind(t) != kind:
        raise TypeError(f"{what}: expected {kind}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {shape}, got {tuple(t.shape)}")


def _strides(t, what):
    """Of a [tokens, heads, d] bf16 tensor, its last dimension contiguous: (token stride, head stride)."""
    if _kinds.get(t.dtype) not in _BF16:
        _bf16(t, what)
    token, head, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return token, head


def _delta(fn, q, k, v, g, beta, out, state, starts, slots, fresh, workspace, scale, l2norm, stream):
    if q.dim() != 3 or v.dim() != 3 or state.dim() != 4 or starts.dim() != 1 or starts.numel() < 1:
        raise ValueError("expected q, k, v as [tokens, heads, d], state as [slots, hv, dk, dv], starts as [count + 1]")
    qk_shape, v_shape = q.shape, v.shape
    (tokens, hk, dk), (_, hv, dv), places, count = qk_shape, v_shape, state.shape[0], starts.numel() - 1
    if k.shape != qk_shape:
        raise ValueError(f"k: expected shape {tuple(qk_shape)}, got {tuple(k.shape)}")
    if v_shape[0] != tokens:
        raise ValueError(f"v: expected {tokens} tokens, got {v_shape[0]}")
    qt, qh = _strides(q, "q")
    kt, kh = _strides(k, "k")
    vt, vh = _strides(v, "v")
    of_heads = (tokens, hv)
    _typed(g, "torch.float32", of_heads, "g")
    _typed(beta, "torch.float32", of_heads, "beta")
    _typed(out, "torch.bfloat16", v_shape, "out")
    _typed(state, "torch.float32", (places, hv, dk, dv), "state")
    _typed(starts, "torch.int32", (count + 1,), "starts")
    if slots is not None:
        _typed(slots, "torch.int32", (count,), "slots")
    elif places < count:
        raise ValueError(f"state: {places} slots for {count} sequences")
    if fresh is not None:
        _typed(fresh, "torch.uint8", (count,), "fresh")
    dev = q.get_device()
    if dev < 0 or k.get_device() != dev or v.get_device() != dev:
        _same_device(q, k, v)
        raise ValueError("expected a device tensor")
    rest = (g, beta, out, state, starts, slots, fresh, *workspace)
    if g.get_device() != dev:
        _same_device(q, *rest)
    _check(fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), *_ptrs(*rest), *map(_nbytes, workspace), tokens, count, places,
              hk, hv, dk, dv, qt, qh, kt, kh, vt, vh, dk ** -0.5 if scale is None else scale, 1 if l2norm else 0,
              _stream(stream)))


def gated_delta_rule_recurrent(q, k, v, g, beta, out, state, starts, slots=None, fresh=None, l2norm: bool = True,
                               scale: float | None = None, stream=None):
    """q, k: [tokens, hk, dk], v: [tokens, hv, dv] bf16, each head's values contiguous; g, beta: [tokens, hv]
    float32; out: [tokens, hv, dv] bf16; state: [slots, hv, dk, dv] float32, updated in place; starts: [count + 1],
    slots: [count] int32; fresh: [count] uint8.  scale: dk ** -0.5 by default."""
    _delta(lib().gated_delta_rule_recurrent, q, k, v, g, beta, out, state, starts, slots, fresh, (), scale, l2norm,
           stream)


def gated_delta_rule_chunked(q, k, v, g, beta, out, state, starts, workspace, slots=None, fresh=None,
                             l2norm: bool = True, scale: float | None = None, stream=None):
    """As gated_delta_rule_recurrent, for prompts; workspace: gated_delta_rule_workspace_bytes(...) bytes, uint8."""
    _delta(lib().gated_delta_rule_chunked, q, k, v, g, beta, out, state, starts, slots, fresh,
           (_u8(workspace, "workspace"),), scale, l2norm, stream)


# ---- paged key-value cache ---------------------------------------------------

def kv_cache_page_bytes(page: int, hk: int, d: int, bits: int = 16) -> int:
    """Bytes of a page of the keys', or the values', cache: a cache of n pages is n times as many."""
    return int(lib().kv_cache_page_bytes(page, hk, d, bits))


def paged_attention_workspace_bytes(tokens: int, count: int, hq: int, hk: int, d: int) -> int:
    """Enough for every paged_attention_decode of at most these tokens and sequences."""
    return int(lib().paged_attention_workspace_bytes(tokens, count, hq, hk, d))


def _paged(k_cache, v_cache, starts, lens, table, page, hk, d, bits):
    """Of the sequences and caches of a call: (count, pages, width)."""
    _u8(k_cache, "k_cache")
    if v_cache.dtype != k_cache.dtype or v_cache.shape != k_cache.shape:
        raise ValueError(f"v_cache: expected the keys' bytes {tuple(k_cache.shape)}, got {v_cache.dtype} {tuple(v_cache.shape)}")
    shape = table.shape
    if len(shape) != 2 or starts.dim() != 1 or starts.shape[0] < 1:
        raise ValueError("expected starts as [count + 1] and table as [count, width]")
    count, width = starts.shape[0] - 1, shape[1]
    if _kinds.get(starts.dtype) != "torch.int32" or starts.dtype != lens.dtype or starts.dtype != table.dtype:
        for t, what in ((starts, "starts"), (lens, "lens"), (table, "table")):
            _typed(t, "torch.int32", t.shape, what)
    if shape[0] != count:
        raise ValueError(f"table: expected [{count}, width], got {tuple(shape)}")
    if lens.shape != (count,):
        raise ValueError(f"lens: expected shape {(count,)}, got {tuple(lens.shape)}")
    # (sizes that the library refuses give no bytes; it says why)
    size, held = hk * page * (2 * d if bits == 16 else d + 4), k_cache.nbytes
    if size > 0 and held % size:
        raise ValueError(f"k_cache: {held} bytes are no whole number of pages of {size}")
    return count, held // size if size > 0 else 0, width


def _beside(q, *tensors):
    """Device pointers of contiguous tensors that lie on q's device; the first is not None."""
    ptrs = _ptrs(*tensors)
    if q.get_device() != tensors[0].get_device():
        _same_device(q, *tensors)
        raise ValueError("expected a device tensor")
    return ptrs


def rope_write_kv_cache(q, k, v, q_out, k_cache, v_cache, starts, lens, table, page: int, bits: int = 16, cos_sin=None,
                        positions=None, axis=None, q_norm=None, k_norm=None, eps: float = 1e-6, stream=None):
    """q: [tokens, hq, d], k, v: [tokens, hk, d] bf16, each head's values contiguous; q_out: [tokens, hq, d] bf16 (q and
    q_out may be None); k_cache, v_cache: uint8, whole pages; starts: [count + 1], lens: [count], table: [count, width]
    int32; cos_sin: [angles, 2, rot / 2] float32; positions: [tokens] or [axes, tokens] int32; axis: [rot / 2] uint8;
    q_norm, k_norm: [d] bf16."""
    if k.dim() != 3 or (q is None) != (q_out is None) or (q is not None and q.dim() != 3):
        raise ValueError("expected q, k, v as [tokens, heads, d], and q_out with q alone")
    tokens, hk, d = k.shape
    hq, rot, angles, axes, qs = 0, 0, 0, 0, (0, 0)
    if v.shape != k.shape:
        raise ValueError(f"v: expected shape {tuple(k.shape)}, got {tuple(v.shape)}")
    if q is not None:
        hq = q.shape[1]
        if q.shape[0] != tokens or q.shape[2] != d:
            raise ValueError(f"q: expected [{tokens}, heads, {d}], got {tuple(q.shape)}")
        qs = _strides(q, "q")
        _typed(q_out, "torch.bfloat16", (tokens, hq, d), "q_out")
    if cos_sin is not None:
        if cos_sin.dim() != 3:
            raise ValueError("expected cos_sin as [angles, 2, rot / 2]")
        angles, _, half = cos_sin.shape
        _typed(cos_sin, "torch.float32", (angles, 2, half), "cos_sin")
        rot = 2 * half
    if axis is not None:
        if positions is None or positions.dim() != 2:
            raise ValueError("expected positions as [axes, tokens] with axis")
        axes = positions.shape[0]
        _typed(axis, "torch.uint8", (rot // 2,), "axis")
        _typed(positions, "torch.int32", (axes, tokens), "positions")
    elif positions is not None:
        _typed(positions, "torch.int32", (tokens,), "positions")
    for w, what in ((q_norm, "q_norm"), (k_norm, "k_norm")):
        if w is not None:
            _typed(w, "torch.bfloat16", (d,), what)
    count, pages, width = _paged(k_cache, v_cache, starts, lens, table, page, hk, d, bits)
    k_at, v_at, *rest = _beside(k, k_cache, v_cache, starts, lens, table, cos_sin, positions, axis, q_norm, k_norm, q_out)
    if v.get_device() != k.get_device() or (q is not None and q.get_device() != k.get_device()):
        raise ValueError("q, k and v on different devices")
    _check(lib().rope_write_kv_cache(None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), rest.pop(), k_at, v_at,
                                     *rest, tokens, count,
                                     pages, page, width, bits, hq, hk, d, rot, angles, axes, *qs, *_strides(k, "k"),
                                     *_strides(v, "v"), eps, _stream(stream)))


def read_kv_cache(k_cache, v_cache, k, v, starts, lens, table, page: int, bits: int = 16, stream=None):
    """The new tokens' rows back: k, v: [tokens, hk, d] bf16; the others as in rope_write_kv_cache."""
    if k.dim() != 3:
        raise ValueError("expected k, v as [tokens, hk, d]")
    tokens, hk, d = k.shape
    _typed(k, "torch.bfloat16", (tokens, hk, d), "k")
    _typed(v, "torch.bfloat16", (tokens, hk, d), "v")
    count, pages, width = _paged(k_cache, v_cache, starts, lens, table, page, hk, d, bits)
    _check(lib().read_kv_cache(*_ptrs(k_cache, v_cache, k, v, starts, lens, table), tokens, count, pages, page, width, bits,
                               hk, d, _stream(stream)))


def _attention(fn, q, k_cache, v_cache, out, starts, lens, table, workspace, hk, page, bits, scale, window, cap, stream):
    if q.dim() != 3:
        raise ValueError("expected q as [tokens, hq, d]")
    tokens, hq, d = q.shape
    qs = _strides(q, "q")
    _typed(out, "torch.bfloat16", q.shape, "out")
    count, pages, width = _paged(k_cache, v_cache, starts, lens, table, page, hk, d, bits)
    rest = _beside(q, k_cache, v_cache, out, starts, lens, table, *workspace)
    _check(fn(q.data_ptr(), *rest, *map(_nbytes, workspace), tokens, count, pages, page, width, bits, hq, hk, d, *qs, window,
              d ** -0.5 if scale is None else scale, cap, _stream(stream)))


def paged_attention_decode(q, k_cache, v_cache, out, starts, lens, table, workspace, hk: int, page: int, bits: int = 16,
                           scale: float | None = None, window: int = 0, cap: float = 0.0, stream=None):
    """q: [tokens, hq, d] bf16, each head's values contiguous; out: [tokens, hq, d] bf16; k_cache, v_cache: uint8, whole
    pages; starts: [count + 1], lens: [count], table: [count, width] int32; workspace:
    paged_attention_workspace_bytes(...) bytes, uint8.  scale: d ** -0.5 by default."""
    _attention(lib().paged_attention_decode, q, k_cache, v_cache, out, starts, lens, table, (_u8(workspace, "workspace"),),
               hk, page, bits, scale, window, cap, stream)


def paged_attention_prefill(q, k_cache, v_cache, out, starts, lens, table, hk: int, page: int, bits: int = 16,
                            scale: float | None = None, window: int = 0, cap: float = 0.0, stream=None):
    """As paged_attention_decode, for prompts."""
    _attention(lib().paged_attention_prefill, q, k_cache, v_cache, out, starts, lens, table, (), hk, page, bits, scale,
               window, cap, stream)


def _blockdots(fn, act_q8, w, w_bytes, out_i32, m0, mt, n0, nt, m, n, k, stream):
    import torch
    _need(_u8(act_q8, "act_q8"), q8_1_act_bytes(m, k), "act_q8")
    _need(_u8(w, "w"), w_bytes, "w")
    if out_i32.dtype != torch.int32:
        raise TypeError(f"out_i32: expected int32, got {out_i32.dtype}")
    _need(out_i32, 4 * mt * nt * (k // 32), "out_i32")
    _check(fn(*_ptrs(act_q8, w, out_i32), m0, mt, n0, nt, m, n, k, _stream(stream)))


def q2_0_mmq_blockdots(act_q8, w_q2, out_i32, m0: int, mt: int, n0: int, nt: int, m: int, n: int, k: int,
                       stream=None):
    _blockdots(lib().q2_0_mmq_blockdots, act_q8, w_q2, q2_0_weight_bytes(n, k), out_i32, m0, mt, n0, nt,
               m, n, k, stream)


def q4k_mmq_blockdots(act_q8, w_q4k, out_i32, m0: int, mt: int, n0: int, nt: int, m: int, n: int, k: int,
                      stream=None):
    _blockdots(lib().q4k_mmq_blockdots, act_q8, w_q4k, q4k_weight_bytes(n, k), out_i32, m0, mt, n0, nt,
               m, n, k, stream)
