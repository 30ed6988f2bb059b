"""Python binding of the gfx950 FP8 runtime chain (``libfp8rt.so``).

Argument marshalling only: every function passes device pointers, sizes and
the current HIP stream to the C ABI of ``include/fp8rt.h`` and raises on a
non-OK status.  All arithmetic runs in the library's HIP kernels; there is no
CPU fallback: calling any function without the built library raises.

Tensors are torch tensors on the GPU: inputs ``float32`` or ``bfloat16``,
FP8 codes ``uint8``, scales ``float32``, counters ``int64`` (read as uint64).
Granularities are ``(rows, cols)`` group extents, 0 meaning the whole
dimension: per-tensor (0, 0), per-row (1, 0), per-group (1, 128),
per-block (128, 128), MX-style (1, 32).
"""
from __future__ import annotations

import ctypes as C
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8rt.so")
# FP8RT_LIB names another build of this library to load instead (the
# host-sanitized build of the CPU checks); there is no fallback either way.
if os.environ.get("FP8RT_LIB"):
    LIB_PATH = os.environ["FP8RT_LIB"]

E4M3, E5M2 = 0, 1
F32, BF16 = 0, 1
DYNAMIC, GIVEN = 0, 1
POW2_SCALES = 1
B_PACKED16 = 2
EXACT_PRODUCTS = 4
EXACT_AUTO_BYTES = 1 << 20
FMAX = {E4M3: 448.0, E5M2: 57344.0}

OK, EINVAL, EALIGN, EUNSUPPORTED, EHIP, ESCRATCH = 0, 1, 2, 3, 4, 5
NOALLOC_SCRATCH_BYTES = 16 << 20


class Fp8rtError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__("%s failed: status %d (%s)" % (fn, status, msg))
        self.status = status


class Gran(C.Structure):
    _fields_ = [("rows", C.c_int32), ("cols", C.c_int32)]


class LedgerSpec(C.Structure):
    _fields_ = [("gran", Gran), ("pow2_round_up", C.c_int32)]


class LedgerRow(C.Structure):
    _fields_ = [("gran", Gran), ("pow2_round_up", C.c_int32), ("qparam_count", C.c_int64),
                ("qparam_bytes", C.c_int64), ("quantized_weight_bytes", C.c_int64),
                ("total_state_bytes", C.c_int64), ("weight_mse", C.c_double),
                ("weight_max_abs_err", C.c_double), ("output_mse", C.c_double),
                ("output_cosine", C.c_double), ("saturated", C.c_uint64), ("underflowed", C.c_uint64)]


_lib = None


def lib():
    """Load the built library; raises if it is missing (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libfp8rt.so is not built: run __graft_entry__.build() "
                              "or python dynamic_scaling_scaled_amd/_build.py")
        L = C.CDLL(LIB_PATH)
        P, I64, I32, F, U32 = C.c_void_p, C.c_int64, C.c_int32, C.c_float, C.c_uint32
        L.fp8rt_status_string.restype = C.c_char_p
        L.fp8rt_status_string.argtypes = [C.c_int]
        L.fp8_amax.restype = C.c_int
        L.fp8_amax.argtypes = [P, C.c_int, I64, I64, I64, Gran, P, P]
        L.fp8_compute_scale.restype = C.c_int
        L.fp8_compute_scale.argtypes = [P, I64, C.c_int, F, I32, P, P, P]
        L.fp8_quantize.restype = C.c_int
        L.fp8_quantize.argtypes = [P, C.c_int, I64, I64, I64, Gran, C.c_int, C.c_int, F, I32, P, P,
                                   P, I64, P, P, P]
        L.fp8_quantize_transpose.restype = C.c_int
        L.fp8_quantize_transpose.argtypes = [P, C.c_int, I64, I64, I64, Gran, C.c_int, C.c_int, F, I32,
                                             P, P, P, I64, P, I64, P, P, P]
        L.fp8_dequantize.restype = C.c_int
        L.fp8_dequantize.argtypes = [P, C.c_int, I64, I64, I64, Gran, P, P, C.c_int, I64, P]
        L.fp8_amax_history_update.restype = C.c_int
        L.fp8_amax_history_update.argtypes = [P, I32, P, P, C.c_int, F, I32, P, P, P]
        L.fp8_scaled_gemm.restype = C.c_int
        L.fp8_scaled_gemm.argtypes = [P, C.c_int, I64, Gran, P, P, C.c_int, I64, Gran, P, I64, I64,
                                      I64, P, C.c_int, P, C.c_int, I64, U32, P]
        L.fp8_scaled_gemm_noalloc.restype = C.c_int
        L.fp8_scaled_gemm_noalloc.argtypes = L.fp8_scaled_gemm.argtypes
        L.fp8_quant_error.restype = C.c_int
        L.fp8_quant_error.argtypes = [P, C.c_int, I64, I64, I64, P, C.c_int, I64, Gran, P, P, I64, I64, P, P]
        L.fp8_granularity_ledger.restype = C.c_int
        L.fp8_granularity_ledger.argtypes = [P, C.c_int, I64, I64, I64, P, I64, I64, C.c_int, F,
                                             C.POINTER(LedgerSpec), I32, C.POINTER(LedgerRow), P]
        L.fp8_delayed_scale_update.restype = C.c_int
        L.fp8_delayed_scale_update.argtypes = [P, I32, P, P, C.c_int, C.c_int, I32, F, I32, P, P, P]
        L.fp8_weight_only_gemm.restype = C.c_int
        L.fp8_weight_only_gemm.argtypes = [P, C.c_int, I64, P, C.c_int, I64, Gran, P, I64, I64, I64, P,
                                           C.c_int, P, C.c_int, I64, U32, P]
        L.fp8_pack_weights16.restype = C.c_int
        L.fp8_pack_weights16.argtypes = [P, I64, I64, I64, P, P]
        L.fp8_quantize_packed16.restype = C.c_int
        L.fp8_quantize_packed16.argtypes = [P, C.c_int, I64, I64, I64, Gran, C.c_int, C.c_int, F, I32, P, P,
                                            P, P, P, P]
        L.fp8_scaled_gemm_fp8out.restype = C.c_int
        L.fp8_scaled_gemm_fp8out.argtypes = [P, C.c_int, I64, Gran, P, P, C.c_int, I64, Gran, P, I64, I64,
                                             I64, P, C.c_int, C.c_int, P, P, P, I64, P, P, U32, P]
        L.fp8_rmsnorm_quantize.restype = C.c_int
        L.fp8_rmsnorm_quantize.argtypes = [P, C.c_int, I64, I64, I64, P, I64, P, C.c_int, F, Gran, C.c_int, C.c_int,
                                           F, I32, P, P, P, I64, P, I64, P, P, P]
        L.fp8_rmsnorm_backward.restype = C.c_int
        L.fp8_rmsnorm_backward.argtypes = [P, C.c_int, I64, I64, I64, P, C.c_int, I64, P, C.c_int, P, P, I64, P,
                                           I64, P, P]
        L.fp8_kv_append.restype = C.c_int
        L.fp8_kv_append.argtypes = [P, P, C.c_int, I64, I64, I64, I64, I64, P, P, I64, I64, P, I64, I64, C.c_int, F, I32,
                                    P, P, P, P, I64, I64, I64, I64, P]
        L.fp8_paged_attention.restype = C.c_int
        L.fp8_paged_attention.argtypes = [P, C.c_int, I64, I64, I64, I64, P, P, P, P, C.c_int, I64, I64, I64, I64, P,
                                          I64, I64, P, P, I64, I64, I64, F, I32, I64, P, C.c_int, I64, I64, P, P]
        L.fp8_call_packed.restype = C.c_int
        L.fp8_call_packed.argtypes = [C.c_char_p, I64]
        _lib = L
    return _lib


def _check(fn, status):
    if status != OK:
        raise Fp8rtError(fn, status, lib().fp8rt_status_string(status).decode())


def _ptr(t):
    # a plain int: the c_void_p argtypes convert it, no object per argument
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:  # the current stream's handle, without a Stream object
        return _raw_stream(_device())
    return torch.cuda.current_stream().cuda_stream


def _dtype(t: torch.Tensor) -> int:
    d = t.dtype
    if d is torch.bfloat16:
        return BF16
    if d is torch.float32:
        return F32
    raise TypeError("expected float32 or bfloat16, got %s" % d)


def _mat(t: torch.Tensor):
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError("expected a 2-D row-major tensor with unit column stride")
    rows, cols = t.shape
    return rows, cols, st[0]


def ngroups(n: int, g: int) -> int:
    return 1 if (g <= 0 or g >= n) else -(-n // g)


def scale_shape(shape, gran):
    return (ngroups(shape[0], gran[0]), ngroups(shape[1], gran[1]))


def fp8_amax(x, gran, amax, stream=None):
    rows, cols, ld = _mat(x)
    _check("fp8_amax", lib().fp8_amax(_ptr(x), _dtype(x), rows, cols, ld, Gran(*gran), _ptr(amax),
                                      _stream(stream)))


def fp8_compute_scale(amax, fmt, eps, pow2_round_up, scale, inv_scale=None, stream=None):
    _check("fp8_compute_scale", lib().fp8_compute_scale(_ptr(amax), amax.numel(), fmt, eps,
                                                        int(pow2_round_up), _ptr(scale),
                                                        _ptr(inv_scale), _stream(stream)))


def fp8_quantize(x, gran, fmt, mode, eps, pow2_round_up, scale, inv_scale, q, amax_out=None,
                 sat_underflow=None, stream=None):
    rows, cols, ld = _mat(x)
    _, _, ldq = _mat(q)
    _check("fp8_quantize", lib().fp8_quantize(_ptr(x), _dtype(x), rows, cols, ld, Gran(*gran), fmt,
                                              mode, eps, int(pow2_round_up), _ptr(scale),
                                              _ptr(inv_scale), _ptr(q), ldq, _ptr(amax_out),
                                              _ptr(sat_underflow), _stream(stream)))


def fp8_quantize_transpose(x, gran, fmt, mode, eps, pow2_round_up, scale, inv_scale, q, qt,
                           amax_out=None, sat_underflow=None, stream=None):
    rows, cols, ld = _mat(x)
    _, _, ldq = _mat(q)
    qr, qc, ldqt = _mat(qt)
    if (qr, qc) != (cols, rows):
        raise ValueError("qt must be [cols x rows]")
    _check("fp8_quantize_transpose",
           lib().fp8_quantize_transpose(_ptr(x), _dtype(x), rows, cols, ld, Gran(*gran), fmt, mode, eps,
                                        int(pow2_round_up), _ptr(scale), _ptr(inv_scale), _ptr(q), ldq,
                                        _ptr(qt), ldqt, _ptr(amax_out), _ptr(sat_underflow),
                                        _stream(stream)))


def fp8_dequantize(q, fmt, gran, scale, y, stream=None):
    rows, cols, ldq = _mat(q)
    _, _, ldy = _mat(y)
    _check("fp8_dequantize", lib().fp8_dequantize(_ptr(q), fmt, rows, cols, ldq, Gran(*gran),
                                                  _ptr(scale), _ptr(y), _dtype(y), ldy,
                                                  _stream(stream)))


def fp8_amax_history_update(history, head, amax_new, fmt, eps, pow2_round_up, scale_next,
                            inv_scale_next=None, stream=None):
    _check("fp8_amax_history_update",
           lib().fp8_amax_history_update(_ptr(history), history.numel(), _ptr(head), _ptr(amax_new),
                                         fmt, eps, int(pow2_round_up), _ptr(scale_next),
                                         _ptr(inv_scale_next), _stream(stream)))


class PackedWeights:
    """A fragment-ordered weight image (fp8_pack_weights16): the uint8 device
    tensor `data` and the logical shape [N x K] of the codes it holds."""

    def __init__(self, data, N, K):
        self.data, self.N, self.K = data, int(N), int(K)

    def data_ptr(self):
        return self.data.data_ptr()


def packed16_bytes(N, K):
    return (N + 15) // 16 * 16 * K


def fp8_pack_weights16(q, out=None, stream=None):
    """Fragment-ordered image of row-major codes q [N x K] (K % 128 == 0)."""
    if q.dtype != torch.uint8:
        raise ValueError("q must be uint8 codes")
    N, K, ldq = _mat(q)
    if out is None:
        out = torch.empty(packed16_bytes(N, K), dtype=torch.uint8, device=q.device)
    if out.dtype != torch.uint8 or not out.is_contiguous() or out.numel() < packed16_bytes(N, K):
        raise ValueError("out must be contiguous uint8 with packed16_bytes(N, K) bytes")
    _check("fp8_pack_weights16", lib().fp8_pack_weights16(_ptr(q), N, K, ldq, _ptr(out), _stream(stream)))
    return PackedWeights(out, N, K)


def fp8_quantize_packed16(x, gran, fmt, mode, eps, pow2_round_up, scale, inv_scale, out=None, amax_out=None,
                          sat_underflow=None, stream=None):
    """fp8_quantize of x [N x K] with the codes written straight into the
    fragment-ordered weight image (K % 128 == 0); returns PackedWeights."""
    rows, cols, ld = _mat(x)
    if out is None:
        out = torch.empty(packed16_bytes(rows, cols), dtype=torch.uint8, device=x.device)
    if out.dtype != torch.uint8 or not out.is_contiguous() or out.numel() < packed16_bytes(rows, cols):
        raise ValueError("out must be contiguous uint8 with packed16_bytes(N, K) bytes")
    _check("fp8_quantize_packed16",
           lib().fp8_quantize_packed16(_ptr(x), _dtype(x), rows, cols, ld, Gran(*gran), fmt, mode, eps,
                                       int(pow2_round_up), _ptr(scale), _ptr(inv_scale), _ptr(out),
                                       _ptr(amax_out), _ptr(sat_underflow), _stream(stream)))
    return PackedWeights(out, rows, cols)


def _weight(b, flags):
    """(N, K, ld, flags) of a row-major code matrix or a PackedWeights."""
    if isinstance(b, PackedWeights):
        return b.N, b.K, b.K, flags | B_PACKED16
    N, K, ld = _mat(b)
    return N, K, ld, flags


def fp8_scaled_gemm(a, fa, ga, scale_a, b, fb, gb, scale_b, y, bias=None, flags=0, stream=None):
    M, K, lda = _mat(a)
    N, K2, ldb, flags = _weight(b, flags)
    if K2 != K:
        raise ValueError("A and B disagree on K")
    _, _, ldy = _mat(y)
    bias_t = _dtype(bias) if bias is not None else F32
    _check("fp8_scaled_gemm",
           lib().fp8_scaled_gemm(_ptr(a), fa, lda, Gran(*ga), _ptr(scale_a), _ptr(b), fb, ldb,
                                 Gran(*gb), _ptr(scale_b), M, N, K, _ptr(bias), bias_t, _ptr(y),
                                 _dtype(y), ldy, flags, _stream(stream)))


def fp8_scaled_gemm_noalloc(a, fa, ga, scale_a, b, fb, gb, scale_b, y, bias=None, flags=0, stream=None):
    """fp8_scaled_gemm on the library's fixed device scratch: allocates nothing."""
    M, K, lda = _mat(a)
    N, K2, ldb, flags = _weight(b, flags)
    if K2 != K:
        raise ValueError("A and B disagree on K")
    _, _, ldy = _mat(y)
    bias_t = _dtype(bias) if bias is not None else F32
    _check("fp8_scaled_gemm_noalloc",
           lib().fp8_scaled_gemm_noalloc(_ptr(a), fa, lda, Gran(*ga), _ptr(scale_a), _ptr(b), fb, ldb,
                                         Gran(*gb), _ptr(scale_b), M, N, K, _ptr(bias), bias_t, _ptr(y),
                                         _dtype(y), ldy, flags, _stream(stream)))


def raw_call(name: str, *args) -> int:
    """Call a C entry point with raw ctypes arguments; returns the status."""
    return getattr(lib(), name)(*args)


def fp8_scaled_gemm_fp8out(a, fa, ga, scale_a, b, fb, gb, scale_b, yq, fy, scale_y, inv_scale_y=None,
                           amax_y=None, sat_underflow=None, bias=None, flags=0, stream=None):
    M, K, lda = _mat(a)
    N, K2, ldb, flags = _weight(b, flags)
    if K2 != K:
        raise ValueError("A and B disagree on K")
    My, Ny, ldy = _mat(yq)
    if (My, Ny) != (M, N) or yq.dtype != torch.uint8:
        raise ValueError("yq must be uint8 [M x N]")
    bt = F32 if bias is None else _dtype(bias)
    _check("fp8_scaled_gemm_fp8out",
           lib().fp8_scaled_gemm_fp8out(_ptr(a), fa, lda, Gran(*ga), _ptr(scale_a), _ptr(b), fb, ldb, Gran(*gb),
                                        _ptr(scale_b), M, N, K, _ptr(bias), bt, fy, _ptr(scale_y),
                                        _ptr(inv_scale_y), _ptr(yq), ldy, _ptr(amax_y), _ptr(sat_underflow),
                                        flags, _stream(stream)))


HIST_MAX, HIST_LATEST = 0, 1


def fp8_quant_error(w, q, fmt, gran, scale, stats, x=None, stream=None):
    """stats (float64[7] on the device) <- the quantization error sums of w
    restored from (q, scale); x: optional bf16 inputs [M, K]."""
    N, K, ldw = _mat(w)
    Nq, Kq, ldq = _mat(q)
    if (Nq, Kq) != (N, K) or q.dtype != torch.uint8:
        raise ValueError("q must be uint8 [N x K]")
    if stats.dtype != torch.float64 or stats.numel() < 7:
        raise ValueError("stats must be float64 with 7 entries")
    M, ldx = 0, 0
    if x is not None:
        M, Kx, ldx = _mat(x)
        if Kx != K:
            raise ValueError("x and w disagree on K")
    _check("fp8_quant_error",
           lib().fp8_quant_error(_ptr(w), _dtype(w), N, K, ldw, _ptr(q), fmt, ldq, Gran(*gran), _ptr(scale),
                                 _ptr(x), M, ldx, _ptr(stats), _stream(stream)))


def fp8_granularity_ledger(w, fmt, specs, x=None, eps=1e-12, stream=None):
    """Quantizes w at each (gran, pow2) spec and returns the ledger rows as
    dicts (scale count and bytes, weight / output error, counters)."""
    N, K, ldw = _mat(w)
    M, ldx = 0, 0
    if x is not None:
        M, Kx, ldx = _mat(x)
        if Kx != K:
            raise ValueError("x and w disagree on K")
    sp = (LedgerSpec * len(specs))(*[LedgerSpec(Gran(*g), int(p)) for g, p in specs])
    rows = (LedgerRow * len(specs))()
    _check("fp8_granularity_ledger",
           lib().fp8_granularity_ledger(_ptr(w), _dtype(w), N, K, ldw, _ptr(x), M, ldx, fmt, eps, sp, len(specs),
                                        rows, _stream(stream)))
    out = []
    for r in rows:
        d = {k: getattr(r, k) for k, _ in LedgerRow._fields_ if k != "gran"}
        d["gran"] = (r.gran.rows, r.gran.cols)
        out.append(d)
    return out


def fp8_delayed_scale_update(history, head, amax_new, fmt, fn, margin, eps, pow2, scale_next,
                             inv_scale_next=None, stream=None):
    """Delayed-scaling recipe step: push amax_new into the ring, derive the
    next (s, r) from f * 2^margin (f = window max or latest amax)."""
    if history.dtype != torch.float32 or history.dim() != 1 or not history.is_contiguous():
        raise ValueError("history must be a contiguous float32 vector")
    _check("fp8_delayed_scale_update",
           lib().fp8_delayed_scale_update(_ptr(history), history.numel(), _ptr(head), _ptr(amax_new), fmt, fn,
                                          margin, eps, int(pow2), _ptr(scale_next), _ptr(inv_scale_next),
                                          _stream(stream)))


def fp8_weight_only_gemm(x, w, fw, gw, scale_w, y, bias=None, flags=0, stream=None):
    """y = x (s_w o dec(w))^T + bias: x [M, K] bf16, w [N, K] uint8 codes or
    their PackedWeights image."""
    M, K, ldx = _mat(x)
    N, K2, ldw, flags = _weight(w, flags)
    if K2 != K:
        raise ValueError("x and w disagree on K")
    _, _, ldy = _mat(y)
    bt = F32 if bias is None else _dtype(bias)
    _check("fp8_weight_only_gemm",
           lib().fp8_weight_only_gemm(_ptr(x), _dtype(x), ldx, _ptr(w), fw, ldw, Gran(*gw), _ptr(scale_w),
                                      M, N, K, _ptr(bias), bt, _ptr(y), _dtype(y), ldy, flags,
                                      _stream(stream)))


# At a decode step's sizes the calls below are bound by this side, not by the
# GPU: their checks read each tensor attribute once, and their arguments go as one
# record of 64-bit words (31 ctypes arguments take 3.2 us, the record 0.9).
_NORM = struct.Struct("10qd4qd10q")
_GRAD = struct.Struct("18q")
_APPEND = struct.Struct("17qd10q")
_ATTEND = struct.Struct("24qd8q")


def _call(fn, record):
    st = lib().fp8_call_packed(record, len(record) >> 3)
    if st:
        _check(fn, st)


def _rows(name, t, shape, dtype=None):
    """Leading dimension of a row-major matrix of this shape (and type)."""
    st = t.stride()
    if t.shape != shape or st[1] != 1 or (dtype is not None and t.dtype is not dtype):
        raise ValueError("%s must be row-major [%d x %d]%s" % (name, *shape, "" if dtype is None else " %s" % dtype))
    return st[0]


def _vec(name, t, n, dtype=None):
    if t.shape != (n,) or not t.is_contiguous() or (dtype is not None and t.dtype is not dtype):
        raise ValueError("%s must be a contiguous vector of %d%s" % (name, n, "" if dtype is None else " %s" % dtype))
    return t.data_ptr()


def _per_group(name, t, n):
    if t.dtype is not torch.float32 or t.numel() < n or not t.is_contiguous():
        raise ValueError("%s must be contiguous float32 with one entry per group" % name)
    return t.data_ptr()


def fp8_rmsnorm_quantize(x, weight, norm_eps, gran, fmt, mode, eps, pow2_round_up, scale, q, residual=None,
                         h=None, rstd=None, inv_scale=None, amax_out=None, stream=None):
    """Codes q and scales of RMSnorm(x + residual) * weight; h receives x + residual
    (rounded to x's type), rstd [rows] the norm's factors for the gradient."""
    rows, cols, ld = _mat(x)
    shape, dtype = (rows, cols), x.dtype
    gr, gc = gran
    n = ngroups(rows, gr) * ngroups(cols, gc)
    ldr = ldh = pr = ph = 0
    if residual is not None:
        ldr, pr = _rows("residual", residual, shape, dtype), residual.data_ptr()
    if h is not None:
        ldh, ph = _rows("h", h, shape, dtype), h.data_ptr()
    _call("fp8_rmsnorm_quantize", _NORM.pack(
        0, x.data_ptr(), _dtype(x), rows, cols, ld, pr, ldr, _vec("weight", weight, cols), _dtype(weight),
        norm_eps, gr, gc, fmt, mode, eps, pow2_round_up, _per_group("scale", scale, n),
        0 if inv_scale is None else _per_group("inv_scale", inv_scale, n), q.data_ptr(),
        _rows("q", q, shape, torch.uint8), ph, ldh, 0 if rstd is None else _vec("rstd", rstd, rows, torch.float32),
        0 if amax_out is None else _per_group("amax_out", amax_out, n), _stream(stream)))


def fp8_rmsnorm_backward(dy, h, weight, rstd, dx, dweight=None, dresidual=None, stream=None):
    """dx (the gradient of h = x + residual, dresidual added) and dweight of
    fp8_rmsnorm_quantize, the cast taken as the identity."""
    rows, cols, lddy = _mat(dy)
    shape, dtype = (rows, cols), dy.dtype
    ldr = pr = 0
    if dresidual is not None:
        ldr, pr = _rows("dresidual", dresidual, shape, dtype), dresidual.data_ptr()
    _call("fp8_rmsnorm_backward", _GRAD.pack(
        1, dy.data_ptr(), _dtype(dy), rows, cols, lddy, h.data_ptr(), _dtype(h), _rows("h", h, shape),
        _vec("weight", weight, cols), _dtype(weight), _vec("rstd", rstd, rows, torch.float32), pr, ldr,
        dx.data_ptr(), _rows("dx", dx, shape, dtype),
        0 if dweight is None else _vec("dweight", dweight, cols, torch.float32), _stream(stream)))


def _paged(k_cache, v_cache, k_scale, v_scale, block_table, seq_start, kv_len):
    """(cache shape, width and leading dimension of the table, sequences) of a paged cache and a batch's plan."""
    shape, u8, f32, i32 = k_cache.shape, torch.uint8, torch.float32, torch.int32
    if (len(shape) != 4 or v_cache.shape != shape or k_cache.dtype is not u8 or v_cache.dtype is not u8
            or not k_cache.is_contiguous() or not v_cache.is_contiguous()):
        raise ValueError("k_cache and v_cache must be contiguous uint8 [pages x heads x page_size x head_dim]")
    if (k_scale.dtype is not f32 or v_scale.dtype is not f32 or k_scale.shape != shape[:2]
            or v_scale.shape != k_scale.shape or not k_scale.is_contiguous() or not v_scale.is_contiguous()):
        raise ValueError("k_scale and v_scale must be contiguous float32 [pages x heads]")
    seqs, st, tab = kv_len.numel(), block_table.stride(), block_table.shape
    if (block_table.dtype is not i32 or seq_start.dtype is not i32 or kv_len.dtype is not i32 or len(st) != 2
            or st[1] != 1 or tab[0] != seqs or seq_start.numel() != seqs + 1
            or not seq_start.is_contiguous() or not kv_len.is_contiguous()):
        raise ValueError("block_table [seqs x n], seq_start [seqs + 1] and kv_len [seqs] must be int32 rows")
    return shape, tab[1], max(st[0], tab[1]) if seqs == 1 else st[0], seqs  # (one row: any stride)


def fp8_kv_append(k, v, k_cache, v_cache, k_scale, v_scale, fmt, block_table, seq_start, kv_len, max_new, eps=1e-12,
                  pow2_round_up=False, stream=None):
    """Quantizes new keys and values [tokens x heads x head_dim] into a paged cache of FP8 codes
    [pages x heads x page_size x head_dim] with one scale per page and head."""
    (pages, heads, page, dim), width, ldt, seqs = _paged(k_cache, v_cache, k_scale, v_scale, block_table, seq_start, kv_len)
    shape, sk, sv = k.shape, k.stride(), v.stride()
    if (shape[1:] != (heads, dim) or v.shape != shape or v.dtype is not k.dtype or sk[2] != 1 or sv[2] != 1):
        raise ValueError("k and v must be [tokens x heads x head_dim] of one type with unit last stride")
    _call("fp8_kv_append", _APPEND.pack(
        2, k.data_ptr(), v.data_ptr(), _dtype(k), shape[0], sk[0], sk[1], sv[0], sv[1], seq_start.data_ptr(),
        kv_len.data_ptr(), seqs, max_new, block_table.data_ptr(), width, ldt, fmt, eps, pow2_round_up,
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, heads, page, dim,
        _stream(stream)))


def fp8_paged_attention(q, k_cache, v_cache, k_scale, v_scale, fmt, block_table, seq_start, kv_len, max_new, max_kv,
                        sm_scale, y, causal=True, window=0, lse=None, stream=None):
    """y = attention of the new tokens' queries q [tokens x q_heads x head_dim] (bf16) over the paged FP8
    cache; max_new and max_kv bound the new tokens and the length of one sequence."""
    (pages, heads, page, dim), width, ldt, seqs = _paged(k_cache, v_cache, k_scale, v_scale, block_table, seq_start, kv_len)
    tokens, qh, qd = shape = q.shape
    sq, sy = q.stride(), y.stride()
    if qd != dim or y.shape != shape or sq[2] != 1 or sy[2] != 1:
        raise ValueError("q and y must be [tokens x q_heads x head_dim] with unit last stride")
    if lse is not None and (lse.shape != (tokens, qh) or lse.dtype is not torch.float32 or not lse.is_contiguous()):
        raise ValueError("lse must be contiguous float32 [tokens x q_heads]")
    _call("fp8_paged_attention", _ATTEND.pack(
        3, q.data_ptr(), _dtype(q), tokens, qh, sq[0], sq[1], k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), fmt, pages, heads, page, dim, block_table.data_ptr(), width, ldt,
        seq_start.data_ptr(), kv_len.data_ptr(), seqs, max_new, max_kv, sm_scale, causal, window, y.data_ptr(),
        _dtype(y), sy[0], sy[1], 0 if lse is None else lse.data_ptr(), _stream(stream)))


__all__ = ["fp8_rmsnorm_quantize", "fp8_rmsnorm_backward", "fp8_kv_append", "fp8_paged_attention",
           "fp8_pack_weights16", "fp8_quantize_packed16", "PackedWeights", "packed16_bytes", "B_PACKED16", "fp8_quant_error", "fp8_granularity_ledger", "LedgerSpec", "LedgerRow", "fp8_delayed_scale_update", "HIST_MAX", "HIST_LATEST", "fp8_weight_only_gemm", "fp8_scaled_gemm_fp8out", "fp8_amax", "fp8_compute_scale", "fp8_quantize", "fp8_quantize_transpose", "fp8_dequantize",
           "fp8_amax_history_update", "fp8_scaled_gemm", "lib", "raw_call", "Gran", "Fp8rtError",
           "E4M3", "E5M2", "F32", "BF16", "DYNAMIC", "GIVEN", "POW2_SCALES", "EXACT_PRODUCTS", "EXACT_AUTO_BYTES", "FMAX", "ngroups",
           "scale_shape"]
