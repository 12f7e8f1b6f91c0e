"""Python binding of the gfx950 ragged-M grouped GEMM library.

Argument marshalling only: every step of the computation runs in the HIP
library (``libmoe_ragged_grouped_amd.so``, built from ``csrc/``). PyTorch
supplies device memory and the stream. There is no fallback: if the library
is missing or a call fails, an exception is raised.

    C = grouped_gemm(A, B, offsets)            # A [M_cap,K] bf16, B [E,K,N] bf16,
                                               # offsets int32 [E+1], C [M_cap,N] fp32
"""

from __future__ import annotations

import ctypes
import os

__all__ = ["grouped_gemm", "grouped_gemm_swiglu", "grouped_gemm_gather",
           "grouped_gemm_gather_combine", "grouped_gemm_fp8w", "grouped_gemm_fp8",
           "grouped_gemm_fp8_swiglu", "grouped_gemm_dgrad", "grouped_gemm_dgrad_swiglu",
           "grouped_gemm_wgrad", "mx4_quantize", "mx4_quantize_weights", "mx4_dequantize",
           "grouped_gemm_mx4", "grouped_gemm_mx4_swiglu", "fp8_quantize", "fp8_quantize_weights",
           "grouped_gemm_fp8_block", "grouped_gemm_fp8_block_swiglu", "expert_sort", "expert_spread",
           "expert_combine", "expert_combine_grad", "rms_norm_fp8", "rms_norm_grad", "tile_schedule", "library_path", "load_library",
           "traced_grouped_gemm", "trace_library_path", "load_trace_library",
           "GroupedGemmError", "BM_CHOICES", "TILE_N", "MAX_EXPERTS", "SYMBOLS",
           "TRACE_SYMBOLS", "TRACE_WORKGROUPS", "TRACE_RECORD"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmoe_ragged_grouped_amd.so")

BM_CHOICES = (16, 32, 64, 128, 256)
# narrowest tile width: sizes the host-side upper bound of the tile count
TILE_N = 256
MAX_EXPERTS = 1024
SYMBOLS = ("gg_grouped_gemm_bf16", "gg_grouped_gemm_bf16_bf16out", "gg_grouped_gemm_bf16_swiglu",
           "gg_grouped_gemm_bf16_gather", "gg_grouped_gemm_bf16_gather_combine",
           "gg_grouped_gemm_fp8w", "gg_grouped_gemm_fp8", "gg_grouped_gemm_fp8_bf16out",
           "gg_grouped_gemm_fp8_swiglu", "gg_grouped_gemm_bf16_dgrad",
           "gg_grouped_gemm_bf16_dgrad_bf16out", "gg_grouped_gemm_bf16_dgrad_swiglu",
           "gg_grouped_gemm_bf16_wgrad", "gg_grouped_gemm_bf16_wgrad_bf16out", "gg_mx4_quantize",
           "gg_mx4_quantize_weights", "gg_mx4_dequantize", "gg_grouped_gemm_mx4",
           "gg_grouped_gemm_mx4_bf16out", "gg_grouped_gemm_mx4_swiglu", "gg_fp8_quantize",
           "gg_fp8_quantize_weights", "gg_grouped_gemm_fp8_block", "gg_grouped_gemm_fp8_block_bf16out",
           "gg_grouped_gemm_fp8_block_swiglu", "gg_expert_sort", "gg_expert_sort_workspace",
           "gg_expert_spread", "gg_expert_combine", "gg_expert_combine_grad", "gg_rms_norm_fp8",
           "gg_rms_norm_grad", "gg_rms_norm_grad_workspace", "gg_tile_schedule",
           "gg_status_string")

# the tracing build (include/grouped_gemm_trace.h): a diagnostic library
_TRACE_LIB_PATH = os.path.join(_HERE, "libmoe_ragged_grouped_amd_trace.so")
TRACE_SYMBOLS = ("gg_trace_grouped_gemm_bf16", "gg_trace_clock_khz")
TRACE_WORKGROUPS = 1024
TRACE_RECORD = 8  # uint64 values per record

_lib = None
_trace_lib = None


class GroupedGemmError(RuntimeError):
    pass


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise GroupedGemmError(
                "HIP library %s is not built; run `python -m moe_ragged_grouped_amd.build`" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        lib.gg_grouped_gemm_bf16.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_bf16.restype = ctypes.c_int
        lib.gg_grouped_gemm_bf16_bf16out.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_bf16_bf16out.restype = ctypes.c_int
        lib.gg_grouped_gemm_bf16_swiglu.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_bf16_swiglu.restype = ctypes.c_int
        lib.gg_grouped_gemm_bf16_gather.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                    i32, vp]
        lib.gg_grouped_gemm_bf16_gather.restype = ctypes.c_int
        lib.gg_grouped_gemm_bf16_gather_combine.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, i32,
                                                            i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_bf16_gather_combine.restype = ctypes.c_int
        lib.gg_grouped_gemm_fp8w.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_fp8w.restype = ctypes.c_int
        lib.gg_grouped_gemm_fp8.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.gg_grouped_gemm_fp8.restype = ctypes.c_int
        lib.gg_grouped_gemm_fp8_bf16out.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                    i32, vp]
        lib.gg_grouped_gemm_fp8_bf16out.restype = ctypes.c_int
        lib.gg_grouped_gemm_fp8_swiglu.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                   i32, vp]
        lib.gg_grouped_gemm_fp8_swiglu.restype = ctypes.c_int
        i64 = ctypes.c_int64
        for name, args in (
                ("gg_grouped_gemm_bf16_dgrad", [vp] * 4 + [i32] * 5),
                ("gg_grouped_gemm_bf16_dgrad_bf16out", [vp] * 4 + [i32] * 5),
                ("gg_grouped_gemm_bf16_dgrad_swiglu", [vp] * 6 + [i32] * 5),
                ("gg_grouped_gemm_bf16_wgrad", [vp] * 4 + [i32] * 5),
                ("gg_grouped_gemm_bf16_wgrad_bf16out", [vp] * 4 + [i32] * 4),
                ("gg_mx4_quantize", [vp] * 3 + [i64, i32]),
                ("gg_mx4_quantize_weights", [vp] * 3 + [i32] * 3),
                ("gg_mx4_dequantize", [vp] * 3 + [i32, i64, i32]),
                ("gg_grouped_gemm_mx4", [vp] * 6 + [i32] * 5),
                ("gg_grouped_gemm_mx4_bf16out", [vp] * 6 + [i32] * 5),
                ("gg_grouped_gemm_mx4_swiglu", [vp] * 6 + [i32] * 5),
                ("gg_fp8_quantize", [vp] * 3 + [i64, i32]),
                ("gg_fp8_quantize_weights", [vp] * 3 + [i32] * 4),
                ("gg_grouped_gemm_fp8_block", [vp] * 6 + [i32] * 5),
                ("gg_grouped_gemm_fp8_block_bf16out", [vp] * 6 + [i32] * 5),
                ("gg_grouped_gemm_fp8_block_swiglu", [vp] * 6 + [i32] * 5),
                ("gg_expert_sort", [vp, i32] + [vp] * 6 + [i64, i32, i32]),
                ("gg_expert_spread", [vp] * 5 + [i32, i64, i32, i64, i32, i64]),
                ("gg_expert_combine", [vp, i32, vp, vp, vp, i32, i64, i32, i32, i64]),
                ("gg_expert_combine_grad", [vp, vp, i32] + [vp] * 4 + [i64, i32, i32, i64]),
                ("gg_rms_norm_fp8", [vp] * 7 + [i64, i32, ctypes.c_float]),
                ("gg_rms_norm_grad", [vp] * 7 + [i64, i32, ctypes.c_float])):
            fn = getattr(lib, name)
            fn.argtypes = args + [vp]
            fn.restype = ctypes.c_int
        for name in ("gg_expert_sort_workspace", "gg_rms_norm_grad_workspace"):
            getattr(lib, name).argtypes = [i64, i32]
            getattr(lib, name).restype = i64
        lib.gg_tile_schedule.argtypes = [vp, i32, i32, i32, i32, vp, vp, i32, vp]
        lib.gg_tile_schedule.restype = ctypes.c_int
        lib.gg_status_string.argtypes = [ctypes.c_int]
        lib.gg_status_string.restype = ctypes.c_char_p
        _lib = lib
    return _lib


def _check(status: int, what: str):
    if status != 0:
        msg = load_library().gg_status_string(status).decode()
        raise GroupedGemmError("%s: status %d (%s)" % (what, status, msg))


def _int32(what, sizes):
    """Refuses what the C entry points, which count in int32, would see cut off.
    sizes: all of them OR-ed together, which is one test for the lot. (The
    gradients and 4-bit operators call it only where sizes >> 31 is not 0: on the
    smallest calls the host takes as long as the kernel.)"""
    if sizes >> 31 not in (0, -1):
        _check(3, what)  # GG_ERR_UNSUPPORTED


def _stream_handle(device, stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _new(shape, dtype, like, stream, zero=False):
    """A new tensor beside ``like`` for a call on ``stream`` to write: made (and
    cleared) in that stream's order, and kept for the present stream too."""
    import torch
    if stream is None:
        return like.new_zeros(shape, dtype=dtype) if zero else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_zeros(shape, dtype=dtype) if zero else like.new_empty(shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _keep(stream, *tensors):
    """Keeps the memory of a call's tensors until the stream that the caller named
    has passed it, so that they may be dropped at once."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _grouped_args(A, B, offsets, bm):
    """Checks A bf16 [M_cap, K], B bf16 [E, K, N], offsets int32 [E+1] (device,
    contiguous) and that all sizes fit int32; returns E, K, N, M_cap."""
    import torch
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    if A.dim() != 2 or B.dim() != 3 or offsets.dim() != 1:
        raise ValueError("shapes: A [M_cap,K], B [E,K,N], offsets [E+1]")
    if not (A.is_cuda and B.is_cuda and offsets.is_cuda):
        raise ValueError("A, B and offsets must be device tensors")
    if not (A.is_contiguous() and B.is_contiguous() and offsets.is_contiguous()):
        raise ValueError("A, B and offsets must be contiguous")
    E, K, N = B.shape
    M_cap = A.shape[0]
    if A.shape[1] != K or offsets.shape[0] != E + 1:
        raise ValueError("shape mismatch: A %s, B %s, offsets %s" % (tuple(A.shape), tuple(B.shape),
                                                                      tuple(offsets.shape)))
    _int32("grouped_gemm", E | K | N | M_cap | int(bm))
    return E, K, N, M_cap


def grouped_gemm(A, B, offsets, out=None, bm: int = 0, stream=None, out_dtype=None):
    """C[off[e]:off[e+1]] = A[off[e]:off[e+1]] @ B[e] for every expert e, in one launch.

    A: bf16 [M_cap, K]; B: bf16 [E, K, N]; offsets: int32 [E+1] (device);
    out: optional fp32 or bf16 [M_cap, N] (out_dtype, default fp32, when out
    is not given); bm: 0 (per-expert choice on the device) or
    16/32/64/128/256. A bf16 ``out`` receives the fp32 result rounded to
    nearest even. Rows of ``out`` at or past offsets[E] are left as they
    were. Enqueued on ``stream`` (default: torch's current stream).
    """
    import torch
    lib = load_library()
    E, K, N, M_cap = _grouped_args(A, B, offsets, bm)
    if out is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        if dt not in (torch.float32, torch.bfloat16):
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out = _new((M_cap, N), dt, A, stream)
    elif (out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (M_cap, N)
          or not out.is_contiguous() or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError("out must be a contiguous fp32 or bf16 [M_cap, N] tensor")
    fn = lib.gg_grouped_gemm_bf16 if out.dtype == torch.float32 else lib.gg_grouped_gemm_bf16_bf16out
    st = fn(A.data_ptr(), B.data_ptr(), offsets.data_ptr(), out.data_ptr(), E, K, N, M_cap, int(bm),
            _stream_handle(A.device, stream))
    _check(st, fn.__name__)
    _keep(stream, A, B, offsets, out)
    return out


def grouped_gemm_swiglu(A, B, offsets, out=None, bm: int = 0, stream=None):
    """H[r, j] = silu(C[r, 2j]) * C[r, 2j+1] for C = the grouped product, in one launch.

    A, B, offsets, bm and stream as in grouped_gemm; B's columns hold the
    gate and up projections interleaved (column 2j gate j, column 2j+1 up j).
    out: optional bf16 [M_cap, N // 2]. The activation runs in fp32 in the
    kernel's epilogue and is rounded once to bf16. Rows at or past
    offsets[E] are left as they were.
    """
    import torch
    lib = load_library()
    E, K, N, M_cap = _grouped_args(A, B, offsets, bm)
    if out is None:
        out = _new((M_cap, N // 2), torch.bfloat16, A, stream)
    elif (out.dtype != torch.bfloat16 or tuple(out.shape) != (M_cap, N // 2)
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 [M_cap, N // 2] tensor")
    st = lib.gg_grouped_gemm_bf16_swiglu(A.data_ptr(), B.data_ptr(), offsets.data_ptr(),
                                         out.data_ptr(), E, K, N, M_cap, int(bm),
                                         _stream_handle(A.device, stream))
    _check(st, "gg_grouped_gemm_bf16_swiglu")
    _keep(stream, A, B, offsets, out)
    return out


def grouped_gemm_gather(X, src_rows, B, offsets, dst_rows=None, out=None, bm: int = 0,
                        stream=None):
    """The grouped product with rows gathered and scattered by index, in one launch.

    X: bf16 [n_src, K]; src_rows: int32 [M_cap] (device): grouped row r reads
    X[src_rows[r]] (rows of expert e are offsets[e]..offsets[e+1]-1);
    dst_rows: optional int32 [M_cap]: grouped row r is written to
    out[dst_rows[r]] (default: out[r]); B, offsets, bm, stream as in
    grouped_gemm; out: optional fp32 [M_cap, N]. Indices out of range read
    zeros (src) or are not written (dst).
    """
    import torch
    lib = load_library()
    if X.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("X and B must be bfloat16")
    if src_rows.dtype != torch.int32 or offsets.dtype != torch.int32 or (
            dst_rows is not None and dst_rows.dtype != torch.int32):
        raise TypeError("src_rows, dst_rows and offsets must be int32")
    if X.dim() != 2 or B.dim() != 3 or offsets.dim() != 1 or src_rows.dim() != 1:
        raise ValueError("shapes: X [n_src,K], src_rows [M_cap], B [E,K,N], offsets [E+1]")
    tensors = [X, B, offsets, src_rows] + ([dst_rows] if dst_rows is not None else [])
    if not all(t.is_cuda and t.is_contiguous() for t in tensors):
        raise ValueError("all tensors must be contiguous device tensors")
    E, K, N = B.shape
    n_src, M_cap = X.shape[0], src_rows.shape[0]
    if X.shape[1] != K or offsets.shape[0] != E + 1 or (
            dst_rows is not None and dst_rows.shape[0] != M_cap):
        raise ValueError("shape mismatch")
    _int32("grouped_gemm_gather", E | K | N | M_cap | n_src | int(bm))
    if out is None:
        out = _new((M_cap, N), torch.float32, X, stream)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M_cap, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [M_cap, N] tensor")
    st = lib.gg_grouped_gemm_bf16_gather(
        X.data_ptr(), n_src, src_rows.data_ptr(), B.data_ptr(), offsets.data_ptr(), out.data_ptr(),
        dst_rows.data_ptr() if dst_rows is not None else None, E, K, N, M_cap, int(bm),
        _stream_handle(X.device, stream))
    _check(st, "gg_grouped_gemm_bf16_gather")
    _keep(stream, X, src_rows, B, offsets, dst_rows, out)
    return out


def grouped_gemm_gather_combine(X, src_rows, B, offsets, dst_rows, weights, out=None,
                                n_dst=None, bm: int = 0, stream=None):
    """out[dst_rows[r]] += weights[r] * (X[src_rows[r]] @ B[e(r)]) for every routed row r, in one launch.

    X, src_rows, B, offsets, bm, stream as in grouped_gemm_gather; dst_rows
    int32 [M_cap] and weights fp32 [M_cap] (device) are required. out: fp32
    [n_dst, N], accumulated into (default: zeros with n_dst = n_src rows, the
    token rows). Destinations outside [0, n_dst) are skipped. The adds are
    fp32 atomics, so the rounding of each element's sum depends on the order
    the adds land in.
    """
    import torch
    lib = load_library()
    if X.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("X and B must be bfloat16")
    if (src_rows.dtype != torch.int32 or offsets.dtype != torch.int32
            or dst_rows.dtype != torch.int32):
        raise TypeError("src_rows, dst_rows and offsets must be int32")
    if weights.dtype != torch.float32:
        raise TypeError("weights must be float32")
    if (X.dim() != 2 or B.dim() != 3 or offsets.dim() != 1 or src_rows.dim() != 1
            or dst_rows.dim() != 1 or weights.dim() != 1):
        raise ValueError("shapes: X [n_src,K], src_rows/dst_rows/weights [M_cap], B [E,K,N], "
                         "offsets [E+1]")
    tensors = [X, B, offsets, src_rows, dst_rows, weights]
    if not all(t.is_cuda and t.is_contiguous() for t in tensors):
        raise ValueError("all tensors must be contiguous device tensors")
    E, K, N = B.shape
    n_src, M_cap = X.shape[0], src_rows.shape[0]
    if (X.shape[1] != K or offsets.shape[0] != E + 1 or dst_rows.shape[0] != M_cap
            or weights.shape[0] != M_cap):
        raise ValueError("shape mismatch")
    _int32("grouped_gemm_gather_combine", E | K | N | M_cap | n_src | int(n_dst or 0) | int(bm))
    if out is None:
        out = _new((n_src if n_dst is None else int(n_dst), N), torch.float32, X, stream, zero=True)
    elif out.dtype != torch.float32 or out.dim() != 2 or out.shape[1] != N or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [n_dst, N] tensor")
    _int32("grouped_gemm_gather_combine", out.shape[0])
    st = lib.gg_grouped_gemm_bf16_gather_combine(
        X.data_ptr(), n_src, src_rows.data_ptr(), B.data_ptr(), offsets.data_ptr(),
        dst_rows.data_ptr(), weights.data_ptr(), out.data_ptr(), out.shape[0], E, K, N, M_cap,
        int(bm), _stream_handle(X.device, stream))
    _check(st, "gg_grouped_gemm_bf16_gather_combine")
    _keep(stream, X, src_rows, B, offsets, dst_rows, weights, out)
    return out


def grouped_gemm_fp8w(A, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None):
    """The grouped product with fp8 (OCP E4M3) weights and per-column scales.

    A: bf16 [M_cap, K]; Bq: uint8 (or float8_e4m3fn) [E, K, N]; b_scale: fp32
    [E, N]; offsets: int32 [E+1]. out[r, n] = b_scale[e, n] * sum_k A[r, k] *
    Bq[e, k, n] for the rows r of expert e (fp32 [M_cap, N]).
    """
    import torch
    lib = load_library()
    if A.dtype != torch.bfloat16 or Bq.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError("A must be bfloat16 and Bq uint8 / float8_e4m3fn")
    if b_scale.dtype != torch.float32 or offsets.dtype != torch.int32:
        raise TypeError("b_scale must be float32 and offsets int32")
    if A.dim() != 2 or Bq.dim() != 3 or b_scale.dim() != 2 or offsets.dim() != 1:
        raise ValueError("shapes: A [M_cap,K], Bq [E,K,N], b_scale [E,N], offsets [E+1]")
    if not all(t.is_cuda and t.is_contiguous() for t in (A, Bq, b_scale, offsets)):
        raise ValueError("all tensors must be contiguous device tensors")
    E, K, N = Bq.shape
    M_cap = A.shape[0]
    if A.shape[1] != K or tuple(b_scale.shape) != (E, N) or offsets.shape[0] != E + 1:
        raise ValueError("shape mismatch")
    _int32("grouped_gemm_fp8w", E | K | N | M_cap | int(bm))
    if out is None:
        out = _new((M_cap, N), torch.float32, A, stream)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M_cap, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [M_cap, N] tensor")
    st = lib.gg_grouped_gemm_fp8w(A.data_ptr(), Bq.data_ptr(), b_scale.data_ptr(), offsets.data_ptr(),
                                  out.data_ptr(), E, K, N, M_cap, int(bm),
                                  _stream_handle(A.device, stream))
    _check(st, "gg_grouped_gemm_fp8w")
    _keep(stream, A, Bq, b_scale, offsets, out)
    return out


def grouped_gemm_fp8(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None,
                     out_dtype=None):
    """C = (a_scale * dec(Aq)) @ (dec(Bq[e]) * b_scale[e]) per expert, fp8 matrix cores.

    Aq: uint8 [M_cap, K] E4M3 codes; a_scale: fp32 [M_cap]; Bq: uint8
    [E, K, N] E4M3 codes; b_scale: fp32 [E, N]; offsets int32 [E+1]; out:
    optional fp32 or bf16 [M_cap, N] (out_dtype when out is not given,
    default fp32; bf16 is the fp32 result rounded to nearest even). K and N
    must be multiples of 16.
    """
    import torch
    lib = load_library()
    if Aq.dtype != torch.uint8 or Bq.dtype != torch.uint8:
        raise TypeError("Aq and Bq must be uint8 E4M3 codes")
    if a_scale.dtype != torch.float32 or b_scale.dtype != torch.float32:
        raise TypeError("a_scale and b_scale must be float32")
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    if Aq.dim() != 2 or Bq.dim() != 3 or a_scale.dim() != 1 or b_scale.dim() != 2:
        raise ValueError("shapes: Aq [M_cap,K], a_scale [M_cap], Bq [E,K,N], b_scale [E,N]")
    tensors = [Aq, a_scale, Bq, b_scale, offsets]
    if not all(t.is_cuda and t.is_contiguous() for t in tensors):
        raise ValueError("all tensors must be contiguous device tensors")
    E, K, N = Bq.shape
    M_cap = Aq.shape[0]
    if (Aq.shape[1] != K or a_scale.shape[0] != M_cap or tuple(b_scale.shape) != (E, N)
            or offsets.shape[0] != E + 1):
        raise ValueError("shape mismatch")
    _int32("grouped_gemm_fp8", E | K | N | M_cap | int(bm))
    if out is None:
        dt = torch.float32 if out_dtype is None else out_dtype
        if dt not in (torch.float32, torch.bfloat16):
            raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
        out = _new((M_cap, N), dt, Aq, stream)
    elif (out.dtype not in (torch.float32, torch.bfloat16) or tuple(out.shape) != (M_cap, N)
          or not out.is_contiguous() or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError("out must be a contiguous fp32 or bf16 [M_cap, N] tensor")
    fn = lib.gg_grouped_gemm_fp8 if out.dtype == torch.float32 else lib.gg_grouped_gemm_fp8_bf16out
    st = fn(Aq.data_ptr(), a_scale.data_ptr(), Bq.data_ptr(), b_scale.data_ptr(),
            offsets.data_ptr(), out.data_ptr(), E, K, N, M_cap, int(bm),
            _stream_handle(Aq.device, stream))
    _check(st, fn.__name__)
    _keep(stream, Aq, a_scale, Bq, b_scale, offsets, out)
    return out


def grouped_gemm_fp8_swiglu(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0,
                            stream=None):
    """H[r, j] = silu(C[r, 2j]) * C[r, 2j+1] for C = the fp8 x fp8 product.

    Arguments as in grouped_gemm_fp8; Bq's columns interleave gate (even) and
    up (odd); out: optional bf16 [M_cap, N // 2].
    """
    import torch
    lib = load_library()
    if Aq.dtype != torch.uint8 or Bq.dtype != torch.uint8:
        raise TypeError("Aq and Bq must be uint8 E4M3 codes")
    if a_scale.dtype != torch.float32 or b_scale.dtype != torch.float32:
        raise TypeError("a_scale and b_scale must be float32")
    if offsets.dtype != torch.int32:
        raise TypeError("offsets must be int32")
    tensors = [Aq, a_scale, Bq, b_scale, offsets]
    if not all(t.is_cuda and t.is_contiguous() for t in tensors):
        raise ValueError("all tensors must be contiguous device tensors")
    E, K, N = Bq.shape
    M_cap = Aq.shape[0]
    if (Aq.dim() != 2 or Aq.shape[1] != K or tuple(a_scale.shape) != (M_cap,)
            or tuple(b_scale.shape) != (E, N) or tuple(offsets.shape) != (E + 1,)):
        raise ValueError("shape mismatch")
    _int32("grouped_gemm_fp8_swiglu", E | K | N | M_cap | int(bm))
    if out is None:
        out = _new((M_cap, N // 2), torch.bfloat16, Aq, stream)
    elif (out.dtype != torch.bfloat16 or tuple(out.shape) != (M_cap, N // 2)
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous bf16 [M_cap, N // 2] tensor")
    st = lib.gg_grouped_gemm_fp8_swiglu(Aq.data_ptr(), a_scale.data_ptr(), Bq.data_ptr(),
                                        b_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(),
                                        E, K, N, M_cap, int(bm), _stream_handle(Aq.device, stream))
    _check(st, "gg_grouped_gemm_fp8_swiglu")
    _keep(stream, Aq, a_scale, Bq, b_scale, offsets, out)
    return out


# ---- gradients and 4-bit operators

def _device_args(what, *tensors):
    """Checks that every (name, tensor, dtype, rank) is a contiguous device
    tensor of its dtype and rank, all on one device; returns that device."""
    first = tensors[0][1]
    index = first.get_device()
    ok = first.is_cuda
    for _, t, dtype, dims in tensors:
        ok = (ok and t.dtype is dtype and t.dim() == dims and t.is_contiguous()
              and t.get_device() == index)
    if ok:
        return first.device
    for name, t, dtype, dims in tensors:
        if t.dtype is not dtype:
            raise TypeError("%s: %s must be %s" % (what, name, dtype))
        if t.dim() != dims:
            raise ValueError("%s: %s must have %d dimensions, not %d" % (what, name, dims, t.dim()))
    for name, t, _, _ in tensors:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("%s: %s must be a contiguous device tensor" % (what, name))
    for name, t, _, _ in tensors:
        if t.get_device() != index:
            raise ValueError("%s: %s is on device %d, others on %d" % (what, name, t.get_device(), index))


def _match(what, ok, *tensors):
    if not ok:
        raise ValueError("%s: shape mismatch: %s" % (what, ", ".join(str(tuple(t.shape)) for t in tensors)))


def _out(what, out, shape, dtypes, dtype, like, stream):
    """The given output, checked, or a new one of ``dtype`` (default: the first
    of ``dtypes``) beside ``like``."""
    if dtype is not None and dtype not in dtypes:
        raise TypeError("%s: out_dtype must be %s" % (what, " or ".join(str(d) for d in dtypes)))
    if out is None:
        dtype = dtypes[0] if dtype is None else dtype
        if stream is None:
            return like.new_empty(shape, dtype=dtype)
        return _new(shape, dtype, like, stream)
    if (out.dtype not in dtypes or (dtype is not None and out.dtype is not dtype)
            or out.shape != shape or not out.is_contiguous() or out.device != like.device):
        raise ValueError("%s: out must be a contiguous %s %s tensor on %s" % (
            what, " or ".join(str(d) for d in ([dtype] if dtype else dtypes)), list(shape), like.device))
    return out


def _call(name, dev, stream, tensors, *args):
    """Calls one entry point on the tensors' device, whichever is current."""
    import torch
    fn = getattr(load_library(), name)
    if stream is not None:
        if stream.device != dev:
            raise ValueError("%s: the stream is on %s, the tensors on %s" % (name, stream.device, dev))
        handle = stream.cuda_stream
    else:  # torch's current stream as a number: the Stream object costs 2 us
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch._C._cuda_getDevice() == dev.index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st == 1:  # (null pointers do not come from here)
        raise GroupedGemmError("%s: status 1 (invalid size or tile height, or an output that shares "
                               "memory with another array)" % name)
    if st != 0:
        _check(st, name)
    if stream is not None:
        _keep(stream, *tensors)


def grouped_gemm_dgrad(dC, B, offsets, out=None, bm: int = 0, stream=None, out_dtype=None):
    """dA[off[e]:off[e+1]] = dC[off[e]:off[e+1]] @ B[e].T for every expert e, in one launch.

    The gradient of grouped_gemm(A, B, offsets) with respect to A. dC: bf16
    [M_cap, N]; B: bf16 [E, K, N], as the product takes it; out: optional fp32
    or bf16 [M_cap, K] (out_dtype, default fp32, when out is not given; bf16 is
    the fp32 sum rounded to nearest even). offsets, bm and stream as in
    grouped_gemm. Rows at or past offsets[E] are left as they were.

    Here and below: with ``stream``, the call is ordered on that stream alone (it
    waits for no other), and the memory of its tensors is kept until it is done.
    An output may not share memory with another argument.
    """
    import torch
    what = "grouped_gemm_dgrad"
    dev = _device_args(what, ("dC", dC, torch.bfloat16, 2), ("B", B, torch.bfloat16, 3),
                       ("offsets", offsets, torch.int32, 1))
    E, K, N = B.shape
    M_cap = dC.shape[0]
    _match(what, dC.shape[1] == N and offsets.shape[0] == E + 1, dC, B, offsets)
    sizes = E | K | N | M_cap | int(bm)
    if sizes >> 31:
        _int32(what, sizes)
    out = _out(what, out, (M_cap, K), (torch.float32, torch.bfloat16), out_dtype, dC, stream)
    name = "gg_grouped_gemm_bf16_dgrad" + ("" if out.dtype == torch.float32 else "_bf16out")
    _call(name, dev, stream, (dC, B, offsets, out), dC.data_ptr(), B.data_ptr(), offsets.data_ptr(),
          out.data_ptr(), E, K, N, M_cap, int(bm))
    return out


def grouped_gemm_dgrad_swiglu(dY, B, offsets, C, out=None, out_h=None, with_h: bool = False,
                              bm: int = 0, stream=None):
    """The gradient of H = silu(gate) * up, Y = grouped_gemm(H, B, offsets), in one launch.

    dY: bf16 [M_cap, N]; B: bf16 [E, K, N], the down projection; C: bf16
    [M_cap, 2K], gate in column 2j and up in column 2j+1 (grouped_gemm with bf16
    output on interleaved weights). Returns dC, bf16 [M_cap, 2K], the gradient
    of C (``out``, which may be C itself); with with_h or out_h also H, bf16
    [M_cap, K], which the down projection's weight gradient needs. The gradient
    of H stays in fp32 registers; everything is rounded once. Rows at or past
    offsets[E] are left as they were. offsets, bm, stream as in grouped_gemm.
    """
    import torch
    what = "grouped_gemm_dgrad_swiglu"
    bf = torch.bfloat16
    dev = _device_args(what, ("dY", dY, bf, 2), ("B", B, bf, 3), ("offsets", offsets, torch.int32, 1),
                       ("C", C, bf, 2))
    E, K, N = B.shape
    M_cap = dY.shape[0]
    _match(what, dY.shape[1] == N and offsets.shape[0] == E + 1
           and C.shape == (M_cap, 2 * K), dY, B, offsets, C)
    sizes = E | K | N | M_cap | int(bm)
    if sizes >> 31:
        _int32(what, sizes)
    out = _out(what, out, (M_cap, 2 * K), (bf,), None, dY, stream)
    h = None
    if with_h or out_h is not None:
        h = _out(what, out_h, (M_cap, K), (bf,), None, dY, stream)
    outs = (out,) if h is None else (out, h)
    _call("gg_grouped_gemm_bf16_dgrad_swiglu", dev, stream, (dY, B, offsets, C, *outs), dY.data_ptr(),
          B.data_ptr(), offsets.data_ptr(), C.data_ptr(), out.data_ptr(),
          None if h is None else h.data_ptr(), E, K, N, M_cap, int(bm))
    return out if h is None else (out, h)


def grouped_gemm_wgrad(A, dC, offsets, out=None, accumulate: bool = False, stream=None,
                       out_dtype=None):
    """dB[e] = A[off[e]:off[e+1]].T @ dC[off[e]:off[e+1]] for every expert e, in one launch.

    The gradient of grouped_gemm(A, B, offsets) with respect to B. A: bf16
    [M_cap, K]; dC: bf16 [M_cap, N]; offsets: int32 [E+1]; out: optional fp32 or
    bf16 [E, K, N] (out_dtype, default fp32, when out is not given; bf16 is the
    fp32 sum rounded to nearest even). An expert with no rows gets zeros. With
    accumulate the sums are added to ``out``, which must then be given and fp32.
    The sums take no atomics: equal inputs give equal bits, M_cap being one (it
    takes part in the choice of the tile, and so in the order of summation).
    """
    import torch
    what = "grouped_gemm_wgrad"
    dev = _device_args(what, ("A", A, torch.bfloat16, 2), ("dC", dC, torch.bfloat16, 2),
                       ("offsets", offsets, torch.int32, 1))
    M_cap, K = A.shape
    N = dC.shape[1]
    E = offsets.shape[0] - 1
    _match(what, dC.shape[0] == M_cap and E >= 1, A, dC, offsets)
    sizes = E | K | N | M_cap
    if sizes >> 31:
        _int32(what, sizes)
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("%s: accumulate needs an fp32 out to add to" % what)
    out = _out(what, out, (E, K, N), (torch.float32, torch.bfloat16), out_dtype, A, stream)
    args = ((A, dC, offsets, out), A.data_ptr(), dC.data_ptr(), offsets.data_ptr(), out.data_ptr())
    if out.dtype == torch.float32:
        _call("gg_grouped_gemm_bf16_wgrad", dev, stream, *args, int(bool(accumulate)), E, K, N, M_cap)
    else:
        _call("gg_grouped_gemm_bf16_wgrad_bf16out", dev, stream, *args, E, K, N, M_cap)
    return out


def _mx4_slices(K: int) -> int:
    """Slices of 256 k: the first dimension of a scale tensor."""
    return -(-K // 256)


def mx4_quantize(X, out=None, out_scale=None, stream=None):
    """bf16 rows [M, K] -> 4-bit microscaled (codes uint8 [M, K/2], scales uint8 [ceil(K/256), M, 8]).

    Blocks of 32 values along K share the scale 2^(floor(log2 max|x|) - 2); a
    value goes to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times it, ties to the
    even code, at most 6. A block with an infinity or a NaN stands for NaN. K is
    a multiple of 32. Byte j of a row of codes holds k = 2j (low half) and
    2j + 1; block b of row r has its scale byte at scales[b // 8, r, b % 8].
    """
    import torch
    what = "mx4_quantize"
    dev = _device_args(what, ("X", X, torch.bfloat16, 2))
    M, K = X.shape
    if K >> 31:
        _int32(what, K)
    u8 = (torch.uint8,)
    q = _out(what, out, (M, K // 2), u8, None, X, stream)
    s = _out(what, out_scale, (_mx4_slices(K), M, 8), u8, None, X, stream)
    _call("gg_mx4_quantize", dev, stream, (X, q, s), X.data_ptr(), q.data_ptr(), s.data_ptr(), M, K)
    return q, s


def mx4_quantize_weights(B, out=None, out_scale=None, stream=None):
    """bf16 weights [E, K, N] -> (codes uint8 [E, N, K/2], scales uint8 [E, ceil(K/256), N, 8]).

    The rule of mx4_quantize, blocks along K: what grouped_gemm_mx4 takes as
    weights, made once when the weights are loaded.
    """
    import torch
    what = "mx4_quantize_weights"
    dev = _device_args(what, ("B", B, torch.bfloat16, 3))
    E, K, N = B.shape
    sizes = E | K | N
    if sizes >> 31:
        _int32(what, sizes)
    u8 = (torch.uint8,)
    q = _out(what, out, (E, N, K // 2), u8, None, B, stream)
    s = _out(what, out_scale, (E, _mx4_slices(K), N, 8), u8, None, B, stream)
    _call("gg_mx4_quantize_weights", dev, stream, (B, q, s), B.data_ptr(), q.data_ptr(), s.data_ptr(), E,
          K, N)
    return q, s


def mx4_dequantize(q, scales, out=None, stream=None):
    """The bf16 values that 4-bit codes and scales stand for.

    q: uint8 [M, K/2] with scales [ceil(K/256), M, 8], or weights [E, N, K/2]
    with [E, ceil(K/256), N, 8]; returns bf16 [M, K] or [E, N, K].
    """
    import torch
    what = "mx4_dequantize"
    if q.dim() not in (2, 3):
        raise ValueError("%s: codes are [M, K/2] or [E, N, K/2]" % what)
    dev = _device_args(what, ("q", q, torch.uint8, q.dim()), ("scales", scales, torch.uint8, q.dim() + 1))
    batch = q.shape[0] if q.dim() == 3 else 1
    rows, K = q.shape[-2], 2 * q.shape[-1]
    sizes = batch | K
    if sizes >> 31:
        _int32(what, sizes)
    lead = (batch,) if q.dim() == 3 else ()
    _match(what, scales.shape == lead + (_mx4_slices(K), rows, 8), q, scales)
    y = _out(what, out, lead + (rows, K), (torch.bfloat16,), None, q, stream)
    _call("gg_mx4_dequantize", dev, stream, (q, scales, y), q.data_ptr(), scales.data_ptr(),
          y.data_ptr(), batch, rows, K)
    return y


def _mx4_args(what, Aq, a_scale, Bq, b_scale, offsets, bm):
    import torch
    u8 = torch.uint8
    dev = _device_args(what, ("Aq", Aq, u8, 2), ("a_scale", a_scale, u8, 3), ("Bq", Bq, u8, 3),
                       ("b_scale", b_scale, u8, 4), ("offsets", offsets, torch.int32, 1))
    E, N, half = Bq.shape
    M_cap, K = Aq.shape[0], 2 * half
    _match(what, Aq.shape[1] == half and offsets.shape[0] == E + 1
           and a_scale.shape == (_mx4_slices(K), M_cap, 8)
           and b_scale.shape == (E, _mx4_slices(K), N, 8), Aq, a_scale, Bq, b_scale, offsets)
    sizes = E | K | N | M_cap | bm
    if sizes >> 31:
        _int32(what, sizes)
    return dev, E, K, N, M_cap


def grouped_gemm_mx4(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None,
                     out_dtype=None):
    """C = val(Aq, a_scale) @ val(Bq[e], b_scale[e]).T per expert, 4-bit matrix cores, one launch.

    Aq, a_scale: codes and scales of the rows (mx4_quantize); Bq, b_scale: of the
    weights (mx4_quantize_weights); offsets int32 [E+1]; out: optional fp32 or
    bf16 [M_cap, N] (out_dtype when out is not given, default fp32; bf16 is the
    fp32 result rounded to nearest even). N must be a multiple of 8. Rows at or
    past offsets[E] are left as they were. bm and stream as in grouped_gemm.
    """
    import torch
    what = "grouped_gemm_mx4"
    dev, E, K, N, M_cap = _mx4_args(what, Aq, a_scale, Bq, b_scale, offsets, int(bm))
    out = _out(what, out, (M_cap, N), (torch.float32, torch.bfloat16), out_dtype, Aq, stream)
    name = "gg_grouped_gemm_mx4" + ("" if out.dtype == torch.float32 else "_bf16out")
    _call(name, dev, stream, (Aq, a_scale, Bq, b_scale, offsets, out), Aq.data_ptr(), a_scale.data_ptr(),
          Bq.data_ptr(), b_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(), E, K, N, M_cap, int(bm))
    return out


def grouped_gemm_mx4_swiglu(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None):
    """H[r, j] = silu(C[r, 2j]) * C[r, 2j+1] for C = grouped_gemm_mx4 (interleaved columns).

    Arguments of grouped_gemm_mx4; out: optional bf16 [M_cap, N // 2]. The
    activation runs in fp32 in the epilogue and is rounded once to bf16.
    """
    import torch
    what = "grouped_gemm_mx4_swiglu"
    dev, E, K, N, M_cap = _mx4_args(what, Aq, a_scale, Bq, b_scale, offsets, int(bm))
    out = _out(what, out, (M_cap, N // 2), (torch.bfloat16,), None, Aq, stream)
    _call("gg_grouped_gemm_mx4_swiglu", dev, stream, (Aq, a_scale, Bq, b_scale, offsets, out),
          Aq.data_ptr(), a_scale.data_ptr(), Bq.data_ptr(), b_scale.data_ptr(), offsets.data_ptr(),
          out.data_ptr(), E, K, N, M_cap, int(bm))
    return out


# ---- around the experts' products: 8-bit blocks, rows to the experts and back, the norm

_BLOCK = 128
_SORT_RECOUNT = 8192  # choices that gg_expert_sort takes without a workspace, whatever E


def _fp8(t):
    """E4M3 codes, as uint8 or as torch's float8_e4m3fn (either is taken)."""
    import torch
    return torch.float8_e4m3fn if t.dtype is torch.float8_e4m3fn else torch.uint8


def fp8_quantize(X, out=None, out_scale=None, stream=None):
    """bf16 rows [M, K] -> 8 bits (codes float8_e4m3fn [M, K], scales fp32 [ceil(K/128), M]).

    Blocks of 128 values along K share a scale. With top a block's largest
    magnitude (2^-100 at least) and m = 448 / top cut to 16 significant bits, a
    value goes to the code nearest to x * m, ties to even, and the scale is
    1 / m. A block with an infinity or a NaN stands for NaN. K is a multiple of 16.
    """
    import torch
    what = "fp8_quantize"
    dev = _device_args(what, ("X", X, torch.bfloat16, 2))
    M, K = X.shape
    if K >> 31:
        _int32(what, K)
    q = _out(what, out, (M, K), (torch.float8_e4m3fn, torch.uint8), None, X, stream)
    s = _out(what, out_scale, (-(-K // _BLOCK), M), (torch.float32,), None, X, stream)
    _call("gg_fp8_quantize", dev, stream, (X, q, s), X.data_ptr(), q.data_ptr(), s.data_ptr(), M, K)
    return q, s


def fp8_quantize_weights(B, for_grad: bool = False, out=None, out_scale=None, stream=None):
    """bf16 weights [E, K, N] -> (codes float8_e4m3fn [E, N, K], scales fp32 [E, ceil(N/128), ceil(K/128)]).

    The rule of fp8_quantize with blocks of 128 x 128: what grouped_gemm_fp8_block
    takes as weights, made once. With for_grad the same values as codes [E, K, N]
    and scales [E, ceil(K/128), ceil(N/128)]: the weights of the data gradient,
    dA = grouped_gemm_fp8_block(*fp8_quantize(dC), *those, offsets). K is a multiple
    of 16 and N of 8 (for_grad: N of 16 and K of 8).
    """
    import torch
    what = "fp8_quantize_weights"
    dev = _device_args(what, ("B", B, torch.bfloat16, 3))
    E, K, N = B.shape
    sizes = E | K | N
    if sizes >> 31:
        _int32(what, sizes)
    rows, cols = (K, N) if for_grad else (N, K)
    q = _out(what, out, (E, rows, cols), (torch.float8_e4m3fn, torch.uint8), None, B, stream)
    s = _out(what, out_scale, (E, -(-rows // _BLOCK), -(-cols // _BLOCK)), (torch.float32,), None, B, stream)
    _call("gg_fp8_quantize_weights", dev, stream, (B, q, s), B.data_ptr(), q.data_ptr(), s.data_ptr(),
          int(bool(for_grad)), E, K, N)
    return q, s


def _fp8_block_args(what, Aq, a_scale, Bq, b_scale, offsets, bm):
    import torch
    f32 = torch.float32
    dev = _device_args(what, ("Aq", Aq, _fp8(Aq), 2), ("a_scale", a_scale, f32, 2),
                       ("Bq", Bq, _fp8(Bq), 3), ("b_scale", b_scale, f32, 3),
                       ("offsets", offsets, torch.int32, 1))
    E, N, K = Bq.shape
    M_cap = Aq.shape[0]
    slices = -(-K // _BLOCK)
    _match(what, Aq.shape[1] == K and offsets.shape[0] == E + 1 and a_scale.shape == (slices, M_cap)
           and b_scale.shape == (E, -(-N // _BLOCK), slices), Aq, a_scale, Bq, b_scale, offsets)
    sizes = E | K | N | M_cap | bm
    if sizes >> 31:
        _int32(what, sizes)
    return dev, E, K, N, M_cap


def grouped_gemm_fp8_block(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None,
                           out_dtype=None):
    """C = val(Aq, a_scale) @ val(Bq[e], b_scale[e]).T per expert, fp8 matrix cores, one launch.

    Aq, a_scale: E4M3 codes [M_cap, K] (float8_e4m3fn or uint8) and fp32 scales
    [ceil(K/128), M_cap], one for 128 values of a row (fp8_quantize); Bq, b_scale:
    codes [E, N, K] and scales [E, ceil(N/128), ceil(K/128)], one for 128 x 128
    values (fp8_quantize_weights). The scales are any fp32 numbers; where the product
    of two is below fp32's normal numbers, the block's part is off by up to 2^-125. offsets int32 [E+1]; out:
    optional fp32 or bf16 [M_cap, N] (out_dtype when out is not given, default
    fp32; bf16 is the fp32 result rounded to nearest even). K is a multiple of 16,
    N of 8. Rows at or past offsets[E] are left as they were. bm and stream as in
    grouped_gemm. Blocks are scaled and added in fp32; inside a block of 128 the
    matrix cores drop what is 2^-14 of the largest of 8 neighbouring products.
    """
    import torch
    what = "grouped_gemm_fp8_block"
    dev, E, K, N, M_cap = _fp8_block_args(what, Aq, a_scale, Bq, b_scale, offsets, int(bm))
    out = _out(what, out, (M_cap, N), (torch.float32, torch.bfloat16), out_dtype, Aq, stream)
    name = "gg_grouped_gemm_fp8_block" + ("" if out.dtype == torch.float32 else "_bf16out")
    _call(name, dev, stream, (Aq, a_scale, Bq, b_scale, offsets, out), Aq.data_ptr(), a_scale.data_ptr(),
          Bq.data_ptr(), b_scale.data_ptr(), offsets.data_ptr(), out.data_ptr(), E, K, N, M_cap, int(bm))
    return out


def grouped_gemm_fp8_block_swiglu(Aq, a_scale, Bq, b_scale, offsets, out=None, bm: int = 0, stream=None):
    """H[r, j] = silu(C[r, 2j]) * C[r, 2j+1] for C = grouped_gemm_fp8_block (interleaved columns).

    Arguments of grouped_gemm_fp8_block; out: optional bf16 [M_cap, N // 2]. The
    activation runs in fp32 in the epilogue and is rounded once to bf16.
    """
    import torch
    what = "grouped_gemm_fp8_block_swiglu"
    dev, E, K, N, M_cap = _fp8_block_args(what, Aq, a_scale, Bq, b_scale, offsets, int(bm))
    out = _out(what, out, (M_cap, N // 2), (torch.bfloat16,), None, Aq, stream)
    _call("gg_grouped_gemm_fp8_block_swiglu", dev, stream, (Aq, a_scale, Bq, b_scale, offsets, out),
          Aq.data_ptr(), a_scale.data_ptr(), Bq.data_ptr(), b_scale.data_ptr(), offsets.data_ptr(),
          out.data_ptr(), E, K, N, M_cap, int(bm))
    return out


def expert_sort(experts, E: int, weights=None, out=None, stream=None):
    """A router's choices grouped by expert: (offsets, rows, pos) or, with weights, (..., row_weights).

    experts: int32 or int64 [T, k], the k experts of each token; a choice outside
    [0, E) (another rank's, or none) gets no row. weights: optional fp32 [T, k].
    offsets: int32 [E+1], expert e's rows are offsets[e]..offsets[e+1]-1, in the
    order of their choices; rows: int32 [T*k], each row's token; pos: int32 [T, k],
    each choice's row; row_weights: fp32 [T*k], each row's weight. Past offsets[E]
    rows holds -1 and row_weights 0; pos is -1 where a choice has no row. offsets
    is what the products take; rows is src_rows (and dst_rows) of
    grouped_gemm_gather and grouped_gemm_gather_combine, row_weights the weights of
    the latter; pos is what expert_spread and expert_combine take. out: optional
    tuple of the tensors that are returned. The order is the same on every call.
    """
    import torch
    what = "expert_sort"
    kind = experts.dtype
    if kind is not torch.int64:
        kind = torch.int32
    if weights is None:
        dev = _device_args(what, ("experts", experts, kind, 2))
    else:
        dev = _device_args(what, ("experts", experts, kind, 2), ("weights", weights, torch.float32, 2))
        _match(what, weights.shape == experts.shape, experts, weights)
    T, k = experts.shape
    E, n = int(E), T * k
    sizes = E | k | n
    if sizes >> 31:
        _int32(what, sizes)
    if E > MAX_EXPERTS:  # before memory is taken for so many offsets
        _check(3, what)
    i32 = torch.int32
    if out is None and stream is None:
        new = experts.new_empty
        out = (new((max(E, 0) + 1,), dtype=i32), new((n,), dtype=i32), new((T, k), dtype=i32))
        if weights is not None:
            out += (new((n,), dtype=torch.float32),)
    else:
        wanted = [((max(E, 0) + 1,), i32), ((n,), i32), ((T, k), i32)]
        if weights is not None:
            wanted.append(((n,), torch.float32))
        if out is None:
            out = (None,) * len(wanted)
        if len(out) != len(wanted):
            raise ValueError("%s: out must hold %d tensors" % (what, len(wanted)))
        out = tuple(_out(what, o, shape, (dt,), None, experts, stream) for o, (shape, dt) in zip(out, wanted))
    space = None
    if n > _SORT_RECOUNT:
        space = _out(what, None, (load_library().gg_expert_sort_workspace(n, E),), (torch.uint8,), None, experts,
                     stream)
    _call("gg_expert_sort", dev, stream, (experts, weights, *out, space), experts.data_ptr(),
          int(kind is torch.int64), None if weights is None else weights.data_ptr(), out[0].data_ptr(),
          out[1].data_ptr(), out[2].data_ptr(), None if weights is None else out[3].data_ptr(),
          None if space is None else space.data_ptr(), T, k, E)
    return out


def expert_spread(X, pos, scale=None, M_cap=None, out=None, out_scale=None, stream=None):
    """out[pos[t, j]] = X[t]: each token's row to the rows of its choices, in one launch.

    X: [T, K] of any type whose rows are a multiple of 16 bytes (bf16, fp32, fp8
    or 4-bit codes); pos: int32 [T, k] (expert_sort), entries outside [0, M_cap) are
    skipped; out: optional [M_cap, K] like X (default: M_cap = T*k rows, or M_cap
    where it is given). Rows that no choice names are left as they were; a row that
    two choices name (expert_sort makes none) is undefined, parts of both tokens'
    codes and scales. scale: the block scales of X, which go with their rows: fp32 [ceil(K/128), T]
    (fp8_quantize, rms_norm_fp8) or uint8 [ceil(K/256), T, 8] (mx4_quantize); then
    (out, out_scale) is returned, out_scale [.., M_cap(, 8)]. The gradient with
    respect to X is expert_combine(d_out, pos).
    """
    import torch
    what = "expert_spread"
    args = [("X", X, X.dtype, 2), ("pos", pos, torch.int32, 2)]
    sb = 0
    if scale is not None:
        sb = 8 if scale.dtype is torch.uint8 else 4
        args.append(("scale", scale, torch.uint8 if sb == 8 else torch.float32, 3 if sb == 8 else 2))
    dev = _device_args(what, *args)
    T, k = pos.shape
    K = X.shape[1]
    _match(what, X.shape[0] == T and (scale is None or scale.shape[1:] == ((T, 8) if sb == 8 else (T,))),
           X, pos, *([] if scale is None else [scale]))
    row_bytes = K * X.element_size()
    if scale is not None and scale.shape[0] != -(-row_bytes // _BLOCK):
        raise ValueError("%s: rows of %d bytes have %d slices of scales, not %d" % (
            what, row_bytes, -(-row_bytes // _BLOCK), scale.shape[0]))
    if M_cap is None:
        M_cap = T * k if out is None else out.shape[0]
    slices = 0 if scale is None else scale.shape[0]
    sizes = k | T * k | M_cap | slices
    if sizes >> 31:
        _int32(what, sizes)
    o = _out(what, out, (M_cap, K), (X.dtype,), None, X, stream)
    s = None
    if scale is not None:
        s = _out(what, out_scale, (slices, M_cap) + ((8,) if sb == 8 else ()), (scale.dtype,), None, X, stream)
    _call("gg_expert_spread", dev, stream, (X, pos, o, scale, s), X.data_ptr(), pos.data_ptr(), o.data_ptr(),
          None if s is None else scale.data_ptr(), None if s is None else s.data_ptr(), sb if slices else 0, T,
          k, row_bytes, slices, M_cap)
    return o if s is None else (o, s)


def expert_combine(Y, pos, weights=None, out=None, stream=None, out_dtype=None):
    """out[t] = sum_j weights[t, j] * Y[pos[t, j]]: the experts' rows back to their tokens, in one launch.

    Y: bf16 or fp32 [M_cap, N], the rows; pos: int32 [T, k] (expert_sort), entries
    outside [0, M_cap) are skipped; weights: optional fp32 [T, k] (default 1); out:
    optional bf16 or fp32 [T, N] (out_dtype when out is not given, default Y's). A
    token with no rows gets zeros. fp32 sums in the order of j, rounded once: equal
    inputs give equal bits. N is a multiple of 8.
    """
    import torch
    what = "expert_combine"
    kinds = (torch.bfloat16, torch.float32)
    args = [("Y", Y, Y.dtype if Y.dtype in kinds else kinds[0], 2), ("pos", pos, torch.int32, 2)]
    if weights is not None:
        args.append(("weights", weights, torch.float32, 2))
    dev = _device_args(what, *args)
    T, k = pos.shape
    M_cap, N = Y.shape
    _match(what, weights is None or weights.shape == (T, k), Y, pos, *([] if weights is None else [weights]))
    sizes = k | T * k | M_cap | N
    if sizes >> 31:
        _int32(what, sizes)
    if out is None and out_dtype is None:
        out_dtype = Y.dtype
    out = _out(what, out, (T, N), kinds, out_dtype, Y, stream)
    _call("gg_expert_combine", dev, stream, (Y, pos, weights, out), Y.data_ptr(), int(Y.dtype is kinds[1]),
          pos.data_ptr(), None if weights is None else weights.data_ptr(), out.data_ptr(),
          int(out.dtype is kinds[1]), T, k, N, M_cap)
    return out


def expert_combine_grad(dO, Y, pos, weights, out=None, out_weights=None, stream=None):
    """The gradient of expert_combine(Y, pos, weights): (dY, dweights), in one launch.

    dO: [T, N] and Y: [M_cap, N], both bf16 or both fp32; pos: int32 [T, k];
    weights: fp32 [T, k]. dY[pos[t, j]] = weights[t, j] * dO[t], like Y (``out``;
    rows that no choice names are left as they were, a row that two choices name is
    undefined, parts of both); dweights[t, j] = <dO[t],
    Y[pos[t, j]]>, fp32 [T, k] (``out_weights``), 0 where a choice has no row.
    Everything in fp32, dY rounded once, sums in a fixed order.
    """
    import torch
    what = "expert_combine_grad"
    kind = torch.float32 if Y.dtype is torch.float32 else torch.bfloat16
    dev = _device_args(what, ("dO", dO, kind, 2), ("Y", Y, kind, 2), ("pos", pos, torch.int32, 2),
                       ("weights", weights, torch.float32, 2))
    T, k = pos.shape
    M_cap, N = Y.shape
    _match(what, dO.shape == (T, N) and weights.shape == (T, k), dO, Y, pos, weights)
    sizes = k | T * k | M_cap | N
    if sizes >> 31:
        _int32(what, sizes)
    dY = _out(what, out, (M_cap, N), (kind,), None, Y, stream)
    dw = _out(what, out_weights, (T, k), (torch.float32,), None, Y, stream)
    _call("gg_expert_combine_grad", dev, stream, (dO, Y, pos, weights, dY, dw), dO.data_ptr(), Y.data_ptr(),
          int(kind is torch.float32), pos.data_ptr(), weights.data_ptr(), dY.data_ptr(), dw.data_ptr(), T, k,
          N, M_cap)
    return dY, dw


def rms_norm_fp8(X, weight, residual=None, eps: float = 1e-6, with_norm: bool = False, out=None,
                 out_scale=None, out_sum=None, out_norm=None, stream=None):
    """Root-mean-square norm of X + residual in 8 bits: (q, scales[, sum][, norm]), in one launch.

    X, residual: bf16 [T, K]; weight: bf16 [K]. With z = X + residual rounded to
    bf16 (X without a residual) and y = z / sqrt(mean z^2 + eps) * weight in fp32:
    q float8_e4m3fn [T, K] and scales fp32 [ceil(K/128), T] hold y by the rule of
    fp8_quantize; sum is z, bf16 [T, K], returned where a residual is given
    (out_sum may be X or residual itself); norm, with with_norm or out_norm, is y
    rounded once to bf16 (a router's input). K is a multiple of 16, at most 16384.
    What is not finite, and zeros with eps = 0, stands for NaN in its row.
    """
    import torch
    what = "rms_norm_fp8"
    bf = torch.bfloat16
    args = [("X", X, bf, 2), ("weight", weight, bf, 1)]
    if residual is not None:
        args.append(("residual", residual, bf, 2))
    dev = _device_args(what, *args)
    T, K = X.shape
    _match(what, weight.shape[0] == K and (residual is None or residual.shape == (T, K)), X, weight,
           *([] if residual is None else [residual]))
    if out_sum is not None and residual is None:
        raise ValueError("%s: out_sum needs a residual" % what)
    if K >> 31:
        _int32(what, K)
    q = _out(what, out, (T, K), (torch.float8_e4m3fn, torch.uint8), None, X, stream)
    s = _out(what, out_scale, (-(-K // _BLOCK), T), (torch.float32,), None, X, stream)
    z = None if residual is None else _out(what, out_sum, (T, K), (bf,), None, X, stream)
    y = _out(what, out_norm, (T, K), (bf,), None, X, stream) if with_norm or out_norm is not None else None
    _call("gg_rms_norm_fp8", dev, stream, (X, weight, residual, q, s, z, y), X.data_ptr(),
          None if residual is None else residual.data_ptr(), weight.data_ptr(), q.data_ptr(), s.data_ptr(),
          None if z is None else z.data_ptr(), None if y is None else y.data_ptr(), T, K, float(eps))
    return (q, s) + (() if z is None else (z,)) + (() if y is None else (y,))


def rms_norm_grad(dY, Z, weight, d_residual=None, eps: float = 1e-6, out=None, out_weight=None, stream=None):
    """The gradient of y = z / sqrt(mean z^2 + eps) * weight: (dZ, dweight).

    dY: bf16 [T, K], the gradient of y (of an y in 8 bits: of its values before
    they were rounded); Z: bf16 [T, K], the sum that was normalised; weight: bf16
    [K]; d_residual: optional bf16 [T, K], the gradient that reaches z past the
    norm, added. dZ: bf16 [T, K], rounded once: the gradient of X and of residual
    alike. dweight: fp32 [K], summed without atomics in an order that T and K fix.
    """
    import torch
    what = "rms_norm_grad"
    bf = torch.bfloat16
    args = [("dY", dY, bf, 2), ("Z", Z, bf, 2), ("weight", weight, bf, 1)]
    if d_residual is not None:
        args.append(("d_residual", d_residual, bf, 2))
    dev = _device_args(what, *args)
    T, K = Z.shape
    _match(what, dY.shape == (T, K) and weight.shape[0] == K
           and (d_residual is None or d_residual.shape == (T, K)), dY, Z, weight,
           *([] if d_residual is None else [d_residual]))
    if K >> 31:
        _int32(what, K)
    dZ = _out(what, out, (T, K), (bf,), None, Z, stream)
    dg = _out(what, out_weight, (K,), (torch.float32,), None, Z, stream)
    space = _out(what, None, (load_library().gg_rms_norm_grad_workspace(T, K),), (torch.uint8,), None, Z, stream)
    _call("gg_rms_norm_grad", dev, stream, (dY, Z, weight, d_residual, dZ, dg, space), dY.data_ptr(),
          Z.data_ptr(), weight.data_ptr(), None if d_residual is None else d_residual.data_ptr(),
          dZ.data_ptr(), dg.data_ptr(), space.data_ptr(), T, K, float(eps))
    return dZ, dg


def tile_schedule(offsets, N: int, M_cap: int, bm: int = 0, max_tiles: int = None, stream=None):
    """The device-built tile list: int32 tensor [n_tiles, 5] of (expert, row0, rows, col0, bm)."""
    import torch
    lib = load_library()
    if offsets.dtype != torch.int32 or not offsets.is_cuda or offsets.dim() != 1:
        raise TypeError("offsets must be a 1-D int32 device tensor")
    E = offsets.shape[0] - 1
    if max_tiles is None:
        hmin = bm if bm else BM_CHOICES[0]
        max_tiles = (M_cap // hmin + E) * (-(-N // TILE_N))
    _int32("tile_schedule", E | N | M_cap | int(bm) | int(max_tiles))
    tiles = _new((max(max_tiles, 1), 5), torch.int32, offsets, stream)
    n = _new((1,), torch.int32, offsets, stream, zero=True)
    st = lib.gg_tile_schedule(offsets.data_ptr(), E, N, M_cap, int(bm), tiles.data_ptr(), n.data_ptr(),
                              int(max_tiles), _stream_handle(offsets.device, stream))
    _check(st, "gg_tile_schedule")
    _keep(stream, offsets)
    with torch.cuda.stream(stream):  # (None: the current one)
        count = int(n.item())
    return tiles[:min(count, max_tiles)], count


def trace_library_path() -> str:
    return _TRACE_LIB_PATH


def load_trace_library():
    """Load the tracing build (raises if it has not been built)."""
    global _trace_lib
    if _trace_lib is None:
        if not os.path.exists(_TRACE_LIB_PATH):
            raise GroupedGemmError(
                "HIP library %s is not built; run `python -m moe_ragged_grouped_amd.build`"
                % _TRACE_LIB_PATH)
        lib = ctypes.CDLL(_TRACE_LIB_PATH)
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        lib.gg_trace_grouped_gemm_bf16.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, i32, vp,
                                                   i32, vp]
        lib.gg_trace_grouped_gemm_bf16.restype = ctypes.c_int
        lib.gg_trace_clock_khz.argtypes = [ctypes.POINTER(ctypes.c_int32)]
        lib.gg_trace_clock_khz.restype = ctypes.c_int
        lib.gg_status_string.argtypes = [ctypes.c_int]
        lib.gg_status_string.restype = ctypes.c_char_p
        _trace_lib = lib
    return _trace_lib


def traced_grouped_gemm(A, B, offsets, max_tiles: int, out=None, bm: int = 0, stream=None,
                        trace=None):
    """grouped_gemm (fp32 C) through the tracing build, with its timeline.

    Returns (C, trace, khz): trace is the uint64 record buffer of
    gg_trace_grouped_gemm_bf16 as an int64 device tensor
    [TRACE_WORKGROUPS + max_tiles, TRACE_RECORD], khz the rate of its
    counter. A trace tensor passed in is written as it is (records the launch
    does not write keep their values); otherwise a cleared one is allocated.
    """
    import torch
    lib = load_trace_library()
    E, K, N, M_cap = _grouped_args(A, B, offsets, bm)
    _int32("traced_grouped_gemm", int(max_tiles))
    if out is None:
        out = _new((M_cap, N), torch.float32, A, stream)
    elif out.dtype != torch.float32 or tuple(out.shape) != (M_cap, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 [M_cap, N] tensor")
    shape = (TRACE_WORKGROUPS + int(max_tiles), TRACE_RECORD)
    if trace is None:
        trace = _new(shape, torch.int64, A, stream, zero=True)
    elif (trace.dtype != torch.int64 or tuple(trace.shape) != shape or not trace.is_contiguous()
          or trace.device != A.device):
        raise ValueError("trace must be a contiguous int64 [%d, %d] tensor on A's device" % shape)
    st = lib.gg_trace_grouped_gemm_bf16(A.data_ptr(), B.data_ptr(), offsets.data_ptr(),
                                        out.data_ptr(), E, K, N, M_cap, int(bm), trace.data_ptr(),
                                        int(max_tiles), _stream_handle(A.device, stream))
    if st != 0:
        raise GroupedGemmError("gg_trace_grouped_gemm_bf16: status %d (%s)"
                               % (st, lib.gg_status_string(st).decode()))
    _keep(stream, A, B, offsets, out, trace)
    khz = ctypes.c_int32(0)
    st = lib.gg_trace_clock_khz(ctypes.byref(khz))
    if st != 0:
        raise GroupedGemmError("gg_trace_clock_khz: status %d" % st)
    return out, trace, int(khz.value)
