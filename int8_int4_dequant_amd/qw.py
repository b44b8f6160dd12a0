"""Thin Python binding of libqw (include/qw.h).

Argument marshalling only: every step of quantization, unpacking and the
products runs in the HIP kernels of libqw.so.  PyTorch provides device
memory and the current HIP stream.  If the library has not been built this
module raises; there is no CPU fallback.

Low-level functions carry the C names (``qw_quantize_pack``, ``qw_unpack``,
``qw_gemv``, ``qw_gemm``) and take preallocated tensors; the convenience
layer (``quantize_pack``, ``unpack``, ``gemv``, ``gemm``) allocates outputs
and returns a record shaped like the pages' ``pack`` result:
``{bits, group, shape, payload, scales}``.
"""

import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqw.so")

#: matrices per kernel launch in the batched calls (QW_BATCH_PER_LAUNCH in qw.h)
BATCH_PER_LAUNCH = 256

QW_OK = 0
STATUS_NAMES = {0: "QW_OK", -1: "QW_EBITS", -2: "QW_EGROUP", -3: "QW_ESHAPE", -4: "QW_EM",
                -5: "QW_ENULL", -6: "QW_EHIP", -7: "QW_ECOUNT", -8: "QW_EWORK", -9: "QW_EARG",
                -10: "QW_ESCRATCH"}

#: symbols declared in include/qw.h
EXPORTS = ["qw_payload_bytes", "qw_num_scales", "qw_status_string", "qw_last_error",
           "qw_quantize_pack", "qw_quantize_pack_batched", "qw_unpack", "qw_unpack_batched",
           "qw_gemv",
           "qw_gemv_batched", "qw_gemv_chain", "qw_gemm", "qw_matmul_work_bytes", "qw_matmul",
           "qw_matmul_noalloc",
           "qw_debug_path",
           "qw_gptq_hessian_work_bytes", "qw_gptq_hessian", "qw_gptq_factor_work_bytes",
           "qw_gptq_factor", "qw_gptq_quantize_work_bytes", "qw_gptq_quantize_pack",
           "qw_block_pitch", "qw_block_num_scales", "qw_block_quantize",
           "qw_block_quantize_swiglu", "qw_block_unpack", "qw_block_gemm",
           "qw_block_matmul_work_bytes", "qw_block_matmul", "qw_block_gemm_grouped",
           "qw_moe_sort_work_bytes", "qw_moe_sort", "qw_moe_gather", "qw_moe_gather_block",
           "qw_moe_combine", "qw_moe_combine_backward", "qw_moe_mlp_work_bytes", "qw_moe_mlp",
           "qw_block_debug_path"]

#: symbols declared in include/qw_mx.h
EXPORTS_MX = ["qw_mx_pitch", "qw_mx_quantize", "qw_mx_unpack", "qw_mx_gemm",
              "qw_mx_matmul_work_bytes", "qw_mx_matmul", "qw_rms_norm", "qw_rms_norm_block",
              "qw_rms_norm_mx", "qw_rms_norm_backward_work_bytes", "qw_rms_norm_backward",
              "qw_mx_gated", "qw_mx_gated_codes", "qw_mx_gated_backward",
              "qw_mx_mlp_work_bytes", "qw_mx_mlp", "qw_mx_debug_path"]


# Rows up to which qw_matmul runs the codes GEMV (QW_MATMUL_GEMV_MAX_M in qw.h).
MATMUL_GEMV_MAX_M = 4
# Bytes of the static scratch of qw_matmul_noalloc (QW_MATMUL_NOALLOC_MAX_BYTES).
MATMUL_NOALLOC_MAX_BYTES = 32 << 20

# Values per scale along a row of block-scaled e4m3 codes (QW_BLOCK).
BLOCK = 128
# Values per scale of microscaled 4-bit codes (QW_MX_BLOCK).
MX_BLOCK = 32
# QW_F32 and QW_BF16 (enum qw_type), by tensor type.
TYPES = {torch.float32: 0, torch.bfloat16: 1}
# Most experts and slots of the expert calls (QW_MOE_MAX_EXPERTS, QW_MOE_MAX_SLOTS).
MOE_MAX_EXPERTS = 512
MOE_MAX_SLOTS = 1 << 30


class QwQuantDesc(ctypes.Structure):
    """Mirror of `qw_quant_desc` in include/qw.h."""
    _fields_ = [("w", ctypes.c_void_p), ("payload", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QwUnpackDesc(ctypes.Structure):
    """Mirror of `qw_unpack_desc` in include/qw.h."""
    _fields_ = [("payload", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("w_out", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QwGemvDesc(ctypes.Structure):
    """Mirror of `qw_gemv_desc` in include/qw.h."""
    _fields_ = [("payload", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]

_lib = None


class QwError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        msg = f"{what}: {STATUS_NAMES.get(status, status)} ({_text(status)})"
        if status == -6:
            msg += f": {_lib.qw_last_error().decode()}"
        super().__init__(msg)


def _text(status):
    return _lib.qw_status_string(status).decode() if _lib else str(status)


def lib():
    """Load libqw.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    L = ctypes.CDLL(LIB_PATH)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    L.qw_payload_bytes.argtypes = [i32, i64, i64]
    L.qw_payload_bytes.restype = i64
    L.qw_num_scales.argtypes = [i64, i64, i64]
    L.qw_num_scales.restype = i64
    L.qw_status_string.argtypes = [i32]
    L.qw_status_string.restype = ctypes.c_char_p
    L.qw_last_error.argtypes = []
    L.qw_last_error.restype = ctypes.c_char_p
    L.qw_quantize_pack.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp]
    L.qw_quantize_pack.restype = i32
    L.qw_quantize_pack_batched.argtypes = [i32, ctypes.POINTER(QwQuantDesc), vp]
    L.qw_quantize_pack_batched.restype = i32
    L.qw_unpack.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp]
    L.qw_unpack.restype = i32
    L.qw_unpack_batched.argtypes = [i32, ctypes.POINTER(QwUnpackDesc), vp]
    L.qw_unpack_batched.restype = i32
    L.qw_gemv.argtypes = [i32, i64, i64, i64, vp, vp, i64, vp, vp, vp]
    L.qw_gemv.restype = i32
    L.qw_gemv_batched.argtypes = [i32, ctypes.POINTER(QwGemvDesc), i64, vp]
    L.qw_gemv_batched.restype = i32
    L.qw_gemv_chain.argtypes = [i32, ctypes.POINTER(QwGemvDesc), ctypes.POINTER(ctypes.c_int32),
                                i64, vp]
    L.qw_gemv_chain.restype = i32
    L.qw_gemm.argtypes = [i32, i64, i64, i64, vp, vp, i64, vp, vp, vp]
    L.qw_gemm.restype = i32
    L.qw_matmul_work_bytes.argtypes = [i64, i64]
    L.qw_matmul_work_bytes.restype = i64
    L.qw_matmul.argtypes = [i32, i64, i64, i64, vp, vp, i64, vp, vp, vp, i64, vp]
    L.qw_matmul.restype = i32
    L.qw_matmul_noalloc.argtypes = [i32, i64, i64, i64, vp, vp, i64, vp, vp, vp]
    L.qw_matmul_noalloc.restype = i32
    L.qw_debug_path.argtypes = [i32, i32, i64, i64, i64, vp, vp]
    L.qw_debug_path.restype = i32
    L.qw_gptq_hessian_work_bytes.argtypes = [i64, i64]
    L.qw_gptq_hessian_work_bytes.restype = i64
    L.qw_gptq_hessian.argtypes = [i64, i64, vp, vp, vp, i64, vp]
    L.qw_gptq_hessian.restype = i32
    L.qw_gptq_factor_work_bytes.argtypes = [i64]
    L.qw_gptq_factor_work_bytes.restype = i64
    L.qw_gptq_factor.argtypes = [i64, vp, ctypes.c_double, vp, vp, vp, i64, vp]
    L.qw_gptq_factor.restype = i32
    L.qw_gptq_quantize_work_bytes.argtypes = [i64, i64]
    L.qw_gptq_quantize_work_bytes.restype = i64
    L.qw_gptq_quantize_pack.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, i64, vp]
    L.qw_gptq_quantize_pack.restype = i32
    L.qw_block_pitch.argtypes = [i64]
    L.qw_block_pitch.restype = i64
    L.qw_block_num_scales.argtypes = [i32, i64, i64]
    L.qw_block_num_scales.restype = i64
    L.qw_block_quantize.argtypes = [i32, i64, i64, i64, i32, vp, vp, vp, vp]
    L.qw_block_quantize.restype = i32
    L.qw_block_quantize_swiglu.argtypes = [i64, i64, i32, vp, vp, vp, vp, vp]
    L.qw_block_quantize_swiglu.restype = i32
    L.qw_block_unpack.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp]
    L.qw_block_unpack.restype = i32
    L.qw_block_gemm.argtypes = [i32, i64, i64, vp, vp, i64, vp, vp, i32, vp, vp]
    L.qw_block_gemm.restype = i32
    L.qw_block_matmul_work_bytes.argtypes = [i64, i64]
    L.qw_block_matmul_work_bytes.restype = i64
    L.qw_block_matmul.argtypes = [i32, i64, i64, vp, vp, i64, i32, vp, i32, vp, vp, i64, vp]
    L.qw_block_matmul.restype = i32
    L.qw_block_gemm_grouped.argtypes = [i32, i64, i64, i64, vp, vp, i64, vp, vp, vp, i32, vp, vp]
    L.qw_block_gemm_grouped.restype = i32
    L.qw_moe_sort_work_bytes.argtypes = [i64, i64, i64]
    L.qw_moe_sort_work_bytes.restype = i64
    L.qw_moe_sort.argtypes = [i64, i64, i64, i32, vp, vp, vp, vp, vp, i64, vp]
    L.qw_moe_sort.restype = i32
    L.qw_moe_gather.argtypes = [i64, i64, i64, i64, i32, vp, vp, vp, vp]
    L.qw_moe_gather.restype = i32
    L.qw_moe_gather_block.argtypes = [i64, i64, i64, i64, i32, vp, vp, vp, vp, vp]
    L.qw_moe_gather_block.restype = i32
    L.qw_moe_combine.argtypes = [i64, i64, i64, i64, i32, vp, vp, vp, i32, vp, vp]
    L.qw_moe_combine.restype = i32
    L.qw_moe_combine_backward.argtypes = [i64, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp]
    L.qw_moe_combine_backward.restype = i32
    L.qw_moe_mlp_work_bytes.argtypes = [i64, i64, i64, i64, i64]
    L.qw_moe_mlp_work_bytes.restype = i64
    L.qw_moe_mlp.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, i64, i64, i32, vp, i32, vp, vp,
                             i32, vp, vp, i64, vp]
    L.qw_moe_mlp.restype = i32
    L.qw_block_debug_path.argtypes = [i32, i64, i64, i64, i64, i32]
    L.qw_block_debug_path.restype = i32
    f32 = ctypes.c_float
    L.qw_mx_pitch.argtypes = [i64]
    L.qw_mx_pitch.restype = i64
    L.qw_mx_quantize.argtypes = [i32, i64, i64, i32, vp, vp, vp, vp]
    L.qw_mx_quantize.restype = i32
    L.qw_mx_unpack.argtypes = [i64, i64, vp, vp, vp, vp]
    L.qw_mx_unpack.restype = i32
    L.qw_mx_gemm.argtypes = [i64, i64, vp, vp, i64, vp, vp, i32, vp, vp]
    L.qw_mx_gemm.restype = i32
    L.qw_mx_matmul_work_bytes.argtypes = [i64, i64]
    L.qw_mx_matmul_work_bytes.restype = i64
    L.qw_mx_matmul.argtypes = [i64, i64, vp, vp, i64, i32, vp, i32, vp, vp, i64, vp]
    L.qw_mx_matmul.restype = i32
    L.qw_rms_norm.argtypes = [i64, i64, i32, vp, vp, vp, i32, vp, f32, i32, vp, vp]
    L.qw_rms_norm.restype = i32
    L.qw_rms_norm_block.argtypes = [i64, i64, i32, vp, vp, vp, i32, vp, f32, vp, vp, vp]
    L.qw_rms_norm_block.restype = i32
    L.qw_rms_norm_mx.argtypes = [i64, i64, i32, vp, vp, vp, i32, vp, f32, vp, vp, vp]
    L.qw_rms_norm_mx.restype = i32
    L.qw_rms_norm_backward_work_bytes.argtypes = [i64, i64]
    L.qw_rms_norm_backward_work_bytes.restype = i64
    L.qw_rms_norm_backward.argtypes = [i64, i64, i32, vp, vp, i32, vp, f32, vp, vp, vp, vp, i64, vp]
    L.qw_rms_norm_backward.restype = i32
    L.qw_mx_gated.argtypes = [i64, i64, vp, vp, i64, vp, vp, i32, vp, vp]
    L.qw_mx_gated.restype = i32
    L.qw_mx_gated_codes.argtypes = [i64, i64, vp, vp, i64, vp, vp, vp, vp, vp]
    L.qw_mx_gated_codes.restype = i32
    L.qw_mx_gated_backward.argtypes = [i64, i64, vp, vp, i64, vp, vp, i32, vp, vp, vp, vp]
    L.qw_mx_gated_backward.restype = i32
    L.qw_mx_mlp_work_bytes.argtypes = [i64, i64, i64]
    L.qw_mx_mlp_work_bytes.restype = i64
    L.qw_mx_mlp.argtypes = [i64, i64, vp, vp, vp, vp, i64, i32, vp, i32, vp, vp, i64, vp]
    L.qw_mx_mlp.restype = i32
    L.qw_mx_debug_path.argtypes = [i32, i64, i64, i64]
    L.qw_mx_debug_path.restype = i32
    _lib = L
    return L


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return t  # raw integer address
    if t.numel() and not t.is_cuda:
        raise ValueError("libqw takes device tensors")
    return t.data_ptr() if t.numel() else None


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _check(status, what):
    if status != QW_OK:
        raise QwError(status, what)


# ------------------------------------------------------------ C-name layer


def qw_payload_bytes(bits, n, k):
    return lib().qw_payload_bytes(bits, n, k)


def qw_num_scales(group, n, k):
    return lib().qw_num_scales(group, n, k)


def qw_quantize_pack(bits, group, n, k, w, payload, scales, stream=None):
    return lib().qw_quantize_pack(bits, group, n, k, _ptr(w), _ptr(payload), _ptr(scales),
                                  _stream(stream))


def make_quant_descs(items):
    """items: iterable of (bits, group, n, k, w, payload, scales); returns a
    ctypes array for qw_quantize_pack_batched and its length."""
    items = list(items)
    arr = (QwQuantDesc * max(1, len(items)))()
    for i, (bits, group, n, k, w, payload, scales) in enumerate(items):
        arr[i] = QwQuantDesc(_ptr(w), _ptr(payload), _ptr(scales), n, k, group, bits, 0)
    return arr, len(items)


def qw_quantize_pack_batched(count, descs, stream=None):
    return lib().qw_quantize_pack_batched(count, descs, _stream(stream))


def qw_unpack(bits, group, n, k, payload, scales, w_out, stream=None):
    return lib().qw_unpack(bits, group, n, k, _ptr(payload), _ptr(scales), _ptr(w_out),
                           _stream(stream))


def make_unpack_descs(items):
    """items: iterable of (bits, group, n, k, payload, scales, w_out); returns
    a ctypes array for qw_unpack_batched and its length."""
    items = list(items)
    arr = (QwUnpackDesc * max(1, len(items)))()
    for i, (bits, group, n, k, payload, scales, w_out) in enumerate(items):
        arr[i] = QwUnpackDesc(_ptr(payload), _ptr(scales), _ptr(w_out), n, k, group, bits, 0)
    return arr, len(items)


def qw_unpack_batched(count, descs, stream=None):
    return lib().qw_unpack_batched(count, descs, _stream(stream))


def qw_gemv(bits, group, n, k, payload, scales, m, x, y, stream=None):
    return lib().qw_gemv(bits, group, n, k, _ptr(payload), _ptr(scales), m, _ptr(x), _ptr(y),
                         _stream(stream))


def make_gemv_descs(items):
    """items: iterable of (bits, group, n, k, payload, scales, x, y) with
    device tensors (or raw addresses); returns a ctypes array for
    qw_gemv_batched."""
    items = list(items)
    arr = (QwGemvDesc * max(1, len(items)))()
    for i, (bits, group, n, k, payload, scales, x, y) in enumerate(items):
        arr[i] = QwGemvDesc(_ptr(payload), _ptr(scales), _ptr(x), _ptr(y), n, k, group, bits, 0)
    return arr, len(items)


def qw_gemv_batched(count, descs, m, stream=None):
    return lib().qw_gemv_batched(count, descs, m, _stream(stream))


def qw_gemv_chain(count, descs, stages, m, stream=None):
    """``stages``: a ctypes int32 array (or a list) of ``count`` stage numbers."""
    if not isinstance(stages, ctypes.Array):
        stages = (ctypes.c_int32 * max(1, len(stages)))(*stages)
    return lib().qw_gemv_chain(count, descs, stages, m, _stream(stream))


def qw_gemm(bits, group, n, k, payload, scales, m, x_bf16, y, stream=None):
    return lib().qw_gemm(bits, group, n, k, _ptr(payload), _ptr(scales), m, _ptr(x_bf16),
                         _ptr(y), _stream(stream))


def qw_matmul_work_bytes(m, k):
    return lib().qw_matmul_work_bytes(m, k)


def qw_matmul(bits, group, n, k, payload, scales, m, x, y, work, work_bytes, stream=None):
    return lib().qw_matmul(bits, group, n, k, _ptr(payload), _ptr(scales), m, _ptr(x), _ptr(y),
                           _ptr(work), work_bytes, _stream(stream))


def qw_matmul_noalloc(bits, group, n, k, payload, scales, m, x, y, stream=None):
    return lib().qw_matmul_noalloc(bits, group, n, k, _ptr(payload), _ptr(scales), m, _ptr(x),
                                   _ptr(y), _stream(stream))


def qw_debug_path(op, bits, group, n, k, a=None, b=None):
    return lib().qw_debug_path(op, bits, group, n, k, _ptr(a), _ptr(b))


def qw_gptq_hessian_work_bytes(k, t):
    return lib().qw_gptq_hessian_work_bytes(k, t)


def qw_gptq_hessian(k, t, x, h, work, work_bytes, stream=None):
    return lib().qw_gptq_hessian(k, t, _ptr(x), _ptr(h), _ptr(work), work_bytes,
                                 _stream(stream))


def qw_gptq_factor_work_bytes(k):
    return lib().qw_gptq_factor_work_bytes(k)


def qw_gptq_factor(k, h, damp, u, info, work, work_bytes, stream=None):
    return lib().qw_gptq_factor(k, _ptr(h), damp, _ptr(u), _ptr(info), _ptr(work), work_bytes,
                                _stream(stream))


def qw_gptq_quantize_work_bytes(n, k):
    return lib().qw_gptq_quantize_work_bytes(n, k)


def qw_gptq_quantize_pack(bits, group, n, k, w, u, payload, scales, work, work_bytes,
                          stream=None):
    return lib().qw_gptq_quantize_pack(bits, group, n, k, _ptr(w), _ptr(u), _ptr(payload),
                                       _ptr(scales), _ptr(work), work_bytes, _stream(stream))


def qw_block_pitch(k):
    return lib().qw_block_pitch(k)


def qw_block_num_scales(block_rows, n, k):
    return lib().qw_block_num_scales(block_rows, n, k)


def qw_block_quantize(block_rows, count, n, k, type, w, codes, scales, stream=None):
    return lib().qw_block_quantize(block_rows, count, n, k, type, _ptr(w), _ptr(codes),
                                   _ptr(scales), _stream(stream))


def qw_block_quantize_swiglu(rows, f, type, h, used, codes, scales, stream=None):
    return lib().qw_block_quantize_swiglu(rows, f, type, _ptr(h), _ptr(used), _ptr(codes),
                                          _ptr(scales), _stream(stream))


def qw_block_unpack(block_rows, count, n, k, codes, scales, out, stream=None):
    return lib().qw_block_unpack(block_rows, count, n, k, _ptr(codes), _ptr(scales), _ptr(out),
                                 _stream(stream))


def qw_block_gemm(block_rows, n, k, codes, scales, m, x_codes, x_scales, y_type, y, stream=None):
    return lib().qw_block_gemm(block_rows, n, k, _ptr(codes), _ptr(scales), m, _ptr(x_codes),
                               _ptr(x_scales), y_type, _ptr(y), _stream(stream))


def qw_block_matmul_work_bytes(m, k):
    return lib().qw_block_matmul_work_bytes(m, k)


def qw_block_matmul(block_rows, n, k, codes, scales, m, x_type, x, y_type, y, work, work_bytes,
                    stream=None):
    return lib().qw_block_matmul(block_rows, n, k, _ptr(codes), _ptr(scales), m, x_type, _ptr(x),
                                 y_type, _ptr(y), _ptr(work), work_bytes, _stream(stream))


def qw_block_gemm_grouped(block_rows, experts, n, k, codes, scales, rows, x_codes, x_scales,
                          offsets, y_type, y, stream=None):
    return lib().qw_block_gemm_grouped(block_rows, experts, n, k, _ptr(codes), _ptr(scales), rows,
                                       _ptr(x_codes), _ptr(x_scales), _ptr(offsets), y_type,
                                       _ptr(y), _stream(stream))


def qw_moe_sort_work_bytes(t, topk, experts):
    return lib().qw_moe_sort_work_bytes(t, topk, experts)


def qw_moe_sort(t, topk, experts, id_bytes, ids, pos, order, offsets, work, work_bytes,
                stream=None):
    return lib().qw_moe_sort(t, topk, experts, id_bytes, _ptr(ids), _ptr(pos), _ptr(order),
                             _ptr(offsets), _ptr(work), work_bytes, _stream(stream))


def qw_moe_gather(t, topk, d, rows, type, x, pos, xs, stream=None):
    return lib().qw_moe_gather(t, topk, d, rows, type, _ptr(x), _ptr(pos), _ptr(xs),
                               _stream(stream))


def qw_moe_gather_block(t, topk, d, rows, type, x, pos, codes, scales, stream=None):
    return lib().qw_moe_gather_block(t, topk, d, rows, type, _ptr(x), _ptr(pos), _ptr(codes),
                                     _ptr(scales), _stream(stream))


def qw_moe_combine(t, topk, d, rows, type, ys, pos, weights, y_type, y, stream=None):
    return lib().qw_moe_combine(t, topk, d, rows, type, _ptr(ys), _ptr(pos), _ptr(weights),
                                y_type, _ptr(y), _stream(stream))


def qw_moe_combine_backward(t, topk, d, rows, type, dy, ys, pos, weights, dys, dweights,
                            stream=None):
    return lib().qw_moe_combine_backward(t, topk, d, rows, type, _ptr(dy), _ptr(ys), _ptr(pos),
                                         _ptr(weights), _ptr(dys), _ptr(dweights),
                                         _stream(stream))


def qw_moe_mlp_work_bytes(t, topk, experts, d, f):
    return lib().qw_moe_mlp_work_bytes(t, topk, experts, d, f)


def qw_moe_mlp(block_rows, experts, d, f, gate_up, gate_up_scales, down, down_scales, t, topk,
               x_type, x, id_bytes, ids, weights, y_type, y, work, work_bytes, stream=None):
    return lib().qw_moe_mlp(block_rows, experts, d, f, _ptr(gate_up), _ptr(gate_up_scales),
                            _ptr(down), _ptr(down_scales), t, topk, x_type, _ptr(x), id_bytes,
                            _ptr(ids), _ptr(weights), y_type, _ptr(y), _ptr(work), work_bytes,
                            _stream(stream))


def qw_block_debug_path(op, experts, m, n, k, y_type):
    return lib().qw_block_debug_path(op, experts, m, n, k, y_type)


def qw_mx_pitch(k):
    return lib().qw_mx_pitch(k)


def qw_mx_quantize(transpose, n, k, type, w, codes, scales, stream=None):
    return lib().qw_mx_quantize(transpose, n, k, type, _ptr(w), _ptr(codes), _ptr(scales),
                                _stream(stream))


def qw_mx_unpack(n, k, codes, scales, out, stream=None):
    return lib().qw_mx_unpack(n, k, _ptr(codes), _ptr(scales), _ptr(out), _stream(stream))


def qw_mx_gemm(n, k, codes, scales, m, x_codes, x_scales, y_type, y, stream=None):
    return lib().qw_mx_gemm(n, k, _ptr(codes), _ptr(scales), m, _ptr(x_codes), _ptr(x_scales),
                            y_type, _ptr(y), _stream(stream))


def qw_mx_matmul_work_bytes(m, k):
    return lib().qw_mx_matmul_work_bytes(m, k)


def qw_mx_matmul(n, k, codes, scales, m, x_type, x, y_type, y, work, work_bytes, stream=None):
    return lib().qw_mx_matmul(n, k, _ptr(codes), _ptr(scales), m, x_type, _ptr(x), y_type,
                              _ptr(y), _ptr(work), work_bytes, _stream(stream))


def qw_rms_norm(rows, d, type, x, residual, sum, weight_type, weight, eps, y_type, y,
                stream=None):
    return lib().qw_rms_norm(rows, d, type, _ptr(x), _ptr(residual), _ptr(sum), weight_type,
                             _ptr(weight), eps, y_type, _ptr(y), _stream(stream))


def qw_rms_norm_block(rows, d, type, x, residual, sum, weight_type, weight, eps, codes, scales,
                      stream=None):
    return lib().qw_rms_norm_block(rows, d, type, _ptr(x), _ptr(residual), _ptr(sum), weight_type,
                                   _ptr(weight), eps, _ptr(codes), _ptr(scales), _stream(stream))


def qw_rms_norm_mx(rows, d, type, x, residual, sum, weight_type, weight, eps, codes, scales,
                   stream=None):
    return lib().qw_rms_norm_mx(rows, d, type, _ptr(x), _ptr(residual), _ptr(sum), weight_type,
                                _ptr(weight), eps, _ptr(codes), _ptr(scales), _stream(stream))


def qw_rms_norm_backward_work_bytes(rows, d):
    return lib().qw_rms_norm_backward_work_bytes(rows, d)


def qw_rms_norm_backward(rows, d, type, dy, s, weight_type, weight, eps, dsum, ds, dweight, work,
                         work_bytes, stream=None):
    return lib().qw_rms_norm_backward(rows, d, type, _ptr(dy), _ptr(s), weight_type, _ptr(weight),
                                      eps, _ptr(dsum), _ptr(ds), _ptr(dweight), _ptr(work),
                                      work_bytes, _stream(stream))


def qw_mx_gated(f, k, codes, scales, m, x_codes, x_scales, h_type, h, stream=None):
    return lib().qw_mx_gated(f, k, _ptr(codes), _ptr(scales), m, _ptr(x_codes), _ptr(x_scales),
                             h_type, _ptr(h), _stream(stream))


def qw_mx_gated_codes(f, k, codes, scales, m, x_codes, x_scales, h_codes, h_scales, stream=None):
    return lib().qw_mx_gated_codes(f, k, _ptr(codes), _ptr(scales), m, _ptr(x_codes),
                                   _ptr(x_scales), _ptr(h_codes), _ptr(h_scales), _stream(stream))


def qw_mx_gated_backward(f, k, codes, scales, m, x_codes, x_scales, type, dh, dgate_up, h,
                         stream=None):
    return lib().qw_mx_gated_backward(f, k, _ptr(codes), _ptr(scales), m, _ptr(x_codes),
                                      _ptr(x_scales), type, _ptr(dh), _ptr(dgate_up), _ptr(h),
                                      _stream(stream))


def qw_mx_mlp_work_bytes(m, d, f):
    return lib().qw_mx_mlp_work_bytes(m, d, f)


def qw_mx_mlp(d, f, gate_up, gate_up_scales, down, down_scales, m, x_type, x, y_type, y, work,
              work_bytes, stream=None):
    return lib().qw_mx_mlp(d, f, _ptr(gate_up), _ptr(gate_up_scales), _ptr(down),
                           _ptr(down_scales), m, x_type, _ptr(x), y_type, _ptr(y), _ptr(work),
                           work_bytes, _stream(stream))


def qw_mx_debug_path(op, m, n, k):
    return lib().qw_mx_debug_path(op, m, n, k)


# -------------------------------------------------------- convenience layer


def _nk(shape):
    if len(shape) != 2:
        raise ValueError("weights are 2-D [n][k]")
    return int(shape[0]), int(shape[1])


def _check_tensor(t, dtype, numel, what, shape=None):
    """A tensor the kernels read or write: of `dtype`, contiguous, holding
    exactly `numel` elements (of `shape` when given).  The C ABI takes bare
    pointers and cannot see sizes, so a buffer that is too small would be read
    or written past its end on the device.  (``_on_device`` checks where the
    tensors live once all sizes have been checked.)"""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what} must be a torch tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if t.numel() != numel:
        raise ValueError(f"{what} holds {t.numel()} elements, expected {numel}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _on_device(*ts):
    """Every non-empty tensor the call passes must be a device tensor."""
    for t in ts:
        if isinstance(t, dict):
            _on_device(t["payload"], t["scales"])
        elif isinstance(t, torch.Tensor) and t.numel() and not t.is_cuda:
            raise ValueError("libqw takes device tensors; a host tensor was passed")


def _check_rec(rec, what="record"):
    """(n, k) of a record whose payload and scales match its bits, group and
    shape (qw_payload_bytes / qw_num_scales)."""
    n, k = _nk(rec["shape"])
    bits, group = int(rec["bits"]), int(rec["group"])
    nb = lib().qw_payload_bytes(bits, n, k)
    ns = lib().qw_num_scales(group, n, k)
    if nb < 0 or ns < 0:
        raise ValueError(f"{what}: invalid bits {bits}, group {group} or shape {[n, k]}")
    _check_tensor(rec["payload"], torch.uint8, nb, f"{what} payload")
    _check_tensor(rec["scales"], torch.float32, ns, f"{what} scales")
    return n, k


def quantize_pack(w, bits, group, stream=None):
    """Quantize a contiguous fp32 device tensor [n][k]; returns a record
    ``{bits, group, shape, payload (uint8), scales (float32)}``."""
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise ValueError("w must be a contiguous float32 tensor")
    n, k = _nk(w.shape)
    nb = lib().qw_payload_bytes(bits, n, k)
    ns = lib().qw_num_scales(group, n, k)
    if nb < 0 or ns < 0:
        _check(QW_EBITS if bits not in (4, 8) else -2 if ns < 0 else -3, "quantize_pack")
    payload = torch.empty(nb, dtype=torch.uint8, device=w.device)
    scales = torch.empty(ns, dtype=torch.float32, device=w.device)
    _check(qw_quantize_pack(bits, group, n, k, w, payload, scales, stream), "qw_quantize_pack")
    return dict(bits=bits, group=group, shape=[n, k], payload=payload, scales=scales)


def quantize_pack_batched(ws, bits, group, stream=None):
    """Quantize a list of contiguous fp32 [n][k] device tensors (same bits
    and group) in a few launches; returns their records."""
    recs = []
    for w in ws:
        if w.dtype != torch.float32 or not w.is_contiguous():
            raise ValueError("each w must be a contiguous float32 tensor")
        n, k = _nk(w.shape)
        nb, ns = lib().qw_payload_bytes(bits, n, k), lib().qw_num_scales(group, n, k)
        if nb < 0 or ns < 0:
            _check(-1 if bits not in (4, 8) else -2 if ns < 0 else -3, "quantize_pack_batched")
        recs.append(dict(bits=bits, group=group, shape=[n, k],
                         payload=torch.empty(nb, dtype=torch.uint8, device=w.device),
                         scales=torch.empty(ns, dtype=torch.float32, device=w.device)))
    arr, cnt = make_quant_descs((bits, group, r["shape"][0], r["shape"][1], w, r["payload"],
                                 r["scales"]) for w, r in zip(ws, recs))
    _check(qw_quantize_pack_batched(cnt, arr, stream), "qw_quantize_pack_batched")
    return recs


def unpack_batched(recs, outs=None, stream=None):
    """Unpack a list of records in a few launches; returns fp32 tensors of
    their shapes (or fills ``outs``)."""
    if outs is None:
        outs = [torch.empty(tuple(int(d) for d in r["shape"]), dtype=torch.float32,
                            device=r["payload"].device) for r in recs]
    if len(outs) != len(recs):
        raise ValueError("one output per record")
    items = []
    for r, o in zip(recs, outs):
        n, k = _check_rec(r)
        _check_tensor(o, torch.float32, n * k, "output")
        items.append((r["bits"], r["group"], n, k, r["payload"], r["scales"], o))
    _on_device(*recs, *outs)
    arr, cnt = make_unpack_descs(items)
    _check(qw_unpack_batched(cnt, arr, stream), "qw_unpack_batched")
    return outs


def unpack(rec, out=None, stream=None):
    n, k = _check_rec(rec)
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=rec["payload"].device)
    _check_tensor(out, torch.float32, n * k, "out")
    _on_device(rec, out)
    _check(qw_unpack(rec["bits"], rec["group"], n, k, rec["payload"], rec["scales"], out,
                     stream), "qw_unpack")
    return out


def gemv(rec, x, out=None, stream=None):
    """fp32 x [m][k] (m <= 8) times the quantized weight; returns y [m][n]."""
    n, k = _check_rec(rec)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be a contiguous float32 [m][k] tensor")
    m = x.shape[0]
    _check_tensor(x, torch.float32, m * k, "x")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check_tensor(out, torch.float32, m * n, "out", (m, n))
    _on_device(rec, x, out)
    _check(qw_gemv(rec["bits"], rec["group"], n, k, rec["payload"], rec["scales"], m, x, out,
                   stream), "qw_gemv")
    return out


def gemv_batched(recs, xs, outs=None, stream=None):
    """Independent GEMVs (common m) in a few launches; returns the list of y."""
    if len(xs) != len(recs) or (outs is not None and len(outs) != len(recs)):
        raise ValueError("one x (and one output) per record")
    m = xs[0].shape[0]
    if outs is None:
        outs = [torch.empty((m, r["shape"][0]), dtype=torch.float32, device=x.device)
                for r, x in zip(recs, xs)]
    for r, x, y in zip(recs, xs, outs):
        n, k = _check_rec(r)
        _check_tensor(x, torch.float32, m * k, "x", (m, k))
        _check_tensor(y, torch.float32, m * n, "output", (m, n))
    _on_device(*recs, *xs, *outs)
    arr, cnt = make_gemv_descs((r["bits"], r["group"], r["shape"][0], r["shape"][1], r["payload"],
                                r["scales"], x, y) for r, x, y in zip(recs, xs, outs))
    _check(qw_gemv_batched(cnt, arr, m, stream), "qw_gemv_batched")
    return outs


def gemv_chain(recs, xs, ys, stages, stream=None):
    """A chained decode pass: product i computes ys[i] = xs[i] . W_i^T in
    stage stages[i]; an x may be the y of an earlier stage.  All tensors are
    preallocated, contiguous fp32 [m][k] / [m][n] with a common m."""
    if not len(recs) == len(xs) == len(ys) == len(stages):
        raise ValueError("one x, y and stage per record")
    m = xs[0].shape[0]
    for r, x, y in zip(recs, xs, ys):
        n, k = _check_rec(r)
        _check_tensor(x, torch.float32, m * k, "x", (m, k))
        _check_tensor(y, torch.float32, m * n, "y", (m, n))
    _on_device(*recs, *xs, *ys)
    arr, cnt = make_gemv_descs((r["bits"], r["group"], r["shape"][0], r["shape"][1], r["payload"],
                                r["scales"], x, y) for r, x, y in zip(recs, xs, ys))
    _check(qw_gemv_chain(cnt, arr, list(stages), m, stream), "qw_gemv_chain")
    return ys


def gemm(rec, x_bf16, out=None, stream=None):
    """bf16 x [m][k] (torch.bfloat16, or int16/uint16 bit patterns) times the
    quantized weight on the matrix cores; returns fp32 y [m][n]."""
    n, k = _check_rec(rec)
    if not isinstance(x_bf16, torch.Tensor) or x_bf16.dim() != 2 or x_bf16.shape[1] != k:
        raise ValueError("x must be a contiguous [m][k] tensor")
    m = x_bf16.shape[0]
    _check_tensor(x_bf16, (torch.bfloat16, torch.int16, torch.uint16), m * k, "x (bf16)")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x_bf16.device)
    _check_tensor(out, torch.float32, m * n, "out", (m, n))
    _on_device(rec, x_bf16, out)
    _check(qw_gemm(rec["bits"], rec["group"], n, k, rec["payload"], rec["scales"], m, x_bf16,
                   out, stream), "qw_gemm")
    return out


def matmul(rec, x, out=None, work=None, stream=None):
    """QuantizedMatmul: fp32 x [m][k] (any m) times the quantized weight;
    returns fp32 y [m][n].  Up to QW_MATMUL_GEMV_MAX_M rows (and up to 8 for
    matrices of at most 8192 rows the matrix-core GEMV takes) this is the
    codes GEMV; beyond, x is rounded to bf16 into ``work`` (allocated here
    when not given) and the matrix-core GEMM runs."""
    n, k = _check_rec(rec)
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != k:
        raise ValueError("x must be a contiguous float32 [m][k] tensor")
    m = x.shape[0]
    _check_tensor(x, torch.float32, m * k, "x")
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _check_tensor(out, torch.float32, m * n, "out", (m, n))
    nb = lib().qw_matmul_work_bytes(m, k)
    if work is None:
        work = _work(nb, x.device) if nb > 0 else None
    if work is not None and (not isinstance(work, torch.Tensor) or not work.is_contiguous()):
        raise ValueError("work must be a contiguous tensor")
    _on_device(rec, x, out, work)
    wb = work.numel() * work.element_size() if work is not None else 0
    _check(qw_matmul(rec["bits"], rec["group"], n, k, rec["payload"], rec["scales"], m, x, out,
                     work, wb, stream), "qw_matmul")
    return out


# ------------------------------------------------------------------ GPTQ


def _work(nbytes, device):
    if nbytes < 0:
        raise ValueError("invalid shape for a work-size query")
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def gptq_hessian(x, h=None, stream=None):
    """h += x^T x for a contiguous fp32 device tensor x [t][k]; allocates a
    zero fp64 [k][k] accumulator when ``h`` is None.  Returns h."""
    if x.dtype != torch.float32 or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous float32 [t][k] tensor")
    t, k = int(x.shape[0]), int(x.shape[1])
    if h is None:
        h = torch.zeros((k, k), dtype=torch.float64, device=x.device)
    if h.dtype != torch.float64 or not h.is_contiguous() or tuple(h.shape) != (k, k):
        raise ValueError("h must be a contiguous float64 [k][k] tensor")
    nb = lib().qw_gptq_hessian_work_bytes(k, t)
    work = _work(nb, x.device)
    _check(qw_gptq_hessian(k, t, x, h, work, nb, stream), "qw_gptq_hessian")
    return h


def gptq_factor(h, damp=0.01, stream=None, check=True):
    """U (fp64 [k][k], upper) with (h + damp*mean(diag h)*I)^-1 = U^T U.
    With ``check`` the stream is synchronized and a non-positive-definite h
    raises; otherwise (u, info) is returned with info a device int32."""
    if h.dtype != torch.float64 or not h.is_contiguous() or h.dim() != 2 \
            or h.shape[0] != h.shape[1]:
        raise ValueError("h must be a contiguous float64 [k][k] tensor")
    k = int(h.shape[0])
    u = torch.empty((k, k), dtype=torch.float64, device=h.device)
    info = torch.zeros(1, dtype=torch.int32, device=h.device)
    nb = lib().qw_gptq_factor_work_bytes(k)
    work = _work(nb, h.device)
    _check(qw_gptq_factor(k, h, float(damp), u, info, work, nb, stream), "qw_gptq_factor")
    if not check:
        return u, info
    if k and int(info.item()) != 0:
        raise QwError(-9, "qw_gptq_factor: the damped H is not positive definite")
    return u


def gptq_quantize_pack(w, u, bits, group, stream=None):
    """GPTQ codes of a contiguous fp32 device weight [n][k] with the factor
    ``u`` from gptq_factor; returns a record like quantize_pack."""
    if w.dtype != torch.float32 or not w.is_contiguous():
        raise ValueError("w must be a contiguous float32 tensor")
    n, k = _nk(w.shape)
    if u.dtype != torch.float64 or not u.is_contiguous() or tuple(u.shape) != (k, k):
        raise ValueError("u must be a contiguous float64 [k][k] tensor")
    nb = lib().qw_payload_bytes(bits, n, k)
    ns = lib().qw_num_scales(group, n, k)
    if nb < 0 or ns < 0:
        _check(QW_EBITS if bits not in (4, 8) else -2 if ns < 0 else -3, "gptq_quantize_pack")
    payload = torch.empty(nb, dtype=torch.uint8, device=w.device)
    scales = torch.empty(ns, dtype=torch.float32, device=w.device)
    wb = lib().qw_gptq_quantize_work_bytes(n, k)
    work = _work(wb, w.device)
    _check(qw_gptq_quantize_pack(bits, group, n, k, w, u, payload, scales, work, wb, stream),
           "qw_gptq_quantize_pack")
    return dict(bits=bits, group=group, shape=[n, k], payload=payload, scales=scales)


def gptq(w, h, bits, group, damp=0.01, stream=None):
    """The whole chain from an accumulated h: damping, factor, codes."""
    return gptq_quantize_pack(w, gptq_factor(h, damp, stream), bits, group, stream)


# ------------------------------------------------- block-scaled e4m3 codes
#
# Records: ``{block_rows, shape, codes, scales}``, shape [n][k] (or
# [experts][n][k]), codes float8_e4m3fn [.., n][pitch], scales fp32
# [.., rows of blocks][pitch / 128].
#
# These calls run on the device that their tensors are on, and on its current
# stream where none is given.


def _rows_of_blocks(n, block_rows):
    return (n + block_rows - 1) // block_rows


def _pitch(k):
    return (k + BLOCK - 1) // BLOCK * BLOCK


def _type(t, what):
    code = TYPES.get(t)
    if code is None:
        raise ValueError(f"{what} must be float32 or bfloat16, got {t}")
    return code


def _device_of(*ts):
    """Index of the one device that all tensors of a call are on (None entries
    aside)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d != dev:
            if d < 0:
                raise ValueError("libqw takes device tensors; a host tensor was passed")
            if dev is not None:
                raise ValueError(f"tensors on devices {dev} and {d}")
            dev = d
    return dev


def _run(what, dev, stream, fn, *args):
    """Calls the library with device ``dev`` as the current one (the library
    launches on it) and the stream behind the arguments: tensors as their
    addresses (0 for None and for empty ones)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        if stream.device.index != dev:
            raise ValueError(f"tensors on device {dev} and a stream of {stream.device}")
        raw = stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, raw)
    if status != QW_OK:
        _check(status, what)


def _device_among(args):
    """Index of the device of the first tensor among a call's arguments."""
    for a in args:
        if isinstance(a, dict):
            a = a.get("codes", a.get("pos"))
        if isinstance(a, torch.Tensor) and a.get_device() >= 0:
            return a.get_device()
    return None


def _on_stream(f):
    """``stream`` (a torch stream or a hipStream_t of the tensors' device) as
    the current stream of the whole call, so that what it allocates belongs
    to that stream too."""
    last = f.__code__.co_varnames.index("stream")  # its place if not a keyword

    @functools.wraps(f)
    def call(*args, **kwargs):
        stream = kwargs.pop("stream", None) if kwargs else None
        if len(args) == last + 1 and stream is None:
            *args, stream = args
        if stream is None:
            return f(*args, **kwargs)
        if not isinstance(stream, torch.cuda.Stream):
            dev = _device_among((*args, *kwargs.values()))
            stream = torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):
            return f(*args, stream=stream, **kwargs)
    return call


def _fits(t, dtypes, numel, what):
    """_check_tensor, quick when all is well; the tensor's address."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.numel() != numel \
            or not t.is_contiguous():
        _check_tensor(t, dtypes, numel, what)
    return t.data_ptr()


_CODES = (torch.float8_e4m3fn, torch.uint8)
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _check_block(rec, what="record", dims=(2, 3)):
    """Shape, block_rows and addresses of a block record whose codes and scales
    match them: (experts, n, k, block_rows, codes, scales)."""
    shape = rec["shape"]
    if len(shape) not in dims:
        raise ValueError(f"{what}: shape {list(shape)} has not {' or '.join(map(str, dims))} "
                         "dimensions")
    br = int(rec["block_rows"])
    if br != 1 and br != BLOCK:
        raise ValueError(f"{what}: block_rows must be 1 or {BLOCK}")
    e = int(shape[0]) if len(shape) == 3 else 1
    n, k = int(shape[-2]), int(shape[-1])
    kb = (k + BLOCK - 1) // BLOCK
    codes = _fits(rec["codes"], _CODES, e * n * kb * BLOCK, "record codes")
    scales = _fits(rec["scales"], _F32, e * ((n + br - 1) // br) * kb, "record scales")
    return e, n, k, br, codes, scales


def _empty_block(block_rows, shape, device):
    *lead, n, k = shape
    kp = _pitch(k)
    return dict(block_rows=block_rows, shape=list(shape),
                codes=torch.empty((*lead, n, kp), dtype=torch.float8_e4m3fn, device=device),
                scales=torch.empty((*lead, _rows_of_blocks(n, block_rows), kp // BLOCK),
                                   dtype=torch.float32, device=device))


@_on_stream
def block_quantize(w, block_rows=BLOCK, stream=None):
    """Quantize a contiguous fp32 or bf16 device tensor [n][k] (or
    [experts][n][k]) to e4m3 codes with a scale per block of ``block_rows`` x
    128: 128 for weights, 1 for activations.  Returns a record."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3) or not w.is_contiguous():
        raise ValueError("w must be a contiguous [n][k] or [experts][n][k] tensor")
    t = _type(w.dtype, "w")
    if block_rows not in (1, BLOCK):
        raise ValueError(f"block_rows must be 1 or {BLOCK}")
    dev = _device_of(w)
    rec = _empty_block(block_rows, w.shape, w.device)
    *lead, n, k = w.shape
    _run("qw_block_quantize", dev, stream, lib().qw_block_quantize, block_rows,
         lead[0] if lead else 1, n, k, t, w.data_ptr(), rec["codes"].data_ptr(),
         rec["scales"].data_ptr())
    return rec


@_on_stream
def block_quantize_swiglu(h, used=None, stream=None):
    """Record (1 x 128 blocks) of silu(gate) * up for h [rows][2 f], gate the
    first f columns.  ``used``: a device int32 tensor of one element, the
    number of rows there are; the others' codes are not written."""
    if not isinstance(h, torch.Tensor) or h.dim() != 2 or h.shape[1] % 2 or not h.is_contiguous():
        raise ValueError("h must be a contiguous [rows][2 f] tensor")
    t = _type(h.dtype, "h")
    count = None if used is None else _fits(used, _I32, 1, "used")
    rows, f = h.shape[0], h.shape[1] // 2
    dev = _device_of(h, used)
    rec = _empty_block(1, (rows, f), h.device)
    _run("qw_block_quantize_swiglu", dev, stream, lib().qw_block_quantize_swiglu, rows, f, t,
         h.data_ptr(), count, rec["codes"].data_ptr(), rec["scales"].data_ptr())
    return rec


@_on_stream
def block_unpack(rec, out=None, stream=None):
    """The fp32 values that a record's codes stand for."""
    e, n, k, br, codes, scales = _check_block(rec)
    shape = tuple(int(v) for v in rec["shape"])
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=rec["codes"].device)
    _check_tensor(out, torch.float32, e * n * k, "out", shape)
    dev = _device_of(rec["codes"], rec["scales"], out)
    _run("qw_block_unpack", dev, stream, lib().qw_block_unpack, br, e, n, k, codes, scales,
         out.data_ptr())
    return out


def _output(out, rows, cols, dtype, like):
    """``out`` checked, or a new [rows][cols] tensor of ``dtype`` on ``like``'s
    device; and its type's code."""
    if out is None:
        out = torch.empty((rows, cols), dtype=dtype, device=like.device)
    else:
        _check_tensor(out, tuple(TYPES) if dtype is None else dtype, rows * cols, "out",
                      (rows, cols))
    return out, _type(out.dtype, "out")


@_on_stream
def block_gemm(rec, x, out=None, out_dtype=None, stream=None):
    """y [m][n] = x . W^T of two records: ``rec`` the weight [n][k], ``x`` m
    rows of k values with 1 x 128 blocks; of ``out``'s type, ``out_dtype`` or
    fp32."""
    _, n, k, br, codes, scales = _check_block(rec, "record", (2,))
    _, m, kx, bx, xc, xs = _check_block(x, "x", (2,))
    if kx != k or bx != 1:
        raise ValueError(f"x must be a record of [m][{k}] with block_rows 1")
    out, yt = _output(out, m, n, out_dtype or (torch.float32 if out is None else None), x["codes"])
    dev = _device_of(rec["codes"], rec["scales"], x["codes"], x["scales"], out)
    _run("qw_block_gemm", dev, stream, lib().qw_block_gemm, br, n, k, codes, scales, m, xc, xs,
         yt, out.data_ptr())
    return out


@_on_stream
def block_matmul(rec, x, out=None, out_dtype=None, work=None, stream=None):
    """Float x [m][k] (fp32 or bf16, any m), quantized on the way with 1 x 128
    blocks, times a record's weight; returns y [m][n] of x's type (or
    ``out_dtype``)."""
    _, n, k, br, codes, scales = _check_block(rec, "record", (2,))
    xt = _check_matrix(x, "x", None, k)
    m = x.shape[0]
    out, yt = _output(out, m, n, out_dtype or (x.dtype if out is None else None), x)
    dev = _device_of(rec["codes"], rec["scales"], x, out, work)
    work, wp, wb = _workspace(work, lib().qw_block_matmul_work_bytes(m, k), x)
    _run("qw_block_matmul", dev, stream, lib().qw_block_matmul, br, n, k, codes, scales, m, xt,
         x.data_ptr(), yt, out.data_ptr(), wp, wb)
    return out


def _workspace(work, need, like):
    """(work, address, bytes) of the caller's work buffer, or of a new one of
    ``need`` bytes on ``like``'s device."""
    if work is None:
        if need < 0:
            raise ValueError("invalid shape for a work-size query")
        if need == 0:
            return None, None, 0
        work = torch.empty(need, dtype=torch.uint8, device=like.device)
        return work, work.data_ptr(), need
    if not isinstance(work, torch.Tensor) or not work.is_contiguous():
        raise ValueError("work must be a contiguous tensor")
    return work, work.data_ptr(), work.numel() * work.element_size()


@_on_stream
def block_gemm_grouped(rec, x, offsets, out=None, out_dtype=None, stream=None):
    """Rows sorted by expert times each expert's weight: ``rec`` [experts][n][k],
    ``x`` a record of [rows][k] with 1 x 128 blocks, ``offsets`` device int32
    [experts + 1] (moe_sort); y of ``out``'s type, ``out_dtype`` or fp32.  Rows
    that no expert has are left as they are in ``out``."""
    e, n, k, br, codes, scales = _check_block(rec, "record", (3,))
    _, rows, kx, bx, xc, xs = _check_block(x, "x", (2,))
    if kx != k or bx != 1:
        raise ValueError(f"x must be a record of [rows][{k}] with block_rows 1")
    first = _fits(offsets, _I32, e + 1, "offsets")
    out, yt = _output(out, rows, n, out_dtype or (torch.float32 if out is None else None),
                      x["codes"])
    dev = _device_of(rec["codes"], rec["scales"], x["codes"], x["scales"], offsets, out)
    _run("qw_block_gemm_grouped", dev, stream, lib().qw_block_gemm_grouped, br, e, n, k, codes,
         scales, rows, xc, xs, first, yt, out.data_ptr())
    return out


# ------------------------------------------ tokens sorted by expert and back


_IDS = {torch.int32: 4, torch.int64: 8}


def _check_ids(ids):
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.dtype not in _IDS \
            or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 or int64 [t][topk] tensor")
    return ids.shape[0], ids.shape[1], _IDS[ids.dtype]


@_on_stream
def moe_sort(ids, experts, order=True, work=None, stream=None):
    """Stable sort of the slots of ids [t][topk] by expert; an id outside
    [0, experts) takes its slot out.  Returns ``{pos, order, offsets}``: pos
    [t][topk] the slot's row (-1 if out), order [t * topk] the row's slot (-1
    behind the last row; None if ``order`` is false), offsets [experts + 1]."""
    t, topk, nbytes = _check_ids(ids)
    dev = _device_of(ids, work)
    work, wp, wb = _workspace(work, lib().qw_moe_sort_work_bytes(t, topk, experts), ids)
    pos = torch.empty((t, topk), dtype=torch.int32, device=ids.device)
    back = torch.empty(t * topk, dtype=torch.int32, device=ids.device) if order else None
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=ids.device)
    _run("qw_moe_sort", dev, stream, lib().qw_moe_sort, t, topk, experts, nbytes, ids.data_ptr(),
         pos.data_ptr(), back.data_ptr() if order else None, offsets.data_ptr(), wp, wb)
    return dict(pos=pos, order=back, offsets=offsets)


def _check_pos(route, t=None):
    pos = route["pos"]
    if not isinstance(pos, torch.Tensor) or pos.dim() != 2 or pos.dtype != torch.int32 \
            or not pos.is_contiguous() or (t is not None and pos.shape[0] != t):
        raise ValueError(f"pos must be a contiguous int32 [{'t' if t is None else t}][topk] tensor")
    return pos, pos.shape[0], pos.shape[1]


def _check_matrix(x, what, rows=None, cols=None, dtype=None):
    """The type's code of a contiguous matrix of those sizes."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_contiguous() \
            or (rows is not None and x.shape[0] != rows) or (cols is not None and x.shape[1] != cols):
        raise ValueError(f"{what} must be a contiguous [{'rows' if rows is None else rows}]"
                         f"[{'d' if cols is None else cols}] tensor")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {x.dtype}")
    return _type(x.dtype, what)


def _check_weights(weights, t, topk):
    if weights is None:
        return None
    _check_tensor(weights, torch.float32, t * topk, "weights", (t, topk))
    return weights.data_ptr()


@_on_stream
def moe_gather(x, route, out=None, stream=None):
    """Token rows x [t][d] into expert order, out [rows][d] (t * topk rows if
    not given); a row without a slot is left as it is."""
    xt = _check_matrix(x, "x")
    t, d = x.shape
    pos, _, topk = _check_pos(route, t)
    if out is None:
        out = torch.empty((t * topk, d), dtype=x.dtype, device=x.device)
    _check_matrix(out, "out", None, d, x.dtype)
    dev = _device_of(x, pos, out)
    _run("qw_moe_gather", dev, stream, lib().qw_moe_gather, t, topk, d, out.shape[0], xt,
         x.data_ptr(), pos.data_ptr(), out.data_ptr())
    return out


@_on_stream
def moe_gather_block(x, route, rows=None, stream=None):
    """Token rows x [t][d] into expert order as a record of [rows][d] (t *
    topk rows if not given) with 1 x 128 blocks; the codes of a row without a
    slot are not written."""
    xt = _check_matrix(x, "x")
    t, d = x.shape
    pos, _, topk = _check_pos(route, t)
    rows = t * topk if rows is None else int(rows)
    if rows < 0:
        raise ValueError("rows must not be negative")
    dev = _device_of(x, pos)
    rec = _empty_block(1, (rows, d), x.device)
    _run("qw_moe_gather_block", dev, stream, lib().qw_moe_gather_block, t, topk, d, rows, xt,
         x.data_ptr(), pos.data_ptr(), rec["codes"].data_ptr(), rec["scales"].data_ptr())
    return rec


@_on_stream
def moe_combine(ys, route, weights=None, out=None, out_dtype=None, stream=None):
    """y [t][d] = sum over a token's slots of weights [t][topk] (fp32; all 1
    if None) times their rows of ys [rows][d]; of ys' type or ``out_dtype``."""
    st = _check_matrix(ys, "ys")
    rows, d = ys.shape
    pos, t, topk = _check_pos(route)
    wp = _check_weights(weights, t, topk)
    out, yt = _output(out, t, d, out_dtype or (ys.dtype if out is None else None), ys)
    dev = _device_of(ys, pos, weights, out)
    _run("qw_moe_combine", dev, stream, lib().qw_moe_combine, t, topk, d, rows, st, ys.data_ptr(),
         pos.data_ptr(), wp, yt, out.data_ptr())
    return out


def moe_gather_backward(dxs, route, out=None, stream=None):
    """Gradient of moe_gather: dx [t][d], each token's sum of its rows of dxs."""
    return moe_combine(dxs, route, None, out, None, stream=stream)


@_on_stream
def moe_combine_backward(dy, ys, route, weights=None, dys=None, dweights=None, stream=None):
    """Gradients of moe_combine for dy [t][d]: (dys [rows][d], dweights fp32
    [t][topk]).  dy and ys have one type; rows of dys without a slot are left
    as they are."""
    st = _check_matrix(ys, "ys")
    rows, d = ys.shape
    pos, t, topk = _check_pos(route)
    _check_matrix(dy, "dy", t, d, ys.dtype)
    wp = _check_weights(weights, t, topk)
    if dys is None:
        dys = torch.empty_like(ys)
    _check_matrix(dys, "dys", rows, d, ys.dtype)
    if dweights is None:
        dweights = torch.empty((t, topk), dtype=torch.float32, device=dy.device)
    _check_tensor(dweights, torch.float32, t * topk, "dweights", (t, topk))
    dev = _device_of(dy, ys, pos, weights, dys, dweights)
    _run("qw_moe_combine_backward", dev, stream, lib().qw_moe_combine_backward, t, topk, d, rows,
         st, dy.data_ptr(), ys.data_ptr(), pos.data_ptr(), wp, dys.data_ptr(),
         dweights.data_ptr())
    return dys, dweights


@_on_stream
def moe_mlp(gate_up, down, x, ids, weights=None, out=None, out_dtype=None, work=None,
            stream=None):
    """A gated expert MLP in one call: x [t][d] (fp32 or bf16), ids [t][topk],
    weights fp32 [t][topk]; ``gate_up`` a record of [experts][2 f][d] (gate
    rows, then up rows), ``down`` of [experts][d][f].  y [t][d] of x's type or
    ``out_dtype``; fp32 y has fp32 sums in both products, bf16 y those of the 8-bit
    cores where there are many rows (qw.h)."""
    e, f2, d, br, gc, gs = _check_block(gate_up, "gate_up", (3,))
    ed, dd, f, bd, dc, ds = _check_block(down, "down", (3,))
    if ed != e or dd != d or f2 != 2 * f or bd != br:
        raise ValueError("gate_up must be [experts][2 f][d] and down [experts][d][f], with the "
                         "same block_rows")
    t, topk, nbytes = _check_ids(ids)
    xt = _check_matrix(x, "x", t, d)
    wp = _check_weights(weights, t, topk)
    out, yt = _output(out, t, d, out_dtype or (x.dtype if out is None else None), x)
    dev = _device_of(gate_up["codes"], gate_up["scales"], down["codes"], down["scales"], x, ids,
                     weights, out, work)
    work, kp, kb = _workspace(work, lib().qw_moe_mlp_work_bytes(t, topk, e, d, f), x)
    _run("qw_moe_mlp", dev, stream, lib().qw_moe_mlp, br, e, d, f, gc, gs, dc, ds, t, topk, xt,
         x.data_ptr(), nbytes, ids.data_ptr(), wp, yt, out.data_ptr(), kp, kb)
    return out


# ------------------------------------------- microscaled 4-bit codes, RMS norm
#
# Records: ``{bits: 4, block: 32, shape: [n, k], codes (uint8 [n][pitch / 2]), scales
# (uint8 [n][pitch / 32])}``, pitch being k rounded up to 512.


_CODES4 = (torch.uint8, torch.float4_e2m1fn_x2)
_SCALES4 = (torch.uint8, torch.float8_e8m0fnu)


def _mx_pitch(k):
    return (k + 511) // 512 * 512


def _check_mx(rec, what="record"):
    """Sizes and addresses of a 4-bit record whose codes and scales match its shape:
    (n, k, codes, scales)."""
    if rec.get("bits") != 4 or rec.get("block") != MX_BLOCK:
        raise ValueError(f"{what}: not a record of 4-bit codes with a scale per {MX_BLOCK}")
    n, k = _nk(rec["shape"])
    codes, scales = rec["codes"], rec["scales"]
    bytes32 = n * ((k + 511) // 512 * 16)  # a scale and 16 bytes of codes for 32 values
    if type(codes) is not torch.Tensor or codes.numel() != 16 * bytes32 or codes.dtype not in _CODES4 \
            or not codes.is_contiguous():
        _check_tensor(codes, _CODES4, 16 * bytes32, f"{what} codes")
    if type(scales) is not torch.Tensor or scales.numel() != bytes32 or scales.dtype not in _SCALES4 \
            or not scales.is_contiguous():
        _check_tensor(scales, _SCALES4, bytes32, f"{what} scales")
    return n, k, codes.data_ptr(), scales.data_ptr()


def _result(out, rows, cols, dtype, like):
    """_output, quick for a new tensor."""
    if out is None and dtype in TYPES:
        return like.new_empty((rows, cols), dtype=dtype), TYPES[dtype]
    return _output(out, rows, cols, dtype, like)


def _empty_mx(n, k, device):
    kp = _mx_pitch(k)
    return dict(bits=4, block=MX_BLOCK, shape=[n, k],
                codes=torch.empty((n, kp // 2), dtype=torch.uint8, device=device),
                scales=torch.empty((n, kp // MX_BLOCK), dtype=torch.uint8, device=device))


def _check_x_mx(x, k, what="x"):
    m, kx, codes, scales = _check_mx(x, what)
    if kx != k:
        raise ValueError(f"{what} must be a record of [m][{k}]")
    return m, codes, scales


@_on_stream
def mx_quantize(w, transpose=False, stream=None):
    """Quantize a contiguous fp32 or bf16 device tensor [n][k] to 4-bit
    floating-point codes with a power-of-two scale per 32 values of a row; with
    ``transpose`` the record is that of w's columns, [k][n].  Returns a record."""
    t = _check_matrix(w, "w")
    dev = _device_of(w)
    n, k = w.shape
    rec = _empty_mx(k, n, w.device) if transpose else _empty_mx(n, k, w.device)
    _run("qw_mx_quantize", dev, stream, lib().qw_mx_quantize, 1 if transpose else 0, n, k, t,
         w.data_ptr(), rec["codes"].data_ptr(), rec["scales"].data_ptr())
    return rec


@_on_stream
def mx_unpack(rec, out=None, stream=None):
    """The fp32 values that a record's 4-bit codes stand for."""
    n, k, codes, scales = _check_mx(rec)
    if out is None:
        out = torch.empty((n, k), dtype=torch.float32, device=rec["codes"].device)
    _check_tensor(out, torch.float32, n * k, "out", (n, k))
    dev = _device_of(rec["codes"], rec["scales"], out)
    _run("qw_mx_unpack", dev, stream, lib().qw_mx_unpack, n, k, codes, scales, out.data_ptr())
    return out


@_on_stream
def mx_gemm(rec, x, out=None, out_dtype=None, stream=None):
    """y [m][n] = x . W^T of two records: ``rec`` the weight [n][k], ``x`` m rows
    of k values; of ``out``'s type, ``out_dtype`` or fp32."""
    n, k, codes, scales = _check_mx(rec)
    m, xc, xs = _check_x_mx(x, k)
    out, yt = _result(out, m, n, out_dtype or (torch.float32 if out is None else None), x["codes"])
    dev = _device_of(rec["codes"], rec["scales"], x["codes"], x["scales"], out)
    _run("qw_mx_gemm", dev, stream, lib().qw_mx_gemm, n, k, codes, scales, m, xc, xs, yt,
         out.data_ptr())
    return out


@_on_stream
def mx_matmul(rec, x, out=None, out_dtype=None, work=None, stream=None):
    """Float x [m][k] (fp32 or bf16, any m), quantized to 4 bits on the way, times
    a record's weight; returns y [m][n] of x's type (or ``out_dtype``)."""
    n, k, codes, scales = _check_mx(rec)
    xt = _check_matrix(x, "x", None, k)
    m = x.shape[0]
    out, yt = _result(out, m, n, out_dtype or (x.dtype if out is None else None), x)
    dev = _device_of(rec["codes"], rec["scales"], x, out, work)
    work, wp, wb = _workspace(work, lib().qw_mx_matmul_work_bytes(m, k), x)
    _run("qw_mx_matmul", dev, stream, lib().qw_mx_matmul, n, k, codes, scales, m, xt,
         x.data_ptr(), yt, out.data_ptr(), wp, wb)
    return out


def _check_gain(weight, d):
    """Type's code and address of a norm's weight (or None)."""
    if weight is None:
        return 0, None
    return _type(weight.dtype, "weight"), _fits(weight, tuple(TYPES), d, "weight")


@_on_stream
def rms_norm(x, weight=None, residual=None, eps=1e-6, out=None, out_dtype=None, sum=None,
             quantize=None, stream=None):
    """RMS norm of s = x + residual (x itself without one), x [rows][d]: s / sqrt(mean
    s^2 + eps) * weight.  Returns (y, s).  ``quantize``: None (y is a tensor of
    ``out``'s type, ``out_dtype`` or x's), "block" (a record of e4m3 codes, 1 x 128
    blocks) or "mx" (a record of 4-bit codes).  s has x's type and goes to ``sum`` if
    given, which may be x or residual; weight [d] is fp32 or bf16."""
    t = _check_matrix(x, "x")
    rows, d = x.shape
    wt, wp = _check_gain(weight, d)
    if residual is not None:
        _check_matrix(residual, "residual", rows, d, x.dtype)
        if sum is None:
            sum = torch.empty_like(x)
    if sum is not None:
        _check_matrix(sum, "sum", rows, d, x.dtype)
    if quantize not in (None, "block", "mx"):
        raise ValueError('quantize must be None, "block" or "mx"')
    if quantize and (out is not None or out_dtype is not None):
        raise ValueError("a quantized result has no out and no out_dtype")
    dev = _device_of(x, weight, residual, sum, out)
    args = (rows, d, t, x.data_ptr(), None if residual is None else residual.data_ptr(),
            None if sum is None else sum.data_ptr(), wt, wp, eps)
    if quantize:
        y = _empty_block(1, (rows, d), x.device) if quantize == "block" else _empty_mx(rows, d, x.device)
        name = "qw_rms_norm_" + quantize
        _run(name, dev, stream, getattr(lib(), name), *args, y["codes"].data_ptr(),
             y["scales"].data_ptr())
    else:
        y, yt = _result(out, rows, d, out_dtype or (x.dtype if out is None else None), x)
        _run("qw_rms_norm", dev, stream, lib().qw_rms_norm, *args, yt, y.data_ptr())
    return y, x if sum is None else sum


@_on_stream
def rms_norm_backward(dy, s, weight=None, eps=1e-6, dsum=None, ds=None, dweight=None, work=None,
                      stream=None):
    """Gradients of rms_norm for the output gradient dy [rows][d], s the sum that it
    returned: (ds, dweight).  ds is the gradient of x and of the residual, with
    ``dsum``, the gradient that reaches s past the norm, added.  dy, s, dsum and ds
    have one type; dweight is fp32 [d], None without a weight."""
    t = _check_matrix(s, "s")
    rows, d = s.shape
    _check_matrix(dy, "dy", rows, d, s.dtype)
    wt, wp = _check_gain(weight, d)
    if dsum is not None:
        _check_matrix(dsum, "dsum", rows, d, s.dtype)
    if ds is None:
        ds = torch.empty_like(s)
    _check_matrix(ds, "ds", rows, d, s.dtype)
    if dweight is None and weight is not None:
        dweight = torch.empty(d, dtype=torch.float32, device=s.device)
    if dweight is not None:
        _check_tensor(dweight, torch.float32, d, "dweight", (d,))
    dev = _device_of(dy, s, weight, dsum, ds, dweight, work)
    need = 0 if dweight is None else lib().qw_rms_norm_backward_work_bytes(rows, d)
    work, kp, kb = _workspace(work, need, s)
    _run("qw_rms_norm_backward", dev, stream, lib().qw_rms_norm_backward, rows, d, t,
         dy.data_ptr(), s.data_ptr(), wt, wp, eps, None if dsum is None else dsum.data_ptr(),
         ds.data_ptr(), None if dweight is None else dweight.data_ptr(), kp, kb)
    return ds, dweight


def _check_gate_up(rec):
    """(f, k, codes, scales) of the record of a gate and an up matrix."""
    n, k, codes, scales = _check_mx(rec, "gate_up")
    if n % 2:
        raise ValueError("gate_up must be a record of [2 f][k]")
    return n // 2, k, codes, scales


@_on_stream
def mx_gated(gate_up, x, out=None, out_dtype=None, quantize=False, stream=None):
    """silu(gate) * up in one product: ``gate_up`` a record of [2 f][k] (gate rows,
    then up rows), ``x`` a record of [m][k].  Returns h [m][f] of ``out``'s type,
    ``out_dtype`` or fp32, or with ``quantize`` its record of 4-bit codes."""
    f, k, codes, scales = _check_gate_up(gate_up)
    m, xc, xs = _check_x_mx(x, k)
    dev = _device_of(gate_up["codes"], gate_up["scales"], x["codes"], x["scales"], out)
    if quantize:
        if out is not None or out_dtype is not None:
            raise ValueError("a quantized result has no out and no out_dtype")
        h = _empty_mx(m, f, x["codes"].device)
        _run("qw_mx_gated_codes", dev, stream, lib().qw_mx_gated_codes, f, k, codes, scales, m, xc,
             xs, h["codes"].data_ptr(), h["scales"].data_ptr())
        return h
    out, ht = _result(out, m, f, out_dtype or (torch.float32 if out is None else None), x["codes"])
    _run("qw_mx_gated", dev, stream, lib().qw_mx_gated, f, k, codes, scales, m, xc, xs, ht,
         out.data_ptr())
    return out


@_on_stream
def mx_gated_backward(gate_up, x, dh, out=None, h=True, stream=None):
    """Gradients of mx_gated with regard to gate and up for dh [m][f]: (dgate | dup
    [m][2 f], h [m][f]), of dh's type.  gate and up are computed again.  ``h``: True,
    a tensor for it, or False (None is returned for it)."""
    f, k, codes, scales = _check_gate_up(gate_up)
    m, xc, xs = _check_x_mx(x, k)
    t = _check_matrix(dh, "dh", m, f)
    if out is None:
        out = torch.empty((m, 2 * f), dtype=dh.dtype, device=dh.device)
    _check_matrix(out, "out", m, 2 * f, dh.dtype)
    if h is True:
        h = torch.empty_like(dh)
    elif h is False:
        h = None
    if h is not None:
        _check_matrix(h, "h", m, f, dh.dtype)
    dev = _device_of(gate_up["codes"], gate_up["scales"], x["codes"], x["scales"], dh, out, h)
    _run("qw_mx_gated_backward", dev, stream, lib().qw_mx_gated_backward, f, k, codes, scales, m,
         xc, xs, t, dh.data_ptr(), out.data_ptr(), None if h is None else h.data_ptr())
    return out, h


@_on_stream
def mx_mlp(gate_up, down, x, out=None, out_dtype=None, work=None, stream=None):
    """A gated feed-forward block in one call: x [m][d] (fp32 or bf16), ``gate_up`` a
    record of [2 f][d] (gate rows, then up rows), ``down`` of [d][f]; x and the gated
    values are quantized to 4 bits on the way.  y [m][d] of x's type or ``out_dtype``."""
    f, d, gc, gs = _check_gate_up(gate_up)
    dd, df, dc, ds = _check_mx(down, "down")
    if dd != d or df != f:
        raise ValueError("gate_up must be a record of [2 f][d] and down of [d][f]")
    xt = _check_matrix(x, "x", None, d)
    m = x.shape[0]
    out, yt = _result(out, m, d, out_dtype or (x.dtype if out is None else None), x)
    dev = _device_of(gate_up["codes"], gate_up["scales"], down["codes"], down["scales"], x, out,
                     work)
    work, kp, kb = _workspace(work, lib().qw_mx_mlp_work_bytes(m, d, f), x)
    _run("qw_mx_mlp", dev, stream, lib().qw_mx_mlp, d, f, gc, gs, dc, ds, m, xt, x.data_ptr(), yt,
         out.data_ptr(), kp, kb)
    return out
