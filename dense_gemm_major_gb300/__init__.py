"""Python binding of the GB300 dense row-major GEMM library.

The binding only marshals arguments: every step of the GEMM runs in the
CUDA library ``libdense_gemm.so`` (built in-tree by ``_build.build()``),
whose C ABI is declared in ``include/dense_gemm.h``, (microscaled
operands) ``include/dense_gemm_mx.h`` and (products grouped by expert)
``include/dense_gemm_group.h`` and (4-bit weights with group scales)
``include/dense_gemm_q4.h``.  The functions of the same names as
the C entry points take integers (device addresses, sizes, a
``cudaStream_t`` value); ``matmul``, the ``mx_*``, the ``grouped_*`` functions
and ``q4_linear`` are convenience wrappers for torch tensors on the current device and stream.
There is no fallback: if the library is missing the calls raise.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdense_gemm.so")

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_MISALIGNED = 2
GEMM_ERR_UNSUPPORTED_DEVICE = 3
GEMM_ERR_LAUNCH = 4
GEMM_ERR_DEVICE_TIMEOUT = 5
GEMM_ERR_SCRATCH_LIMIT = 6

PATH_NOOP, PATH_ZERO_FILL, PATH_SIMT_TMA, PATH_SIMT_CPASYNC, PATH_TC_TMA, PATH_SIMT_MIXED = range(6)
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}

# Every symbol the headers under include/ declare.
EXPORTED = ("gemm_f32", "gemm_f16", "gemm_bf16", "gemm_status_string", "gemm_device_check",
            "gemm_plan", "gemm_smem_layout_offset", "gemm_selftest_timeout", "gemm_f32_noalloc",
            "gemm_f32_ex", "gemm_f16_ex", "gemm_bf16_ex", "gemm_plan_ex",
            "gemm_f32_op", "gemm_f16_op", "gemm_bf16_op", "gemm_plan_op", "gemm_host",
            "gemm_host_blocks", "gemm_host_k_blocks", "gemm_selftest_flag_timeout",
            "gemm_plan_resident", "gemm_pair_clusters", "gemm_sgemm_clusters", "gemm_pair_units",
            "gemm_probe_ffma",
            "gemm_probe_ffma_threads",
            "gemm_mx_code_ld", "gemm_mx_scale_bytes", "gemm_mx_quantize", "gemm_mx_dequantize",
            "gemm_mx4", "gemm_mx4_linear", "gemm_mx_grad",
            "gemm_grouped", "gemm_grouped_grad", "gemm_q4_linear")

# Microscaled formats (gemm_mx_format_t).
MXFP4, MXINT8 = 0, 1
_MX_CODES = {"mxfp4": MXFP4, "mxint8": MXINT8, MXFP4: MXFP4, MXINT8: MXINT8}

# Operand storage (gemm_op_t): N = as stored row-major, T = stored transposed
# (A as K x M, B as N x K).
OP_N, OP_T = 0, 1
_OP_CODES = {"N": OP_N, "T": OP_T, OP_N: OP_N, OP_T: OP_T}


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})" if what
                         else f"{status_string(status)} (status {status})")


class Plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("block_m", ctypes.c_int), ("block_n", ctypes.c_int),
                ("block_k", ctypes.c_int), ("stages", ctypes.c_int), ("threads", ctypes.c_int),
                ("ctas", ctypes.c_int), ("tiles", ctypes.c_int), ("smem_bytes", ctypes.c_int),
                ("split_tiles", ctypes.c_int), ("split_pieces", ctypes.c_int),
                ("cluster_ctas", ctypes.c_int), ("splitk_slices", ctypes.c_int),
                ("workspace_bytes", ctypes.c_longlong), ("pack", ctypes.c_int),
                ("pack_bytes", ctypes.c_longlong), ("split_in_k", ctypes.c_int),
                ("streamk_first_tile", ctypes.c_int)]


_lib = None


def load() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built ({LIB_PATH} missing); "
                           "run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    i, vp = ctypes.c_int, ctypes.c_void_p
    gemm_args = [i, i, i, vp, i, vp, i, vp, i, vp]
    for name in ("gemm_f32", "gemm_f16", "gemm_bf16", "gemm_f32_noalloc"):
        fn = getattr(lib, name)
        fn.restype = i
        fn.argtypes = gemm_args
    f = ctypes.c_float
    for name in ("gemm_f32_ex", "gemm_f16_ex", "gemm_bf16_ex"):
        fn = getattr(lib, name)
        fn.restype = i
        fn.argtypes = [i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.gemm_plan_ex.restype = i
    lib.gemm_plan_ex.argtypes = [i, i, i, i, f, vp, i, vp, i, f, vp, i, i, ctypes.POINTER(Plan)]
    for name in ("gemm_f32_op", "gemm_f16_op", "gemm_bf16_op"):
        fn = getattr(lib, name)
        fn.restype = i
        fn.argtypes = [i, i, i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.gemm_plan_op.restype = i
    lib.gemm_plan_op.argtypes = [i, i, i, i, i, i, f, vp, i, vp, i, f, vp, i, i,
                                 ctypes.POINTER(Plan)]
    lib.gemm_plan_resident.restype = i
    lib.gemm_plan_resident.argtypes = [i, i, i, i, i, i, f, vp, i, vp, i, f, vp, i, i, i,
                                       ctypes.POINTER(Plan)]
    lib.gemm_pair_units.restype = i
    lib.gemm_pair_units.argtypes = [ctypes.POINTER(Plan), i, i, i, i,
                                    ctypes.POINTER(ctypes.c_int), i]
    lib.gemm_probe_ffma.restype = i
    lib.gemm_probe_ffma.argtypes = [i, i, vp, vp, ctypes.POINTER(ctypes.c_double)]
    lib.gemm_probe_ffma_threads.restype = i
    lib.gemm_probe_ffma_threads.argtypes = []
    lib.gemm_pair_clusters.restype = i
    lib.gemm_pair_clusters.argtypes = []
    lib.gemm_sgemm_clusters.restype = i
    lib.gemm_sgemm_clusters.argtypes = [i, i]
    lib.gemm_host.restype = i
    lib.gemm_host.argtypes = [i, i, i, i, i, i, f, vp, i, vp, i, f, vp, i, vp]
    lib.gemm_host_blocks.restype = i
    lib.gemm_host_blocks.argtypes = [i, i, i, i]
    lib.gemm_host_k_blocks.restype = i
    lib.gemm_host_k_blocks.argtypes = [i, i, i, i]
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_status_string.argtypes = [i]
    lib.gemm_device_check.restype = i
    lib.gemm_device_check.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.gemm_plan.restype = i
    lib.gemm_plan.argtypes = [i, i, i, i, vp, i, vp, i, vp, i, i, ctypes.POINTER(Plan)]
    lib.gemm_smem_layout_offset.restype = i
    lib.gemm_smem_layout_offset.argtypes = [i, i, i]
    lib.gemm_selftest_timeout.restype = i
    lib.gemm_selftest_timeout.argtypes = [ctypes.c_uint, vp]
    lib.gemm_selftest_flag_timeout.restype = i
    lib.gemm_selftest_flag_timeout.argtypes = [ctypes.c_uint, vp]
    lib.gemm_mx_code_ld.restype = i
    lib.gemm_mx_code_ld.argtypes = [i, i]
    lib.gemm_mx_scale_bytes.restype = ctypes.c_longlong
    lib.gemm_mx_scale_bytes.argtypes = [i, i]
    lib.gemm_mx_quantize.restype = i
    lib.gemm_mx_quantize.argtypes = [i, i, i, i, i, vp, i, vp, i, vp, vp]
    lib.gemm_mx_dequantize.restype = i
    lib.gemm_mx_dequantize.argtypes = [i, i, i, i, vp, i, vp, vp, i, vp]
    lib.gemm_mx4.restype = i
    lib.gemm_mx4.argtypes = [i, i, i, i, f, vp, i, vp, vp, i, vp, f, vp, i, vp]
    lib.gemm_mx4_linear.restype = i
    lib.gemm_mx4_linear.argtypes = [i, i, i, i, vp, i, vp, i, vp, vp, i, vp]
    lib.gemm_mx_grad.restype = i
    lib.gemm_mx_grad.argtypes = [i, i, i, i, i, i, i, f, vp, i, vp, i, vp, f, vp, i, vp]
    ll = ctypes.c_longlong
    lib.gemm_grouped.restype = i
    lib.gemm_grouped.argtypes = [i, i, i, i, i, i, i, f, vp, i, vp, i, ll, vp, f, vp, i, vp]
    lib.gemm_grouped_grad.restype = i
    lib.gemm_grouped_grad.argtypes = [i, i, i, i, i, i, f, vp, i, vp, i, vp, f, vp, i, ll, vp]
    lib.gemm_q4_linear.restype = i
    lib.gemm_q4_linear.argtypes = [i, i, i, i, i, i, vp, i, vp, i, vp, vp, vp, vp, i, vp]
    _lib = lib
    return lib


# ------------------------------------------------------------ C-ABI mirrors

def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_f16(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return load().gemm_bf16(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    """gemm_f32 for callers that cannot allocate device memory: split-K
    partials go to the library's fixed 16 MiB device array."""
    return load().gemm_f32_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_f16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_bf16_ex(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_plan_ex(dtype, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, num_sms=152):
    """Returns (status, Plan) of a scaled call."""
    plan = Plan()
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    st = load().gemm_plan_ex(code, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, num_sms,
                             ctypes.byref(plan))
    return st, plan


def status_string(status: int) -> str:
    return load().gemm_status_string(int(status)).decode()


gemm_status_string = status_string


def gemm_device_check(stream=0):
    """Returns (status, fault_bits)."""
    bits = ctypes.c_uint(0)
    st = load().gemm_device_check(stream, ctypes.byref(bits))
    return st, bits.value


def gemm_plan(dtype, M, N, K, A, lda, B, ldb, C, ldc, num_sms=152):
    """Returns (status, Plan)."""
    plan = Plan()
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    st = load().gemm_plan(code, M, N, K, A, lda, B, ldb, C, ldc, num_sms, ctypes.byref(plan))
    return st, plan


def gemm_smem_layout_offset(layout: int, row: int, col: int) -> int:
    return load().gemm_smem_layout_offset(layout, row, col)


def gemm_selftest_timeout(timeout_us: int, stream=0) -> int:
    return load().gemm_selftest_timeout(timeout_us, stream)


def gemm_selftest_flag_timeout(timeout_us: int, stream=0) -> int:
    return load().gemm_selftest_flag_timeout(timeout_us, stream)

def gemm_plan_op(dtype, op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, num_sms=152):
    """Returns (status, Plan) of a call with operand storages."""
    plan = Plan()
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    st = load().gemm_plan_op(code, _OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A, lda, B,
                             ldb, beta, C, ldc, num_sms, ctypes.byref(plan))
    return st, plan


def gemm_plan_resident(dtype, op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                       num_sms=152, pair_clusters=0):
    """Returns (status, Plan) for a device holding only `pair_clusters` CTA
    pairs at once (0: every SM)."""
    plan = Plan()
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    st = load().gemm_plan_resident(code, _OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A,
                                   lda, B, ldb, beta, C, ldc, num_sms, pair_clusters,
                                   ctypes.byref(plan))
    return st, plan


def gemm_pair_units(plan, M, N, K, pair):
    """The units CTA pair `pair` of a pair-kernel plan runs, in order, as
    tuples (tm, tn, n_off, n_w, kb, ke, kind, slot)."""
    n = load().gemm_pair_units(ctypes.byref(plan), M, N, K, pair, None, 0)
    if n < 0:
        raise ValueError("gemm_pair_units: not a CTA-pair plan or bad arguments")
    buf = (ctypes.c_int * (8 * max(n, 1)))()
    load().gemm_pair_units(ctypes.byref(plan), M, N, K, pair, buf, n)
    return [tuple(buf[8 * j: 8 * j + 8]) for j in range(n)]


def gemm_probe_ffma(blocks, iters, out, stream=0):
    """Launches the FFMA throughput probe; returns (status, flops)."""
    fl = ctypes.c_double(0.0)
    st = load().gemm_probe_ffma(blocks, iters, out, stream, ctypes.byref(fl))
    return st, fl.value


def gemm_probe_ffma_threads() -> int:
    return load().gemm_probe_ffma_threads()


def gemm_pair_clusters() -> int:
    return load().gemm_pair_clusters()


def gemm_sgemm_clusters(config, cluster_size) -> int:
    return load().gemm_sgemm_clusters(config, cluster_size)


def gemm_f32_op(op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f32_op(_OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A, lda, B, ldb,
                              beta, C, ldc, stream)


def gemm_f16_op(op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_f16_op(_OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A, lda, B, ldb,
                              beta, C, ldc, stream)


def gemm_bf16_op(op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return load().gemm_bf16_op(_OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A, lda, B,
                               ldb, beta, C, ldc, stream)


_ENTRY = {"f32": gemm_f32, "f16": gemm_f16, "bf16": gemm_bf16}
_ENTRY_EX = {"f32": gemm_f32_ex, "f16": gemm_f16_ex, "bf16": gemm_bf16_ex}


def gemm(dtype: str, M, N, K, A, lda, B, ldb, C, ldc, stream=0) -> int:
    return _ENTRY[dtype](M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_ex(dtype: str, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    return _ENTRY_EX[dtype](M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


_ENTRY_OP = {"f32": gemm_f32_op, "f16": gemm_f16_op, "bf16": gemm_bf16_op}


def gemm_op(dtype: str, op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
            stream=0) -> int:
    return _ENTRY_OP[dtype](op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_host(dtype, op_a, op_b, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
              stream=0) -> int:
    """gemm_host: A, B, C are host addresses (see include/dense_gemm.h)."""
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_host(code, _OP_CODES[op_a], _OP_CODES[op_b], M, N, K, alpha, A, lda, B,
                            ldb, beta, C, ldc, stream)


def gemm_host_blocks(dtype, M, N, num_sms=152) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_host_blocks(code, M, N, num_sms)


def gemm_host_k_blocks(dtype, M, N, K) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_host_k_blocks(code, M, N, K)


def gemm_mx_code_ld(fmt, K) -> int:
    return load().gemm_mx_code_ld(_MX_CODES.get(fmt, -1), K)


def gemm_mx_scale_bytes(R, K) -> int:
    return load().gemm_mx_scale_bytes(R, K)


def gemm_mx_quantize(fmt, dtype, op, R, K, X, ldx, codes, ldq, scales, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_mx_quantize(_MX_CODES.get(fmt, -1), code, _OP_CODES.get(op, -1), R, K, X,
                                   ldx, codes, ldq, scales, stream)


def gemm_mx_dequantize(fmt, dtype, R, K, codes, ldq, scales, Y, ldy, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_mx_dequantize(_MX_CODES.get(fmt, -1), code, R, K, codes, ldq, scales, Y,
                                     ldy, stream)


def gemm_mx4(dtype, M, N, K, alpha, a_codes, lda, a_scales, b_codes, ldb, b_scales, beta, C, ldc,
             stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_mx4(code, M, N, K, alpha, a_codes, lda, a_scales, b_codes, ldb, b_scales,
                           beta, C, ldc, stream)


def gemm_mx4_linear(dtype, M, N, K, X, ldx, w_codes, ldw, w_scales, Y, ldy, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_mx4_linear(code, M, N, K, X, ldx, w_codes, ldw, w_scales, Y, ldy, stream)


def gemm_mx_grad(fmt, dtype, op_a, dtype_c, M, N, K, alpha, A, lda, b_codes, ldb, b_scales, beta,
                 C, ldc, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    code_c = DTYPE_CODES[dtype_c] if isinstance(dtype_c, str) else int(dtype_c)
    return load().gemm_mx_grad(_MX_CODES.get(fmt, -1), code, _OP_CODES.get(op_a, -1), code_c, M,
                               N, K, alpha, A, lda, b_codes, ldb, b_scales, beta, C, ldc, stream)


def gemm_grouped(dtype, op_b, dtype_c, rows, N, K, groups, alpha, A, lda, B, ldb, stride_b,
                 offsets, beta, C, ldc, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    code_c = DTYPE_CODES[dtype_c] if isinstance(dtype_c, str) else int(dtype_c)
    return load().gemm_grouped(code, _OP_CODES.get(op_b, -1), code_c, rows, N, K, groups, alpha, A,
                               lda, B, ldb, stride_b, offsets, beta, C, ldc, stream)


def gemm_grouped_grad(dtype, dtype_c, rows, M, N, groups, alpha, A, lda, X, ldx, offsets, beta, C,
                      ldc, stride_c, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    code_c = DTYPE_CODES[dtype_c] if isinstance(dtype_c, str) else int(dtype_c)
    return load().gemm_grouped_grad(code, code_c, rows, M, N, groups, alpha, A, lda, X, ldx,
                                    offsets, beta, C, ldc, stride_c, stream)


def gemm_q4_linear(dtype, group, rows, N, K, experts, X, ldx, codes, ldq, scales, zeros, offsets,
                   Y, ldy, stream=0) -> int:
    code = DTYPE_CODES[dtype] if isinstance(dtype, str) else int(dtype)
    return load().gemm_q4_linear(code, group, rows, N, K, experts, X, ldx, codes, ldq, scales,
                                 zeros, offsets, Y, ldy, stream)


# ------------------------------------------------------------ torch wrapper

def _torch_dtype_code(t):
    import torch
    return {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[t.dtype]


def _ld(t, rows, cols):
    if t.dim() != 2 or (cols > 1 and t.stride(1) != 1):
        raise ValueError("operands must be 2-D row-major (unit column stride)")
    return t.stride(0) if rows > 1 else max(cols, t.stride(0), 1)


def _operand(t, rows, cols):
    """(op, ld) of a rows x cols operand: row-major (unit column stride) as
    op N, or a transposed view of a row-major array (unit row stride) as
    op T, read where it is without a copy."""
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if cols <= 1 or t.stride(1) == 1:
        return OP_N, _ld(t, rows, cols)
    if rows <= 1 or t.stride(0) == 1:
        return OP_T, t.stride(1) if cols > 1 else max(rows, 1)
    raise ValueError("operands must have a unit row or column stride")


def matmul(A, B, out=None, stream=None, alpha=1.0, beta=0.0):
    """out = alpha * (A @ B) + beta * out for tensors of one dtype (float32,
    float16, bfloat16), queued on ``stream`` (default: torch's current
    stream).  A and B may be row-major or transposed views of row-major
    arrays (e.g. ``X.t()``), which are read in place (op T); out is
    row-major.  Row-padded views (row stride > width) are accepted; beta != 0
    needs ``out``.  CUDA tensors run on the device as queued work; CPU
    tensors (page-locked or not) go through gemm_host, which stages them on
    the GPU, and the call returns once out holds the result (raising
    GemmError if a device-side wait gave up on the way)."""
    import torch
    on_host = A.device.type == "cpu" and B.device.type == "cpu"
    if not on_host and (A.device.type != "cuda" or B.device.type != "cuda"):
        raise ValueError("operands must be both CUDA tensors or both CPU tensors")
    if A.dtype != B.dtype:
        raise ValueError("A and B must have the same dtype")
    code = _torch_dtype_code(A)
    M, K = A.shape
    K2, N = B.shape
    if K != K2:
        raise ValueError(f"inner dimensions differ: {K} vs {K2}")
    if out is None:
        if beta != 0:
            raise ValueError("beta != 0 needs an existing out")
        out = torch.empty((M, N), dtype=A.dtype, device=A.device, pin_memory=on_host)
    elif out.shape != (M, N) or out.dtype != A.dtype or out.device.type != A.device.type:
        raise ValueError("out has the wrong shape, dtype or device")
    if stream is None:
        stream = (torch.cuda.current_stream() if on_host
                  else torch.cuda.current_stream(A.device)).cuda_stream
    op_a, lda = _operand(A, M, K)
    op_b, ldb = _operand(B, K, N)
    if on_host:
        st = gemm_host(code, op_a, op_b, M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(),
                       ldb, float(beta), out.data_ptr(), _ld(out, M, N), stream)
        if st != GEMM_OK:
            raise GemmError(st, "gemm_host")
        # Waits for the result and reads the device fault word: a bounded
        # device wait that gave up means out does not hold the product.
        st, bits = gemm_device_check(stream)
        if st != GEMM_OK:
            raise GemmError(st, f"gemm_host (fault bits {bits:#x})")
        return out
    if op_a == OP_N and op_b == OP_N and alpha == 1.0 and beta == 0.0:
        st = gemm(code, M, N, K, A.data_ptr(), lda, B.data_ptr(), ldb,
                  out.data_ptr(), _ld(out, M, N), stream)
    else:
        st = gemm_op(code, op_a, op_b, M, N, K, float(alpha), A.data_ptr(), lda, B.data_ptr(),
                     ldb, float(beta), out.data_ptr(), _ld(out, M, N), stream)
    if st != GEMM_OK:
        raise GemmError(st, f"gemm_{code}")
    return out


# ------------------------------------------------------------ microscaled operands
#
# These functions are thin: the extension _mxcall (csrc/mx_python.cpp) reads the
# tensors, allocates the result and calls the C ABI.  A layer of a few tokens
# takes a few microseconds on the GPU, less than the same steps in Python.
#
# ``stream`` is a cudaStream_t value (default: torch's current stream).  A result
# allocated here belongs to the stream that it is written on, and may be used
# on torch's current one as well once that waits for the work.  Operands that
# are freed while work on another stream than their own may still read them
# must be recorded there first (Tensor.record_stream, MXTensor.record_stream).
#
# Like matmul(), none of them takes part in autograd: results never require a
# gradient.  MXLinear in examples/mx_layer.py is a torch.autograd.Function of a
# layer's three products.

_mx = None


def _load_mx():
    """The extension, given torch's objects at its first use."""
    global _mx
    if _mx is None:
        load()
        import torch
        from . import _mxcall as ext
        ext.setup(torch, MXTensor, GemmError)
        _mx = ext
    return _mx


def _on_stream(stream, call):
    """call(), whose result is newly allocated, with ``stream`` as torch's
    current stream: memory of the caller's stream might still be in use there,
    by work queued before it was freed."""
    import torch
    current = torch.cuda.current_stream()
    if stream == current.cuda_stream:
        return call()
    # (1 is cudaStreamLegacy, another name of the default stream.)
    with torch.cuda.stream(torch.cuda.ExternalStream(0 if stream == 1 else stream)):
        result = call()
    result.record_stream(current)
    return result


class MXTensor:
    """A quantised rows x cols array on the GPU: ``codes`` (uint8, rows x
    pitch) and ``scales`` (uint8) in the layout that include/dense_gemm_mx.h
    describes; ``fmt`` is "mxfp4" or "mxint8"."""
    __slots__ = ("_codes", "_scales", "_buffer", "_device", "rows", "cols", "fmt", "_ld")

    def __init__(self, codes, scales, cols, fmt="mxfp4"):
        self.rows, self._ld, self._device = (_mx or _load_mx()).describe(codes, scales, cols, fmt)
        self._codes, self._scales, self._buffer = codes, scales, None
        self.cols, self.fmt = cols, fmt

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def codes(self):
        if self._codes is None:
            self._codes = self._buffer[:self.rows * self._ld].view(self.rows, self._ld)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._scales = self._buffer[self.rows * self._ld:]
        return self._scales

    @property
    def device(self):
        return (self._codes if self._buffer is None else self._buffer).device

    def record_stream(self, stream):
        """Tensor.record_stream of the codes and scales."""
        for t in (self._codes, self._scales) if self._buffer is None else (self._buffer,):
            t.record_stream(stream)


def mx_quantize(X, fmt="mxfp4", stream=None):
    """X (rows x cols; float32, float16 or bfloat16; row-major or a
    transposed view, read in place) in format ``fmt``: blocks of 32 along
    the columns.  Returns an MXTensor."""
    if stream is not None:
        return _on_stream(stream, lambda: mx_quantize(X, fmt))
    q = MXTensor.__new__(MXTensor)
    q._codes = q._scales = None
    q._buffer, q.rows, q.cols, q._ld, q._device = (_mx or _load_mx()).quantize(X, fmt, stream)
    q.fmt = fmt
    return q


def mx_dequantize(q, dtype=None, out=None, stream=None):
    """The values of MXTensor ``q`` as a rows x cols tensor of ``dtype``
    (default bfloat16, or that of ``out``)."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: mx_dequantize(q, dtype))
    return (_mx or _load_mx()).dequantize(q, dtype, out, stream)


def mx_matmul(A, B, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """alpha * (A @ B.T) + beta * out for MXFP4 operands A (M x K) and B
    (N x K); the result is of ``dtype`` (default bfloat16, or that of
    ``out``)."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: mx_matmul(A, B, None, dtype, alpha, beta))
    return (_mx or _load_mx()).matmul(A, B, out, dtype, alpha, beta, stream)


def mx_linear(x, W, out=None, stream=None):
    """x @ W.T with x (M x K, row-major) quantised to MXFP4 on the way and W
    (N x K) an MXFP4 MXTensor; the result has x's dtype and no gradient."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: mx_linear(x, W))
    return (_mx or _load_mx()).linear(x, W, out, stream)


def mx_grad(A, B, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """alpha * (A @ B) + beta * out with A (M x K, float16 or bfloat16,
    row-major or a transposed view) and B a K x N MXTensor: ``mx_grad(dY, W)``
    is the gradient of a layer's input, ``mx_grad(dY.t(), kept_x)`` that of
    its weights.  A has rows of a multiple of 16 bytes, or is contiguous (rows
    of other widths are then copied to aligned ones first).  The result is of A's dtype or float32 (``dtype``, or that
    of ``out``)."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: mx_grad(A, B, None, dtype, alpha, beta))
    return (_mx or _load_mx()).grad(A, B, out, dtype, alpha, beta, stream)


# ------------------------------------------------------------ products grouped by expert
#
# Rows are sorted by group: group g's rows are offsets[g] .. offsets[g + 1] - 1,
# ``offsets`` a contiguous int32 CUDA tensor of groups + 1 elements, which is read
# when the work runs (include/dense_gemm_group.h has the rules).  Thin like the
# mx_* functions (csrc/group_python.cpp); what is said there of streams and
# autograd holds here.  ExpertLinear in examples/expert_layer.py is a
# torch.autograd.Function of the three products.

_group = None


def _load_group():
    """The extension, given torch's objects at its first use."""
    global _group
    if _group is None:
        load()
        import torch
        from . import _groupcall as ext
        ext.setup(torch, Q4Tensor, GemmError)
        _group = ext
    return _group


def grouped_matmul(A, B, offsets, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """out[i] = alpha * (A[i] @ B[g]) + beta * out[i] for the rows i of each
    group g.  A (rows x K) and B (groups x K x N) are float16 or bfloat16, A
    row-major, B's matrices row-major or transposed views, which are read in
    place, one behind the other (or one for all groups: B.expand): with weights W
    stored groups x out x in, ``grouped_matmul(x,
    W.transpose(1, 2), offsets)`` is a layer's forward product and
    ``grouped_matmul(dy, W, offsets)`` the gradient of its input.  The result is
    of the operands' dtype or float32 (``dtype``, or that of ``out``).  Rows of no
    group are not written: a new result does not define them.  Operands have rows
    (and matrices) of a multiple of 16 bytes, or are contiguous (those of other
    widths are then copied to aligned ones first)."""
    if stream is not None and out is None:
        return _on_stream(stream,
                          lambda: grouped_matmul(A, B, offsets, None, dtype, alpha, beta))
    return (_group or _load_group()).grouped_matmul(A, B, offsets, out, dtype, alpha, beta, stream)


def grouped_grad(A, X, offsets, out=None, dtype=None, alpha=1.0, beta=0.0, stream=None):
    """out[g] = alpha * (A[rows of g].T @ X[rows of g]) + beta * out[g] for every
    group g (an empty one's product is zero), groups x M x N from A (rows x M)
    and X (rows x N), both row-major: ``grouped_grad(dy, x, offsets)`` is the
    gradient of weights stored groups x out x in.  Types, alignment and
    ``dtype`` as in grouped_matmul."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: grouped_grad(A, X, offsets, None, dtype, alpha, beta))
    return (_group or _load_group()).grouped_grad(A, X, offsets, out, dtype, alpha, beta, stream)


# ------------------------------------------------------------ 4-bit weights with group scales

class Q4Tensor:
    """Weights (out x in, or experts x out x in) held in 4 bits with a scale for
    each ``group`` of them along a row (a multiple of 32), as
    include/dense_gemm_q4.h describes:  value = scale * (code - zero).

    codes   uint8, (experts x) out x pitch, columns 2j and 2j + 1 in the low and
            high half of byte j; the pitch a multiple of 16 bytes, experts one
            behind the other
    scales  float16 or bfloat16, (experts x) out x ceil(cols / group)
    zeros   uint8 of the scales' shape, 0 .. 15; None: 8 for all
    cols    columns (default: two for each byte of codes)

    codes are kept as they are.  Scales and zeros are kept with the values of a
    group of columns together, as the kernels read them: copied once, here, unless
    they are transposed views of such arrays."""
    __slots__ = ("codes", "_scales", "_zeros", "experts", "rows", "cols", "group", "_ld")

    def __init__(self, codes, scales, zeros=None, cols=None, group=128):
        import torch
        if codes.dim() not in (2, 3) or codes.dtype != torch.uint8 or not codes.is_cuda:
            raise ValueError("codes must be a 2-D or 3-D uint8 CUDA tensor")
        lead, width = codes.shape[:-1], codes.shape[-1]
        cols = 2 * width if cols is None else int(cols)
        group = int(group)
        if group < 32 or group % 32 or group > 2 ** 31 - 32:
            raise ValueError("group must be a multiple of 32")
        if cols < 0 or (cols + 1) // 2 > width:
            raise ValueError("codes have fewer columns than cols")
        if codes.dim() == 3 and not 1 <= lead[0] <= 1024:
            raise ValueError("1 to 1024 experts")
        rows = lead[-1]
        ld = codes.stride(-2) if rows > 1 else -(-width // 16) * 16
        if codes.dim() == 3 and lead[0] > 1 and rows > 0:
            if rows == 1:
                ld = codes.stride(0)
            if codes.stride(0) != rows * ld:
                raise ValueError("experts' codes must follow one another")
        if (width > 1 and codes.stride(-1) != 1) or ld < (cols + 1) // 2:
            raise ValueError("codes' rows must be contiguous and not overlap")
        if ld % 16 or codes.data_ptr() % 16:
            raise ValueError("codes need 16-byte aligned rows")
        shape = (*lead, -(-cols // group))
        if (scales.dtype not in (torch.float16, torch.bfloat16) or tuple(scales.shape) != shape
                or scales.device != codes.device):
            raise ValueError(f"scales must be float16 or bfloat16 of shape {shape} on the codes' "
                             "device")
        if zeros is not None and (zeros.dtype != torch.uint8 or tuple(zeros.shape) != shape
                                  or zeros.device != codes.device):
            raise ValueError(f"zeros must be uint8 of shape {shape} on the codes' device")
        self.codes, self._scales = codes, scales.transpose(-1, -2).contiguous()
        self._zeros = None if zeros is None else zeros.transpose(-1, -2).contiguous()
        self.experts = lead[0] if codes.dim() == 3 else 0
        self.rows, self.cols, self.group, self._ld = rows, cols, group, ld

    @property
    def shape(self):
        return (*self.codes.shape[:-1], self.cols)

    @property
    def scales(self):
        return self._scales.transpose(-1, -2)

    @property
    def zeros(self):
        return None if self._zeros is None else self._zeros.transpose(-1, -2)

    @property
    def device(self):
        return self.codes.device

    def record_stream(self, stream):
        """Tensor.record_stream of the codes, scales and zeros."""
        for t in (self.codes, self._scales, self._zeros):
            if t is not None:
                t.record_stream(stream)


def q4_linear(x, W, offsets=None, out=None, stream=None):
    """x @ W.T with x (rows x in; float16 or bfloat16, row-major) and W a Q4Tensor
    whose scales have x's dtype, which the result has too.  Weights of experts
    take ``offsets``, as grouped_matmul does: the rows of expert g are multiplied
    with its matrix, and rows of no expert are not written.  x has rows of a
    multiple of 16 bytes, or is contiguous (copied to aligned rows first).  For more
    than 8 to 16 rows (8 for each expert) the weights are rounded to x's dtype first:
    a row's result depends that much on how many rows there are, and float16 weights
    beyond 65504 become infinite."""
    if stream is not None and out is None:
        return _on_stream(stream, lambda: q4_linear(x, W, offsets))
    return (_group or _load_group()).q4_linear(x, W, offsets, out, stream)
