"""Python binding of the GB300 BF16 TN GEMM library (libgemm_tn.so).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI declared in ``include/gemm_tn.h``.  There is no CPU
fallback — if the library is missing, every call raises.

Raw entry points take integers (device pointers, a ``cudaStream_t`` handle):

    gemm_bf16_tn(M, N, K, A, lda, B, ldb, C, ldc, D, ldd, alpha, beta, out_dtype, stream)

``gemm()`` is a convenience wrapper over torch tensors (torch supplies device
memory and the current stream).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgemm_tn.so")

OUT_BF16 = 0
OUT_F32 = 1

PATH_AUTO, PATH_1SM, PATH_2SM, PATH_SKINNY = 0, 1, 2, 3

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = -1
GEMM_ERR_MISALIGNED = -2
GEMM_ERR_UNSUPPORTED_DEVICE = -3
GEMM_ERR_LAUNCH = -4
GEMM_ERR_TIMEOUT = -5
GEMM_ERR_NOT_IMPLEMENTED = -6
GEMM_ERR_OUT_OF_MEMORY = -7
GEMM_ERR_CUDA = -8

EXPORTED = ["gemm_bf16_tn", "gemm_bf16_tn_ex", "gemm_get_status", "gemm_get_status_detail",
            "gemm_last_error_string", "gemm_last_launch_info", "gemm_shutdown", "gemm_version",
            "gemm_bf16_tn_skinny_noalloc", "gemm_bf16_tn_bias_act", "gemm_fp8_tn", "gemm_fp8_tn_ex",
            "gemm_bf16_tn_grouped", "gemm_bf16_tn_batched", "gemm_plan", "gemm_stream_read",
            "gemm_mma_rate", "gemm_fp8_tn_bias_act", "gemm_expert_dispatch", "gemm_expert_dispatch_backward",
            "gemm_expert_combine", "gemm_expert_combine_backward", "gemm_w4_tn", "gemm_w4_tn_experts",
            "gemm_bf16_tn_experts", "gemm_bf16_tn_experts_backward_a", "gemm_bf16_tn_experts_backward_w",
            "gemm_experts_config", "gemm_grad_workspace", "gemm_grad_norm", "gemm_clip_grad_norm"]

FP8_E4M3, FP8_E5M2 = 0, 1
SCHED_DEFAULT, SCHED_STATIC, SCHED_CLC = 0, 1, 2

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = 0, 1, 2, 3, 4


class GemmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"gemm error {code}: {msg}")
        self.code = code


class GemmConfig(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("grid", ctypes.c_int), ("raster_group", ctypes.c_int),
                ("skinny_grid", ctypes.c_int), ("wait_timeout_ns", ctypes.c_uint64),
                ("test_fault", ctypes.c_int), ("disable_pdl", ctypes.c_int),
                ("skinny_skew_kb", ctypes.c_int), ("scheduler", ctypes.c_int), ("skinny_bm", ctypes.c_int),
                ("skinny_kgroup", ctypes.c_int), ("tiled_k_parts", ctypes.c_int), ("l2_hints", ctypes.c_int),
                ("cluster_pref", ctypes.c_int), ("b_static", ctypes.c_int), ("skinny_pair", ctypes.c_int),
                ("tail_slices", ctypes.c_int)]


class GemmPlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("skinny_kgroup", ctypes.c_int), ("skinny_stages", ctypes.c_int), ("skinny_grid", ctypes.c_int),
                ("k_parts", ctypes.c_int), ("skinny_skew", ctypes.c_int), ("tail_slices", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class GemmProblem(ctypes.Structure):
    """One problem of gemm_bf16_tn_grouped (device pointers as integers)."""
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("A", ctypes.c_void_p), ("lda", ctypes.c_int64), ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64),
                ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("D", ctypes.c_void_p), ("ldd", ctypes.c_int64)]


class LaunchInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("grid", ctypes.c_int), ("cluster", ctypes.c_int),
                ("block", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("stages", ctypes.c_int), ("smem_bytes", ctypes.c_int), ("kernel", ctypes.c_char_p),
                ("scheduler", ctypes.c_int), ("k_parts", ctypes.c_int), ("cluster_pref", ctypes.c_int),
                ("tail_slices", ctypes.c_int)]

    def as_dict(self):
        return {f: (getattr(self, f).decode() if f == "kernel" and getattr(self, f) else getattr(self, f))
                for f, _ in self._fields_}


class ExpertPlanInfo(ctypes.Structure):
    """gemm_expert_plan: sizes and device pointers of a dispatch plan."""
    _fields_ = [("tokens", ctypes.c_int64), ("slots", ctypes.c_int), ("experts", ctypes.c_int),
                ("offsets", ctypes.c_void_p), ("slot_row", ctypes.c_void_p), ("row_token", ctypes.c_void_p)]


class W4MatrixInfo(ctypes.Structure):
    """gemm_w4_matrix: sizes and device pointers of 4-bit weight matrices."""
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("count", ctypes.c_int64),
                ("group", ctypes.c_int), ("scales_dtype", ctypes.c_int),
                ("codes", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("stride_codes", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("lds", ctypes.c_int64), ("stride_scales", ctypes.c_int64),
                ("zeros", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("stride_zeros", ctypes.c_int64)]


class TensorInfo(ctypes.Structure):
    """gemm_tensor: a dense tensor of gemm_grad_norm and gemm_clip_grad_norm."""
    _fields_ = [("data", ctypes.c_void_p), ("count", ctypes.c_int64), ("dtype", ctypes.c_int)]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m tensor_core_dense_tn_gb300.build`")
        lib = ctypes.CDLL(path)
        i64, vp, f32, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_float, ctypes.c_int
        args = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, f32, f32, i32, vp]
        lib.gemm_bf16_tn.argtypes = args
        lib.gemm_bf16_tn.restype = i32
        lib.gemm_fp8_tn.argtypes = [i64, i64, i64, vp, i64, vp, i64, i32, f32, f32, vp, i64, vp, i64,
                                    f32, f32, i32, vp]
        lib.gemm_fp8_tn.restype = i32
        lib.gemm_fp8_tn_bias_act.argtypes = lib.gemm_fp8_tn.argtypes[:-1] + [vp, i32, i32, vp]
        lib.gemm_fp8_tn_bias_act.restype = i32
        lib.gemm_fp8_tn_ex.argtypes = lib.gemm_fp8_tn.argtypes + [ctypes.POINTER(GemmConfig)]
        lib.gemm_fp8_tn_ex.restype = i32
        lib.gemm_plan.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(GemmConfig), ctypes.POINTER(GemmPlanInfo)]
        lib.gemm_plan.restype = i32
        lib.gemm_bf16_tn_bias_act.argtypes = args[:-1] + [vp, i32, i32, vp]
        lib.gemm_bf16_tn_bias_act.restype = i32
        lib.gemm_bf16_tn_skinny_noalloc.argtypes = args
        lib.gemm_bf16_tn_skinny_noalloc.restype = i32
        lib.gemm_stream_read.argtypes = [vp, i64, i64, i32, i32, i32, vp]
        lib.gemm_stream_read.restype = i32
        lib.gemm_mma_rate.argtypes = [i32, i32, i32, i32, i32, vp, vp]
        lib.gemm_mma_rate.restype = i32
        lib.gemm_bf16_tn_grouped.argtypes = [i32, ctypes.POINTER(GemmProblem), f32, f32, i32, vp]
        lib.gemm_bf16_tn_grouped.restype = i32
        lib.gemm_bf16_tn_batched.argtypes = [i64, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64,
                                             vp, i64, i64, f32, f32, i32, vp]
        lib.gemm_bf16_tn_batched.restype = i32
        lib.gemm_bf16_tn_ex.argtypes = args + [ctypes.POINTER(GemmConfig)]
        lib.gemm_bf16_tn_ex.restype = i32
        plan, w4 = ctypes.POINTER(ExpertPlanInfo), ctypes.POINTER(W4MatrixInfo)
        lib.gemm_expert_dispatch.argtypes = [plan, vp, i64, i32, i64, vp, i64, i32, vp, i64, vp]
        lib.gemm_expert_dispatch.restype = i32
        lib.gemm_expert_dispatch_backward.argtypes = [plan, i64, vp, i64, i32, vp, i64, vp]
        lib.gemm_expert_dispatch_backward.restype = i32
        lib.gemm_expert_combine.argtypes = [plan, i64, vp, i64, i32, vp, i64, i32, vp, i64, vp]
        lib.gemm_expert_combine.restype = i32
        lib.gemm_expert_combine_backward.argtypes = [plan, i64, vp, i64, vp, i64, i32, vp, i64, i32, vp, i64, vp, i64,
                                                     vp]
        lib.gemm_expert_combine_backward.restype = i32
        lib.gemm_w4_tn.argtypes = [i64, vp, i64, w4, vp, i64, f32, i32, i32, vp]
        lib.gemm_w4_tn.restype = i32
        lib.gemm_w4_tn_experts.argtypes = [plan, vp, i64, i32, w4, vp, i64, f32, i32, i32, vp]
        lib.gemm_w4_tn_experts.restype = i32
        lib.gemm_bf16_tn_experts.argtypes = [plan, i64, i64, vp, i64, vp, i64, i64, vp, i64, f32, i32, i32, vp]
        lib.gemm_bf16_tn_experts.restype = i32
        lib.gemm_bf16_tn_experts_backward_a.argtypes = [plan, i64, i64, vp, i64, vp, i64, i64, vp, i64, f32, i32, vp]
        lib.gemm_bf16_tn_experts_backward_a.restype = i32
        lib.gemm_bf16_tn_experts_backward_w.argtypes = [plan, i64, i64, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64,
                                                        f32, f32, i32, vp]
        lib.gemm_bf16_tn_experts_backward_w.restype = i32
        lib.gemm_experts_config.argtypes = [ctypes.POINTER(GemmConfig)]
        lib.gemm_experts_config.restype = i32
        lib.gemm_grad_workspace.argtypes = [i32]
        lib.gemm_grad_workspace.restype = i64
        lib.gemm_grad_norm.argtypes = [i32, vp, vp, vp, vp]
        lib.gemm_grad_norm.restype = i32
        lib.gemm_clip_grad_norm.argtypes = [i32, vp, f32, vp, vp, vp, vp]
        lib.gemm_clip_grad_norm.restype = i32
        lib.gemm_get_status.argtypes = [vp]
        lib.gemm_get_status.restype = i32
        lib.gemm_get_status_detail.restype = i32
        lib.gemm_last_error_string.restype = ctypes.c_char_p
        lib.gemm_last_launch_info.argtypes = [ctypes.POINTER(LaunchInfo)]
        lib.gemm_last_launch_info.restype = i32
        lib.gemm_shutdown.restype = None
        lib.gemm_version.restype = i32
        _lib = lib
        return lib


def last_error() -> str:
    s = load().gemm_last_error_string()
    return s.decode() if s else ""


def _check(rc: int) -> int:
    if rc != GEMM_OK:
        raise GemmError(rc, last_error())
    return rc


def gemm_bf16_tn(M, N, K, A, lda, B, ldb, C, ldc, D, ldd, alpha, beta, out_dtype, stream) -> int:
    """Raw C-ABI call; returns the gemm_status code (does not raise)."""
    return load().gemm_bf16_tn(M, N, K, A, lda, B, ldb, C or None, ldc, D, ldd, alpha, beta,
                               out_dtype, stream or None)


def gemm_bf16_tn_ex(M, N, K, A, lda, B, ldb, C, ldc, D, ldd, alpha, beta, out_dtype, stream,
                    config: GemmConfig | None = None) -> int:
    cfg = ctypes.byref(config) if config is not None else None
    return load().gemm_bf16_tn_ex(M, N, K, A, lda, B, ldb, C or None, ldc, D, ldd, alpha, beta,
                                  out_dtype, stream or None, cfg)


def gemm_bf16_tn_skinny_noalloc(M, N, K, A, lda, B, ldb, C, ldc, D, ldd, alpha, beta, out_dtype,
                                stream) -> int:
    """Raw C-ABI call of the allocation-free skinny entry point (1 <= M <= 64)."""
    return load().gemm_bf16_tn_skinny_noalloc(M, N, K, A, lda, B, ldb, C or None, ldc, D, ldd, alpha,
                                              beta, out_dtype, stream or None)


def gemm_stream_read(src, rows, row_bytes, box_rows, kgroup, grid, stream) -> int:
    """Raw C-ABI call of the TMA streaming-read ceiling kernel (reads rows x
    row_bytes bytes at src in the skinny kernel's box shape, discards them)."""
    return load().gemm_stream_read(src, rows, row_bytes, box_rows, kgroup, grid, stream or None)


def gemm_mma_rate(n, cta_group, fp8, reps, grid, out_ns, stream) -> int:
    """Raw C-ABI call of the tcgen05.mma rate kernel (out_ns: device pointer to two uint64)."""
    return load().gemm_mma_rate(n, cta_group, fp8, reps, grid, out_ns, stream or None)


def gemm_bf16_tn_grouped(problems, alpha, beta, out_dtype, stream) -> int:
    """Raw C-ABI call: `problems` is a sequence of GemmProblem (or of dicts with its fields)."""
    arr = (GemmProblem * max(1, len(problems)))()
    for i, q in enumerate(problems):
        arr[i] = q if isinstance(q, GemmProblem) else GemmProblem(**q)
    return load().gemm_bf16_tn_grouped(len(problems), arr, alpha, beta, out_dtype, stream or None)


def gemm_bf16_tn_batched(batch, M, N, K, A, lda, stride_a, B, ldb, stride_b, C, ldc, stride_c, D, ldd, stride_d,
                         alpha, beta, out_dtype, stream) -> int:
    """Raw C-ABI call of the strided batched GEMM (strides in elements)."""
    return load().gemm_bf16_tn_batched(batch, M, N, K, A, lda, stride_a, B, ldb, stride_b, C or None, ldc,
                                       stride_c, D, ldd, stride_d, alpha, beta, out_dtype, stream or None)


def gemm_bf16_tn_bias_act(M, N, K, A, lda, B, ldb, C, ldc, D, ldd, alpha, beta, out_dtype, bias,
                          bias_dtype, activation, stream) -> int:
    """Raw C-ABI call: D = act(alpha * A B^T + beta * C + bias)."""
    return load().gemm_bf16_tn_bias_act(M, N, K, A, lda, B, ldb, C or None, ldc, D, ldd, alpha, beta,
                                        out_dtype, bias or None, bias_dtype, activation, stream or None)


def gemm_fp8_tn_bias_act(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C, ldc, D, ldd, alpha, beta,
                         out_dtype, bias, bias_dtype, activation, stream) -> int:
    """Raw C-ABI call: D = act(alpha * scale_a * scale_b * A B^T + beta * C + bias), fp8 A and B."""
    return load().gemm_fp8_tn_bias_act(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C or None, ldc, D,
                                       ldd, alpha, beta, out_dtype, bias or None, bias_dtype, activation,
                                       stream or None)


def gemm_fp8_tn(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C, ldc, D, ldd, alpha, beta,
                out_dtype, stream) -> int:
    """Raw C-ABI call: D = alpha * scale_a * scale_b * A B^T + beta * C, fp8 A and B."""
    return load().gemm_fp8_tn(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C or None, ldc, D,
                              ldd, alpha, beta, out_dtype, stream or None)


def gemm_fp8_tn_ex(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C, ldc, D, ldd, alpha, beta,
                   out_dtype, stream, config=None) -> int:
    """gemm_fp8_tn with a GemmConfig of overrides (None = library defaults)."""
    cfg = ctypes.byref(config) if config is not None else None
    return load().gemm_fp8_tn_ex(M, N, K, A, lda, B, ldb, fp8_format, scale_a, scale_b, C or None, ldc, D,
                                 ldd, alpha, beta, out_dtype, stream or None, cfg)


def gemm_plan(M, N, K, fp8_inputs=0, num_sms=152, config=None):
    """Host-only plan of a call: (status, dict of GemmPlanInfo fields)."""
    out = GemmPlanInfo()
    cfg = ctypes.byref(config) if config is not None else None
    rc = load().gemm_plan(M, N, K, fp8_inputs, num_sms, cfg, ctypes.byref(out))
    return rc, out.as_dict()


def gemm_get_status(stream=None) -> int:
    return load().gemm_get_status(stream or None)


def gemm_get_status_detail() -> int:
    return load().gemm_get_status_detail()


def last_launch_info() -> dict:
    info = LaunchInfo()
    load().gemm_last_launch_info(ctypes.byref(info))
    return info.as_dict()


def shutdown() -> None:
    load().gemm_shutdown()


def version() -> int:
    return load().gemm_version()


def gemm(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, out_dtype=None, out=None,
         config: GemmConfig | None = None, stream=None):
    """D = alpha * A @ B.T + beta * C on the current CUDA stream (torch tensors).

    A: (M, K) bf16, B: (N, K) bf16, both with unit stride along K.
    C/out: (M, N) of out_dtype (torch.bfloat16 default, or torch.float32).
    """
    import torch

    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("out_dtype must be torch.bfloat16 or torch.float32")
    for name, t in (("A", A), ("B", B)):
        if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda or t.stride(1) != 1:
            raise ValueError(f"{name} must be a 2-D bf16 CUDA tensor with unit stride along K")
    M, K = A.shape
    N, Kb = B.shape
    if Kb != K:
        raise ValueError("A and B must have the same K")
    given = out
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    if out.shape != (M, N) or out.dtype != out_dtype or out.stride(1) != 1:
        raise ValueError("out must be (M, N), out_dtype, unit column stride")
    c_ptr, ldc = 0, 0
    if beta != 0.0:
        if C is None or C.shape != (M, N) or C.dtype != out_dtype or C.stride(1) != 1:
            raise ValueError("beta != 0 needs C of shape (M, N) and out_dtype")
        c_ptr, ldc = C.data_ptr(), C.stride(0)
    if stream is None:
        stream = torch.cuda.current_stream(A.device).cuda_stream
    code = OUT_F32 if out_dtype == torch.float32 else OUT_BF16
    args = (M, N, K, A.data_ptr(), A.stride(0), B.data_ptr(), B.stride(0), c_ptr, ldc,
            out.data_ptr(), out.stride(0), float(alpha), float(beta), code, stream)
    rc = gemm_bf16_tn_ex(*args, config=config) if config is not None else gemm_bf16_tn(*args)
    _check(rc)
    if given is not None:
        _t()
        _written((given,))
    return out


def gemm_expert_dispatch(plan, ids, ld_ids, ids_64bit, H, X, ldx, dtype, Xs, ldxs, stream) -> int:
    """Raw C-ABI call (plan: ExpertPlanInfo); returns the gemm_status code."""
    return load().gemm_expert_dispatch(plan, ids or None, ld_ids, ids_64bit, H, X or None, ldx, dtype, Xs or None,
                                       ldxs, stream or None)


def gemm_expert_dispatch_backward(plan, H, dXs, lddxs, dtype, dX, lddx, stream) -> int:
    """Raw C-ABI call: dX[t] = sum_j dXs[slot_row[t, j]]."""
    return load().gemm_expert_dispatch_backward(plan, H, dXs or None, lddxs, dtype, dX or None, lddx, stream or None)


def gemm_expert_combine(plan, H, Y, ldy, dtype, weights, ldw, weights_dtype, out, ldo, stream) -> int:
    """Raw C-ABI call: out[t] = sum_j weights[t, j] * Y[slot_row[t, j]]."""
    return load().gemm_expert_combine(plan, H, Y or None, ldy, dtype, weights or None, ldw, weights_dtype,
                                      out or None, ldo, stream or None)


def gemm_expert_combine_backward(plan, H, Y, ldy, dout, lddo, dtype, weights, ldw, weights_dtype, dY, lddy,
                                 dweights, lddw, stream) -> int:
    """Raw C-ABI call of the combine's gradients (dY or dweights may be 0)."""
    return load().gemm_expert_combine_backward(plan, H, Y or None, ldy, dout or None, lddo, dtype, weights or None,
                                               ldw, weights_dtype, dY or None, lddy, dweights or None, lddw,
                                               stream or None)


def gemm_w4_tn(M, A, lda, W, D, ldd, alpha, out_dtype, activation, stream) -> int:
    """Raw C-ABI call (W: W4MatrixInfo): D = act(alpha * A * W^T)."""
    return load().gemm_w4_tn(M, A or None, lda, W, D or None, ldd, alpha, out_dtype, activation, stream or None)


def gemm_w4_tn_experts(plan, A, lda, gather, W, D, ldd, alpha, out_dtype, activation, stream) -> int:
    """Raw C-ABI call: gemm_w4_tn with each expert's matrix for its rows of the plan."""
    return load().gemm_w4_tn_experts(plan, A or None, lda, gather, W, D or None, ldd, alpha, out_dtype, activation,
                                     stream or None)


def gemm_bf16_tn_experts(plan, N, K, A, lda, W, ldw, stride_w, D, ldd, alpha, out_dtype, activation, stream) -> int:
    """Raw C-ABI call: D[r] = act(alpha * A[r] * W_e^T) for the rows r of expert e."""
    return load().gemm_bf16_tn_experts(plan, N, K, A or None, lda, W or None, ldw, stride_w, D or None, ldd, alpha,
                                       out_dtype, activation, stream or None)


def gemm_bf16_tn_experts_backward_a(plan, N, K, dD, lddd, W, ldw, stride_w, dA, ldda, alpha, out_dtype, stream) -> int:
    """Raw C-ABI call: dA[r] = alpha * dD[r] * W_e."""
    return load().gemm_bf16_tn_experts_backward_a(plan, N, K, dD or None, lddd, W or None, ldw, stride_w, dA or None,
                                                  ldda, alpha, out_dtype, stream or None)


def gemm_bf16_tn_experts_backward_w(plan, N, K, dD, lddd, A, lda, C, ldc, stride_c, dW, lddw, stride_dw, alpha, beta,
                                    out_dtype, stream) -> int:
    """Raw C-ABI call: dW_e = alpha * dD_e^T * A_e + beta * C_e."""
    return load().gemm_bf16_tn_experts_backward_w(plan, N, K, dD or None, lddd, A or None, lda, C or None, ldc, stride_c,
                                                  dW or None, lddw, stride_dw, alpha, beta, out_dtype, stream or None)


def gemm_experts_config(config=None) -> int:
    """Raw C-ABI call: wait_timeout_ns and test_fault of a GemmConfig for this thread's products by expert from now on
    (None: the defaults)."""
    return load().gemm_experts_config(ctypes.byref(config) if config is not None else None)


def gemm_grad_workspace(num) -> int:
    """Bytes of workspace for gemm_grad_norm and gemm_clip_grad_norm of `num` tensors."""
    return load().gemm_grad_workspace(num)


def gemm_grad_norm(num, tensors, norm, workspace, stream) -> int:
    """Raw C-ABI call (tensors: an array of TensorInfo)."""
    return load().gemm_grad_norm(num, tensors, norm or None, workspace or None, stream or None)


def gemm_clip_grad_norm(num, tensors, max_norm, out, norm, workspace, stream) -> int:
    """Raw C-ABI call (tensors, out: arrays of TensorInfo; out None: in place)."""
    return load().gemm_clip_grad_norm(num, tensors, max_norm, out, norm or None, workspace or None, stream or None)


_torch = None
_several_gpus = True
_CODES = {}         # torch type -> gemm_out_dtype, filled with _torch


def _t():
    """The torch module, imported by the first wrapper that needs it."""
    global _torch, _several_gpus
    if _torch is None:
        import torch
        _several_gpus = torch.cuda.device_count() > 1
        _CODES.update({torch.bfloat16: OUT_BF16, torch.float32: OUT_F32})
        _torch = torch
    return _torch


def _written(tensors):
    """Counts a call's writes into tensors that the caller gave as in-place changes of them, as autograd expects
    (torch.autograd.graph.increment_version, in half its time; tensors of inference mode, which have no version, are
    left alone)."""
    _torch._C._increment_version(tensors)


def _out_code(dtype, what):
    _torch or _t()
    code = _CODES.get(dtype)
    if code is None:
        raise ValueError(f"{what} must be torch.bfloat16 or torch.float32, not {dtype}")
    return code


def _gpu_of(index, what):
    """Checks that `what`, on the GPU `index` (-1: host memory), is where the library launches.
    Callers skip it for GPU 0 where there is no other: it takes half a microsecond of a decode step's call."""
    if index < 0:
        raise ValueError(f"{what} must be in GPU memory")
    if index != _torch.cuda.current_device():
        raise ValueError(f"{what} is on GPU {index}, but calls go to the current GPU, {_torch.cuda.current_device()}")


def _rows_of(t, rows, width, what, gpu):
    """Checks a (rows, width) matrix on `gpu` with unit column stride and rows that do not overlap; returns its
    row stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or (width is not None and shape[1] != width) or t.get_device() != gpu:
        raise ValueError(f"{what} must be a matrix of {rows} x {'H' if width is None else width} on GPU {gpu}, "
                         f"not {tuple(shape)} on {t.device}")
    ld, wide = stride[0], shape[1]
    if stride[1] != 1 and wide > 1 and rows > 0:
        raise ValueError(f"{what} must have unit column stride")
    if ld < wide:
        if rows > 1:        # a broadcast row, or rows that overlap
            raise ValueError(f"{what} must have a row stride of at least its row length {wide}, not {ld} "
                             "(contiguous() makes a copy that has)")
        ld = wide           # a single row's stride says nothing
    return ld


def _stream_of(t):
    """The current stream of t's device, as an integer (torch.cuda.current_stream() makes an object first,
    several microseconds that a decode step's calls would each wait for)."""
    return _torch._C._cuda_getCurrentRawStream(t.get_device()) or None


class ExpertPlan:
    """A dispatch plan: int32 CUDA tensors offsets (E + 1), slot_row (T, k) and
    row_token (T * k), filled by expert_dispatch() and read by the other calls.
    A serving program keeps one per shape and fills it again at every step; for
    training every layer of every step needs its own until its gradients are
    taken, which read the same arrays.  Filling a plan counts as an in-place
    change of them, so a backward pass that saved them for autograd and finds
    them filled again raises."""

    def __init__(self, tokens: int, slots: int, experts: int, device):
        torch = _t()
        buf = torch.empty(experts + 1 + 2 * tokens * slots, dtype=torch.int32, device=device)
        n = tokens * slots
        self._set(buf[2 * n:], buf[:n].view(tokens, slots), buf[n:2 * n], experts)
        self._versioned = self._versioned[:1]       # views of one tensor share its version

    @classmethod
    def of(cls, offsets, slot_row, row_token, experts: int | None = None):
        """A plan over tensors that the caller filled."""
        plan = cls.__new__(cls)
        plan._set(offsets, slot_row, row_token, offsets.numel() - 1 if experts is None else experts)
        return plan

    def _set(self, offsets, slot_row, row_token, experts):
        torch = _t()
        for name, t in (("offsets", offsets), ("slot_row", slot_row), ("row_token", row_token)):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous int32 tensor")
        if slot_row.dim() != 2 or offsets.numel() != experts + 1 or row_token.numel() != slot_row.numel():
            raise ValueError("a plan has experts + 1 offsets, (tokens, slots) slot rows and tokens * slots row tokens")
        self.gpu = slot_row.get_device()        # -1 in host memory, where no call takes it
        if offsets.get_device() != self.gpu or row_token.get_device() != self.gpu:
            raise ValueError("the arrays of a plan must be on one device")
        self.offsets, self.slot_row, self.row_token = offsets, slot_row, row_token
        self._versioned = tuple(t for t in (offsets, slot_row, row_token) if not t.is_inference())
        self.tokens, self.slots = slot_row.shape
        self.experts, self.rows = experts, slot_row.numel()
        self.info = ExpertPlanInfo(self.tokens, self.slots, experts, offsets.data_ptr(), slot_row.data_ptr(),
                                   row_token.data_ptr())


class W4Matrix:
    """4-bit weights as gemm_w4() and gemm_w4_experts() take them.

    codes: uint8 CUDA tensor (N, bytes) or (E, N, bytes), two codes to a byte
    with the even k in the low half, rows of a multiple of 16 bytes.
    scales: bf16 or fp32 (.., N, ceil(K / group)); zeros: uint8 of that shape,
    or None for a zero point of 8.  W[n, k] = scales[n, k // group] *
    (q[n, k] - zeros[n, k // group])."""

    def __init__(self, codes, scales, zeros=None, K: int | None = None, group: int = 128):
        torch = _t()
        K = 2 * codes.shape[-1] if K is None else K
        if codes.dtype != torch.uint8 or codes.dim() not in (2, 3) or not codes.is_cuda or codes.stride(-1) != 1:
            raise ValueError("codes must be a 2-D or 3-D uint8 CUDA tensor with unit stride along K")
        if codes.shape[-1] * 2 < K:
            raise ValueError(f"codes hold {2 * codes.shape[-1]} values a row, fewer than K = {K}")
        want = tuple(codes.shape[:-1]) + (-(-K // group),)
        self.gpu = codes.get_device()
        for name, t in (("scales", scales), ("zeros", zeros)):
            if t is None:
                continue
            if tuple(t.shape) != want or t.get_device() != self.gpu or (t.stride(-1) != 1 and want[-1] > 1):
                raise ValueError(f"{name} must be a tensor of {want} on the codes' GPU with unit stride along the groups")
        if zeros is not None and zeros.dtype != torch.uint8:
            raise ValueError("zeros must be uint8")
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group
        self.N, self.K, self.count = codes.shape[-2], K, codes.shape[0] if codes.dim() == 3 else 1
        strides = lambda t: (0, 0) if t is None else (t.stride(-2), t.stride(0) if t.dim() == 3 else 0)  # noqa: E731
        (lc, sc), (ls, ss), (lz, sz) = strides(codes), strides(scales), strides(zeros)
        self.info = W4MatrixInfo(self.N, K, self.count, group, _out_code(scales.dtype, "scales"),
                                 codes.data_ptr(), 2 * lc, 2 * sc, scales.data_ptr(), ls, ss,
                                 0 if zeros is None else zeros.data_ptr(), lz, sz)


def expert_dispatch(ids, plan: ExpertPlan, X=None, out=None, stream=None):
    """Fills `plan` from ids (tokens, slots), int32 or int64 with ids outside
    [0, experts) dropped, and returns X's rows in expert order (None without X):
    Xs[plan.slot_row[t, j]] = X[t], zeros past plan.offsets[experts].  Like every
    call here it returns a tensor without an autograd graph; the gradient is
    expert_dispatch_backward()."""
    torch = _torch or _t()
    wide = ids.dtype == torch.int64
    if not wide and ids.dtype != torch.int32:
        raise ValueError("ids must be int32 or int64")
    gpu = plan.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "the plan")
    ld_ids = _rows_of(ids, plan.tokens, plan.slots, "ids", gpu)
    H, x, ldx, o, ldo, code = 0, None, 0, None, 0, OUT_BF16
    given = out if X is not None else None
    if X is not None:
        code, ldx = _out_code(X.dtype, "X"), _rows_of(X, plan.tokens, None, "X", gpu)
        H, x = X.shape[1], X.data_ptr()
        if out is None:
            out, ldo = torch.empty((plan.rows, H), dtype=X.dtype, device=X.device), H
        else:
            if out.dtype != X.dtype:
                raise ValueError("out must have X's type")
            ldo = _rows_of(out, plan.rows, H, "out", gpu)
        o = out.data_ptr()
    rc = (_lib or load()).gemm_expert_dispatch(plan.info, ids.data_ptr(), ld_ids, wide, H, x, ldx, code, o, ldo,
                                               _stream_of(ids) if stream is None else stream or None)
    if rc:
        _check(rc)
    torch._C._increment_version(plan._versioned)    # torch.autograd.graph.increment_version, in half its time
    if given is not None:
        _written((given,))
    return out if X is not None else None


def expert_dispatch_backward(plan: ExpertPlan, dXs, out=None, stream=None):
    """Gradient of expert_dispatch's copy: dX[t] = sum_j dXs[slot_row[t, j]]."""
    return _combine(plan, dXs, None, out, stream)


def expert_combine(plan: ExpertPlan, Y, weights, out=None, stream=None):
    """out[t] = sum_j weights[t, j] * Y[slot_row[t, j]] (weights: (tokens, slots) bf16 or fp32); without an
    autograd graph, the gradients are expert_combine_backward()."""
    return _combine(plan, Y, weights, out, stream)


def _combine(plan, Y, weights, out, stream):
    torch = _torch or _t()
    gpu = plan.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "the plan")
    code, ldy = _out_code(Y.dtype, "rows"), _rows_of(Y, plan.rows, None, "rows", gpu)
    H = Y.shape[1]
    if weights is not None:
        wcode, ldw = _out_code(weights.dtype, "weights"), _rows_of(weights, plan.tokens, plan.slots, "weights", gpu)
    given = out
    if out is None:
        out, ldo = torch.empty((plan.tokens, H), dtype=Y.dtype, device=Y.device), H
    else:
        if out.dtype != Y.dtype:
            raise ValueError("out must have the rows' type")
        ldo = _rows_of(out, plan.tokens, H, "out", gpu)
    lib, s = _lib or load(), _stream_of(Y) if stream is None else stream or None
    if weights is None:
        rc = lib.gemm_expert_dispatch_backward(plan.info, H, Y.data_ptr(), ldy, code, out.data_ptr(), ldo, s)
    else:
        rc = lib.gemm_expert_combine(plan.info, H, Y.data_ptr(), ldy, code, weights.data_ptr(), ldw, wcode,
                                     out.data_ptr(), ldo, s)
    if rc:
        _check(rc)
    if given is not None:
        _written((given,))
    return out


def expert_combine_backward(plan: ExpertPlan, Y, weights, dout, dY=None, dweights=None, stream=None):
    """Gradients of expert_combine: (dY, dweights), in Y's and weights' types."""
    torch = _torch or _t()
    gpu = plan.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "the plan")
    code, ldy = _out_code(Y.dtype, "Y"), _rows_of(Y, plan.rows, None, "Y", gpu)
    H = Y.shape[1]
    if dout.dtype != Y.dtype:
        raise ValueError("dout must have Y's type")
    lddo = _rows_of(dout, plan.tokens, H, "dout", gpu)
    wcode, ldw = _out_code(weights.dtype, "weights"), _rows_of(weights, plan.tokens, plan.slots, "weights", gpu)
    given = dY, dweights
    if dY is None:
        dY = torch.empty((plan.rows, H), dtype=Y.dtype, device=Y.device)
    if dweights is None:
        dweights = torch.empty((plan.tokens, plan.slots), dtype=weights.dtype, device=Y.device)
    if dY.dtype != Y.dtype or dweights.dtype != weights.dtype:
        raise ValueError("dY and dweights must have Y's and weights' types")
    rc = (_lib or load()).gemm_expert_combine_backward(
        plan.info, H, Y.data_ptr(), ldy, dout.data_ptr(), lddo, code, weights.data_ptr(), ldw, wcode, dY.data_ptr(),
        _rows_of(dY, plan.rows, H, "dY", gpu), dweights.data_ptr(),
        _rows_of(dweights, plan.tokens, plan.slots, "dweights", gpu), _stream_of(Y) if stream is None else stream or None)
    if rc:
        _check(rc)
    if given[0] is not None or given[1] is not None:
        _written([t for t in given if t is not None])
    return dY, dweights


def gemm_w4(A, W: W4Matrix, alpha: float = 1.0, activation: int = ACT_NONE, out_dtype=None, out=None, stream=None):
    """D = act(alpha * A @ W.T) for few tokens: A (M, K) bf16, W one matrix of 4-bit weights."""
    return _w4(None, A, W, False, alpha, activation, out_dtype, out, stream)


def gemm_w4_experts(A, W: W4Matrix, plan: ExpertPlan, gather: bool = False, alpha: float = 1.0,
                    activation: int = ACT_NONE, out_dtype=None, out=None, stream=None):
    """gemm_w4 for rows in expert order, W one matrix per expert; zeros in the rows past plan.offsets[experts].
    gather=False: A holds plan.rows rows in expert order; True: A holds the tokens, read through plan.row_token."""
    return _w4(plan, A, W, gather, alpha, activation, out_dtype, out, stream)


def _w4(plan, A, W, gather, alpha, activation, out_dtype, out, stream):
    torch = _torch or _t()
    if A.dtype != torch.bfloat16:
        raise ValueError("A must be bf16")
    gpu = W.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "W")
    if plan is not None and plan.gpu != gpu:
        raise ValueError("the plan and W must be on one GPU")
    rows = A.shape[0] if plan is None else plan.tokens if gather else plan.rows
    lda = _rows_of(A, rows, W.K, "A", gpu)
    M = rows if plan is None else plan.rows
    given = out
    if out is None:
        out, ldd = torch.empty((M, W.N), dtype=out_dtype or torch.bfloat16, device=A.device), W.N
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must have out_dtype")
        ldd = _rows_of(out, M, W.N, "out", gpu)
    code = _out_code(out.dtype, "out")
    lib, s = _lib or load(), _stream_of(A) if stream is None else stream or None
    if plan is None:
        rc = lib.gemm_w4_tn(M, A.data_ptr(), lda, W.info, out.data_ptr(), ldd, alpha, code, activation, s)
    else:
        rc = lib.gemm_w4_tn_experts(plan.info, A.data_ptr(), lda, gather, W.info, out.data_ptr(), ldd, alpha, code,
                                    activation, s)
    if rc:
        _check(rc)
    if given is not None:
        _written((given,))
    return out


def _matrices_of(t, count, N, K, what, gpu):
    """Checks `count` N x K matrices on `gpu` with unit column stride, none overlapping another; returns their row
    stride and the stride from one to the next."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape != (count, N, K) or t.get_device() != gpu:
        raise ValueError(f"{what} must be {count} matrices of {N} x {K} on GPU {gpu}, not {tuple(shape)} on {t.device}")
    apart, ld = stride[0], stride[1]
    if stride[2] != 1 and K > 1 and N > 0:
        raise ValueError(f"{what} must have unit column stride")
    if ld < K:
        if N > 1:
            raise ValueError(f"{what} must have a row stride of at least its row length {K}, not {ld}")
        ld = K
    if apart < N * ld:
        if count > 1:       # one matrix for all experts, or matrices that overlap
            raise ValueError(f"{what} must have a stride of at least {N * ld} from one expert's matrix to the next, not "
                             f"{apart} (contiguous() makes a copy that has)")
        apart = N * ld
    return ld, apart


def gemm_experts(A, W, plan: ExpertPlan, alpha: float = 1.0, activation: int = ACT_NONE, out_dtype=None, out=None,
                 stream=None):
    """D[r] = act(alpha * A[r] @ W[e].T) for the rows r of expert e in `plan`: A (plan.rows, K) bf16 in expert order,
    W (experts, N, K) bf16; zeros in the rows past plan.offsets[experts].  Nothing waits for the row counts.  Without
    an autograd graph: the gradients of the product without an activation are gemm_experts_backward_a() and _w().
    Rows of A and W start on 16 bytes, those of the result without `out` follow one another without gaps: where N is
    not a multiple of 8, the next product wants an `out` whose rows are N rounded up to 8 apart.
    Without `out` the result is the current stream's memory: a `stream` of the caller's waits for that one first."""
    return _experts_rows(False, A, W, plan, alpha, activation, out_dtype, out, stream)


def gemm_experts_backward_a(dD, W, plan: ExpertPlan, alpha: float = 1.0, out_dtype=None, out=None, stream=None):
    """Gradient of gemm_experts' rows: dA[r] = alpha * dD[r] @ W[e], zeros past plan.offsets[experts].  Rows of dD and W
    start on 16 bytes, as gemm_experts()' do."""
    return _experts_rows(True, dD, W, plan, alpha, ACT_NONE, out_dtype, out, stream)


def _experts_rows(backward, X, W, plan, alpha, activation, out_dtype, out, stream):
    torch = _torch or _t()
    if X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16 or W.dim() != 3:
        raise ValueError(f"{'dD' if backward else 'A'} and W must be bf16, W one matrix per expert")
    gpu = plan.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "the plan")
    _, N, K = W.shape
    ldw, apart = _matrices_of(W, plan.experts, N, K, "W", gpu)
    ldx = _rows_of(X, plan.rows, N if backward else K, "dD" if backward else "A", gpu)
    width = K if backward else N
    given = out
    if out is None:
        out, ldo = torch.empty((plan.rows, width), dtype=out_dtype or torch.bfloat16, device=X.device), width
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must have out_dtype")
        ldo = _rows_of(out, plan.rows, width, "out", gpu)
    code = _out_code(out.dtype, "out")
    lib, s = _lib or load(), _stream_of(X) if stream is None else stream or None
    if backward:
        rc = lib.gemm_bf16_tn_experts_backward_a(plan.info, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, apart,
                                                 out.data_ptr(), ldo, alpha, code, s)
    else:
        rc = lib.gemm_bf16_tn_experts(plan.info, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, apart, out.data_ptr(), ldo,
                                      alpha, code, activation, s)
    if rc:
        _check(rc)
    if given is not None:
        _written((given,))
    return out


def gemm_experts_backward_w(dD, A, plan: ExpertPlan, alpha: float = 1.0, beta: float = 0.0, C=None, out_dtype=None,
                            out=None, stream=None):
    """Gradients of gemm_experts' matrices: dW[e] = alpha * dD_e.T @ A_e (+ beta * C[e]) over e's rows of dD
    (plan.rows, N) and A (plan.rows, K), both bf16; (experts, N, K) of out_dtype, by default bf16.  C has out's type
    and may be out itself, to add to what it holds."""
    torch = _torch or _t()
    if dD.dtype != torch.bfloat16 or A.dtype != torch.bfloat16:
        raise ValueError("dD and A must be bf16")
    gpu = plan.gpu
    if gpu or _several_gpus:
        _gpu_of(gpu, "the plan")
    lddd, lda = _rows_of(dD, plan.rows, None, "dD", gpu), _rows_of(A, plan.rows, None, "A", gpu)
    N, K, E = dD.shape[1], A.shape[1], plan.experts
    given = out
    if out is None:
        dtype = out_dtype or (torch.bfloat16 if C is None or beta == 0.0 else C.dtype)
        out = torch.empty((E, N, K), dtype=dtype, device=A.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out must have out_dtype")
    code = _out_code(out.dtype, "out")
    ldo, apart = _matrices_of(out, E, N, K, "out", gpu)
    c, ldc, apart_c = None, 0, 0
    if beta != 0.0:
        if C is None or C.dtype != out.dtype:
            raise ValueError("beta != 0 needs C of out's type")
        ldc, apart_c = _matrices_of(C, E, N, K, "C", gpu)
        c = C.data_ptr()
    rc = (_lib or load()).gemm_bf16_tn_experts_backward_w(
        plan.info, N, K, dD.data_ptr(), lddd, A.data_ptr(), lda, c, ldc, apart_c, out.data_ptr(), ldo, apart, alpha,
        beta, code, _stream_of(A) if stream is None else stream or None)
    if rc:
        _check(rc)
    if given is not None:
        _written((given,))
    return out


def _dense(t):
    """Whether t's values fill their memory without gaps and none is there twice, in whatever order of dimensions."""
    step = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size != 1:
            if stride != step:
                return False
            step *= size
    return True


def _tensor_list(tensors, what):
    """gemm_tensor array (three 64-bit words each) of dense bf16 and fp32 tensors, as bytes, their counts, their GPU, and
    whether all are contiguous.  One pass per property and struct.pack: for a list of small gradients this is
    most of a call (a ctypes array filled from the words takes six times as long as the bytes)."""
    gpus = {t.get_device() for t in tensors}
    if len(gpus) > 1:
        raise ValueError(f"all {what} must be on one GPU")
    gpu = gpus.pop() if gpus else _torch.cuda.current_device()
    if gpu or _several_gpus:
        _gpu_of(gpu, f"{what}: a tensor")
    words = [0] * (3 * len(tensors))
    Tensor = _torch.Tensor
    words[0::3] = [*map(Tensor.data_ptr, tensors)]
    words[1::3] = counts = [*map(Tensor.numel, tensors)]
    words[2::3] = codes = [_CODES.get(t.dtype) for t in tensors]
    if None in codes:
        raise ValueError(f"{what} must be bf16 or fp32, not {tensors[codes.index(None)].dtype}")
    flat = all(map(Tensor.is_contiguous, tensors))
    if not flat:
        for i, t in enumerate(tensors):
            if t.numel() and not t.is_contiguous() and not _dense(t):
                raise ValueError(f"{what}: tensor {i} must be dense, not {tuple(t.shape)} with strides {t.stride()}")
    return struct.pack(f"={len(words)}q", *words), counts, gpu, flat


_GRAD_WORKSPACE = {}        # number of tensors -> bytes


def _norm_buffers(num, gpu, norm, stream):
    """The norm's tensor and the workspace.  With a stream of the caller's they come from that stream's memory: the
    workspace is given back when the call returns, and must neither be in use on the current stream still nor be used
    there while the kernels run on the other."""
    torch = _torch
    if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1 or norm.get_device() != gpu):
        raise ValueError(f"norm must be one fp32 on GPU {gpu}")
    nbytes = _GRAD_WORKSPACE.get(num) or _GRAD_WORKSPACE.setdefault(num, (_lib or load()).gemm_grad_workspace(num))
    if stream is not None:
        with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=gpu) if stream else torch.cuda.default_stream(gpu)):
            return _norm_buffers(num, gpu, norm, None)
    work = torch.empty(nbytes, dtype=torch.uint8, device=gpu)
    return torch.empty((), dtype=torch.float32, device=gpu) if norm is None else norm, work


def grad_norm(tensors, norm=None, stream=None):
    """sqrt of the sum of the squares of all values of `tensors` (dense bf16 and fp32 CUDA tensors, mixed), as an fp32
    tensor without dimensions, or in `norm`.  Nothing waits for the GPU."""
    _torch or _t()
    tensors = list(tensors)
    words, _, gpu, _ = _tensor_list(tensors, "tensors")
    given = norm
    norm, work = _norm_buffers(len(tensors), gpu, norm, stream)
    s = _torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream
    rc = (_lib or load()).gemm_grad_norm(len(tensors), words, norm.data_ptr(), work.data_ptr(), s or None)
    if rc:
        _check(rc)
    if given is not None:
        _written((given,))
    return norm


def clip_grad_norm(tensors, max_norm: float, out=None, norm=None, stream=None):
    """Multiplies all values by max_norm / norm where their norm (grad_norm()) is above max_norm, in place, or into the
    tensors `out` (bf16 or fp32, contiguous for contiguous tensors, else of their strides; also where nothing is
    scaled).  No tensor may be there twice or overlap another.  Returns the norm from
    before.  A norm that is not finite changes nothing.  In place, values within max_norm are not written; the
    tensors' versions count as changed all the same."""
    torch = _torch or _t()
    tensors = list(tensors)
    words, counts, gpu, flat = _tensor_list(tensors, "tensors")
    to = None
    if out is not None:
        out = list(out)
        to, counts_out, gpu_out, flat_out = _tensor_list(out, "out")
        if counts_out != counts:
            raise ValueError("out must have a tensor of the same size for each tensor")
        if gpu_out != gpu:
            raise ValueError("tensors and out must be on one GPU")
        if not (flat and flat_out):
            for i, (o, t) in enumerate(zip(out, tensors)):
                if t.numel() and not (o.is_contiguous() and t.is_contiguous()) and \
                        (o.shape != t.shape or o.stride() != t.stride()):
                    raise ValueError(f"out: tensor {i} must have its tensor's shape and order of dimensions")
    given = norm
    norm, work = _norm_buffers(len(tensors), gpu, norm, stream)
    s = torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream
    rc = (_lib or load()).gemm_clip_grad_norm(len(tensors), words, max_norm, to, norm.data_ptr(), work.data_ptr(),
                                               s or None)
    if rc:
        _check(rc)
    _written(tensors if out is None else out)
    if given is not None:
        _written((given,))
    return norm
