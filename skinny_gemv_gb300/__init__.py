"""Python binding of the GB300 bf16 GEMM / skinny-GEMV C library.

Argument marshalling only: every function here forwards device pointers, sizes
and the current CUDA stream to ``libskinny_gemm.so`` through ctypes; all of C is
computed by the library's sm_103a kernels.  PyTorch is used for device memory
and streams.  If the library has not been built the import of any compute
function raises -- there is no fallback.

    import torch, skinny_gemv_gb300 as sg
    C = sg.gemm_bf16(A, B)        # A [M, K], B [N, K] bf16 on cuda -> C [M, N] = A @ B.T
    C = sg.gemv_bf16(x, W)        # x [M <= 64, K]
"""
from __future__ import annotations

import ctypes
import os
import re

from . import _build

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "skinny_gemm.h")

SG_OK = 0
SG_ERR_INVALID_ARG = 1
SG_ERR_MISALIGNED = 2
SG_ERR_UNSUPPORTED_DEVICE = 3
SG_ERR_CUDA = 4
SG_ERR_TIMEOUT = 5
SG_ERR_OUT_OF_MEMORY = 6
SG_ERR_BAD_INDEX = 7

PATH_AUTO = 0
PATH_CUDA_CORE = 1
PATH_TENSOR_CORE = 2
PATH_GEMM = 3
PATH_GEMM_PAIR = 4
PATH_STREAM = 5  # attention_kv_nvfp4 only
PATH_NAMES = {PATH_AUTO: "auto", PATH_CUDA_CORE: "cuda_core", PATH_TENSOR_CORE: "tensor_core",
              PATH_GEMM: "gemm", PATH_GEMM_PAIR: "gemm_pair", PATH_STREAM: "stream"}


class SgError(RuntimeError):
    def __init__(self, status: int, where: str, lib=None):
        self.status = status
        msg = lib.sg_status_string(status).decode() if lib is not None else f"status {status}"
        if status == SG_ERR_CUDA and lib is not None:
            msg += f" (cudaError {lib.sg_last_cuda_error()})"
        super().__init__(f"{where}: {msg}")


class PlanInfo(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("tiles_m", ctypes.c_int32), ("tiles_n", ctypes.c_int32),
                ("k_steps", ctypes.c_int32), ("grid", ctypes.c_int32), ("dp_tiles", ctypes.c_int32),
                ("sk_tiles", ctypes.c_int32), ("sk_units", ctypes.c_int64), ("group_m", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("split_k", ctypes.c_int32), ("rows_per_cta", ctypes.c_int32),
                ("wave_efficiency", ctypes.c_double), ("cluster_size", ctypes.c_int32),
                ("ctas_per_sm", ctypes.c_int32), ("prefetch_steps", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class DeviceInfo(ctypes.Structure):
    _fields_ = [("sm_count", ctypes.c_int32), ("cc_major", ctypes.c_int32), ("cc_minor", ctypes.c_int32),
                ("smem_optin_bytes", ctypes.c_int32), ("l2_bytes", ctypes.c_int32),
                ("global_mem_bytes", ctypes.c_int64), ("clock_khz", ctypes.c_int32),
                ("mem_clock_khz", ctypes.c_int32), ("mem_bus_bits", ctypes.c_int32)]


_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False):
    """The loaded ctypes library.  Raises if it is not built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB_PATH):
        if not build_if_missing:
            raise RuntimeError(f"CUDA library not built: {_build.LIB_PATH} is missing; "
                               "run __graft_entry__.build() (nvcc, sm_103a)")
        _build.build()
    lib = ctypes.CDLL(_build.LIB_PATH)
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    for name in ("gemm_bf16", "gemv_bf16", "gemv_bf16_noalloc"):
        f = getattr(lib, name)
        f.argtypes = [p, p, p, i64, i64, i64, i64, i64, i64, p]
        f.restype = ctypes.c_int
    for name in ("gemv_bf16_path", "gemm_bf16_path"):
        f = getattr(lib, name)
        f.argtypes = [p, p, p, i64, i64, i64, i64, i64, i64, ctypes.c_int, p]
        f.restype = ctypes.c_int
    lib.gemm_bf16_swiglu.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, p]
    lib.gemm_bf16_swiglu.restype = ctypes.c_int
    lib.gemm_bf16_swiglu_path.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, ctypes.c_int, p]
    lib.gemm_bf16_swiglu_path.restype = ctypes.c_int
    lib.gemm_bf16_residual.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, i64, p]
    lib.gemm_bf16_residual.restype = ctypes.c_int
    lib.gemm_bf16_residual_path.argtypes = [p, p, p, p, i64, i64, i64, i64, i64, i64, i64, ctypes.c_int, p]
    lib.gemm_bf16_residual_path.restype = ctypes.c_int
    pp, p64 = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64)
    lib.gemv_bf16_batched.argtypes = [p, i64, i64, i64, pp, p64, p64, pp, p64, ctypes.c_int, ctypes.c_int, p]
    lib.gemv_bf16_batched.restype = ctypes.c_int
    lib.gemm_nvfp4.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i64, i64, ctypes.c_float, p]
    lib.gemm_nvfp4.restype = ctypes.c_int
    lib.nvfp4_scale_bytes.argtypes = [i64, i64]
    lib.nvfp4_scale_bytes.restype = i64
    lib.nvfp4_pack_scales.argtypes = [p, i64, i64, i64, p, p]
    lib.nvfp4_pack_scales.restype = ctypes.c_int
    lib.sg_plan_nvfp4.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.gemm_nvfp4_path.argtypes = [p, p, p, p, p, i64, i64, i64, i64, i64, i64, ctypes.c_float, ctypes.c_int, p]
    lib.gemm_nvfp4_path.restype = ctypes.c_int
    lib.attention_bf16.argtypes = [p, p, p, p] + [i64] * 10 + [ctypes.c_int, ctypes.c_float, p]
    lib.attention_bf16.restype = ctypes.c_int
    lib.attention_bf16_path.argtypes = [p, p, p, p] + [i64] * 10 + [ctypes.c_int, ctypes.c_float, ctypes.c_int, p]
    lib.attention_bf16_path.restype = ctypes.c_int
    lib.sg_plan_nvfp4.restype = ctypes.c_int
    f32, ci = ctypes.c_float, ctypes.c_int
    lib.kv_nvfp4_page_bytes.argtypes = [i64, i64]
    lib.kv_nvfp4_page_bytes.restype = i64
    lib.kv_pages_assign.argtypes = [p, p, i64, p, i64, p, p, i64, i64, i64, p, p, i64, p, p, p, p, p]
    lib.kv_pages_assign.restype = ci
    lib.qk_norm_rope_bf16.argtypes = [p, p, p, p] + [i64] * 8 + [p, p, f32, p, i64, i64, p, ci, p]
    lib.qk_norm_rope_bf16.restype = ci
    lib.kv_append_nvfp4.argtypes = [p, p] + [i64] * 5 + [p, i64, i64, i64, p, f32, f32, p]
    lib.kv_append_nvfp4.restype = ci
    lib.kv_read_nvfp4.argtypes = [p, i64, i64, i64, p, i64, i64, i64, p, p, i64, i64, f32, f32, p]
    lib.kv_read_nvfp4.restype = ci
    lib.attention_kv_nvfp4.argtypes = [p, p, p, p, i64, i64, p, p] + [i64] * 11 + [ci, f32, f32, f32, p]
    lib.attention_kv_nvfp4.restype = ci
    lib.attention_kv_nvfp4_path.argtypes = [p, p, p, p, i64, i64, p, p] + [i64] * 11 + [ci, f32, f32, f32, ci, p]
    lib.attention_kv_nvfp4_path.restype = ci
    lib.sg_status_string.argtypes = [ctypes.c_int]
    lib.sg_status_string.restype = ctypes.c_char_p
    lib.sg_last_cuda_error.argtypes = []
    lib.sg_last_cuda_error.restype = ctypes.c_int
    lib.sg_check_device_errors.argtypes = [p, ctypes.POINTER(ctypes.c_uint32)]
    lib.sg_check_device_errors.restype = ctypes.c_int
    lib.sg_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.sg_set_wait_timeout_ns.restype = None
    lib.sg_debug_inject_missing_tx.argtypes = [ctypes.c_uint32]
    lib.sg_debug_inject_missing_tx.restype = None
    lib.sg_plan.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.sg_plan.restype = ctypes.c_int
    lib.sg_plan_swiglu.argtypes = [i64, i64, i64, i32, i32, ctypes.POINTER(PlanInfo)]
    lib.sg_plan_swiglu.restype = ctypes.c_int
    lib.sg_plan_item.argtypes = [ctypes.POINTER(PlanInfo), i32, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.sg_plan_item.restype = ctypes.c_int
    lib.sg_wave_efficiency.argtypes = [i64, i64]
    lib.sg_wave_efficiency.restype = ctypes.c_double
    lib.sg_device_query.argtypes = [ctypes.POINTER(DeviceInfo)]
    lib.sg_device_query.restype = ctypes.c_int
    dp = ctypes.POINTER(ctypes.c_double)
    lib.sg_bench_tcgen05_peak.argtypes = [i64, dp, dp, p]
    lib.sg_bench_tcgen05_peak.restype = ctypes.c_int
    lib.sg_bench_copy.argtypes = [p, p, i64, i32, dp, p]
    lib.sg_bench_copy.restype = ctypes.c_int
    lib.sg_bench_read.argtypes = [p, i64, i32, p, dp, p]
    lib.sg_bench_read.restype = ctypes.c_int
    _lib = lib
    return lib


def declared_symbols() -> list[str]:
    """Function names declared in include/skinny_gemm.h."""
    text = open(HEADER).read()
    return re.findall(r"^SG_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)


def _check(status: int, where: str) -> None:
    if status != SG_OK:
        raise SgError(status, where, load())


# ------------------------------------------------------------------ raw pointers
def gemm_bf16_ptr(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                  stream: int = 0, path: int = PATH_AUTO) -> int:
    """C-ABI call with raw device pointers; returns the sg_status code."""
    return load().gemm_bf16_path(A, B, C, M, N, K, lda, ldb, ldc, path, stream)


def gemv_bf16_ptr(A: int, B: int, C: int, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                  stream: int = 0, path: int = PATH_AUTO) -> int:
    return load().gemv_bf16_path(A, B, C, M, N, K, lda, ldb, ldc, path, stream)


# ------------------------------------------------------------------ torch tensors
_torch_module = None  # imported on the first use of a tensor; its names below are set with it
_bf16 = _i32 = _u8 = _f32 = _get_device = _raw_stream = None


def _torch():
    global _torch_module, _bf16, _i32, _u8, _f32, _get_device, _raw_stream
    if _torch_module is None:
        import torch
        _bf16, _i32, _u8, _f32 = torch.bfloat16, torch.int32, torch.uint8, torch.float32
        # private names, 3 us a call cheaper; a torch without them takes the public ones
        _get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None) or
                       (lambda device: torch.cuda.current_stream(device).cuda_stream))
        _torch_module = torch
    return _torch_module


def _operand(t, name: str):
    torch = _torch()
    if t.dtype != torch.bfloat16 or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D bfloat16 CUDA tensor, got {t.dtype} {tuple(t.shape)} {t.device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), max(t.stride(0), t.shape[1])


def _stream_handle(stream) -> int:
    if stream is None:  # the current stream's handle, without the Stream object (3 us a call)
        _torch()
        return _raw_stream(_get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(fn_name: str, A, B, C=None, stream=None, path: int | None = None):
    torch = _torch()
    a_ptr, lda = _operand(A, "A")
    b_ptr, ldb = _operand(B, "B")
    M, K = A.shape
    N, Kb = B.shape
    if Kb != K:
        raise ValueError(f"K mismatch: A is {tuple(A.shape)}, B is {tuple(B.shape)}")
    if C is None:
        ld = -(-N // 8) * 8  # rows 16-byte aligned, as the library requires
        C = torch.empty((M, ld), dtype=torch.bfloat16, device=A.device)[:, :N]
    c_ptr, ldc = _operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    s = _stream_handle(stream)
    lib = load()
    with torch.cuda.device(A.device):
        if fn_name == "gemm_bf16":
            st = lib.gemm_bf16_path(a_ptr, b_ptr, c_ptr, M, N, K, lda, ldb, ldc,
                                    PATH_AUTO if path is None else path, s)
        elif fn_name == "gemv_bf16_noalloc":
            st = lib.gemv_bf16_noalloc(a_ptr, b_ptr, c_ptr, M, N, K, lda, ldb, ldc, s)
        else:
            st = lib.gemv_bf16_path(a_ptr, b_ptr, c_ptr, M, N, K, lda, ldb, ldc,
                                    PATH_AUTO if path is None else path, s)
    _check(st, fn_name)
    return C


def gemm_bf16(A, B, C=None, stream=None, path: int = PATH_AUTO):
    """C[M, N] = A[M, K] @ B[N, K]^T in bf16 with fp32 accumulation; ``path``
    picks the kernel (PATH_AUTO, PATH_GEMM, PATH_GEMM_PAIR, or a skinny PATH_*)."""
    return _call("gemm_bf16", A, B, C, stream, path)


def gemm_bf16_swiglu(A, Wg, Wu, C=None, stream=None, path: int = PATH_AUTO):
    """C[M, N] = silu(A @ Wg^T) * (A @ Wu^T) in one launch (fp32 accumulation and
    epilogue, bf16 out); Wg and Wu are [N, K] with one leading dimension."""
    torch = _torch()
    a_ptr, lda = _operand(A, "A")
    g_ptr, ldg = _operand(Wg, "Wg")
    u_ptr, ldu = _operand(Wu, "Wu")
    M, K = A.shape
    N = Wg.shape[0]
    if tuple(Wg.shape) != (N, K) or tuple(Wu.shape) != (N, K):
        raise ValueError(f"Wg and Wu must both be {(N, K)}: {tuple(Wg.shape)} {tuple(Wu.shape)}")
    if ldg != ldu:
        raise ValueError(f"Wg and Wu must share a leading dimension ({ldg} vs {ldu})")
    if C is None:
        ld = -(-N // 8) * 8
        C = torch.empty((M, ld), dtype=torch.bfloat16, device=A.device)[:, :N]
    c_ptr, ldc = _operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    with torch.cuda.device(A.device):
        st = load().gemm_bf16_swiglu_path(a_ptr, g_ptr, u_ptr, c_ptr, M, N, K, lda, ldg, ldc, path,
                                          _stream_handle(stream))
    _check(st, "gemm_bf16_swiglu")
    return C


def gemm_bf16_residual(A, B, R, C=None, stream=None, path: int = PATH_AUTO):
    """C[M, N] = A @ B^T + R with the sum in fp32 and one bf16 rounding; R may be C
    (in place)."""
    torch = _torch()
    a_ptr, lda = _operand(A, "A")
    b_ptr, ldb = _operand(B, "B")
    r_ptr, ldr = _operand(R, "R")
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(R.shape) != (M, N):
        raise ValueError(f"shapes: A {tuple(A.shape)}, B {tuple(B.shape)}, R {tuple(R.shape)}")
    if C is None:
        ld = -(-N // 8) * 8
        C = torch.empty((M, ld), dtype=torch.bfloat16, device=A.device)[:, :N]
    c_ptr, ldc = _operand(C, "C")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C must be {(M, N)}, got {tuple(C.shape)}")
    with torch.cuda.device(A.device):
        st = load().gemm_bf16_residual_path(a_ptr, b_ptr, r_ptr, c_ptr, M, N, K, lda, ldb, ldr, ldc, path,
                                            _stream_handle(stream))
    _check(st, "gemm_bf16_residual")
    return C


def _bytes_operand(t, name: str):
    torch = _torch()
    if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D uint8 CUDA tensor, got {t.dtype} {tuple(t.shape)} {t.device}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along its last dimension")
    return t.data_ptr(), max(t.stride(0), t.shape[1])


def nvfp4_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the scale-atom buffer gemm_nvfp4 reads for `rows` rows."""
    return int(load().nvfp4_scale_bytes(rows, K))


def nvfp4_pack_scales(plain, K: int | None = None, atoms=None, stream=None):
    """Plain row-major E4M3 scale codes (uint8 [rows, >= K/16]) to the scale atoms
    gemm_nvfp4 reads (a flat uint8 tensor); padding is written as 0."""
    torch = _torch()
    p_ptr, ld = _bytes_operand(plain, "plain")
    rows = plain.shape[0]
    K = 16 * plain.shape[1] if K is None else K
    n = nvfp4_scale_bytes(rows, K)
    if atoms is None:
        atoms = torch.empty(max(n, 1), dtype=torch.uint8, device=plain.device)
    if atoms.dtype != torch.uint8 or not atoms.is_cuda or atoms.numel() < n or not atoms.is_contiguous():
        raise ValueError(f"atoms must be a contiguous uint8 CUDA tensor of at least {n} bytes")
    with torch.cuda.device(plain.device):
        st = load().nvfp4_pack_scales(p_ptr, rows, K, ld, atoms.data_ptr(), _stream_handle(stream))
    _check(st, "nvfp4_pack_scales")
    return atoms


def gemm_nvfp4(A, SFA, B, SFB, K: int | None = None, C=None, alpha: float = 1.0, stream=None,
               path: int = PATH_AUTO):
    """C[M, N] (fp16) = alpha * (A . SFA) @ (B . SFB)^T for packed E2M1 operands
    (uint8 [M, >= K/2] and [N, >= K/2]) and their E4M3 scale atoms (from
    nvfp4_pack_scales)."""
    torch = _torch()
    a_ptr, lda = _bytes_operand(A, "A")
    b_ptr, ldb = _bytes_operand(B, "B")
    M, N = A.shape[0], B.shape[0]
    K = 2 * A.shape[1] if K is None else K
    if 2 * A.shape[1] < K or 2 * B.shape[1] < K:
        raise ValueError(f"K = {K} needs {K // 2} bytes per row: A {tuple(A.shape)}, B {tuple(B.shape)}")
    for t, rows, name in ((SFA, M, "SFA"), (SFB, N, "SFB")):
        if t.dtype != torch.uint8 or not t.is_cuda or t.numel() < nvfp4_scale_bytes(rows, K):
            raise ValueError(f"{name} must hold nvfp4_scale_bytes({rows}, {K}) uint8 scale-atom bytes")
    if C is None:
        ld = -(-N // 8) * 8
        C = torch.empty((M, ld), dtype=torch.float16, device=A.device)[:, :N]
    if C.dtype != torch.float16 or tuple(C.shape) != (M, N) or not C.is_cuda or (N > 1 and C.stride(1) != 1):
        raise ValueError(f"C must be a float16 CUDA tensor of shape {(M, N)}")
    ldc = max(C.stride(0), N)
    with torch.cuda.device(A.device):
        st = load().gemm_nvfp4_path(a_ptr, SFA.data_ptr(), b_ptr, SFB.data_ptr(), C.data_ptr(), M, N, K, lda, ldb,
                                    ldc, float(alpha), int(path), _stream_handle(stream))
    _check(st, "gemm_nvfp4_path")
    return C


def _tokens_heads(t, name: str):
    """A [B, S, heads, D] bfloat16 CUDA tensor whose (heads, D) block is dense:
    returns (pointer, token pitch in elements)."""
    torch = _torch()
    if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_cuda:
        raise ValueError(f"{name} must be a 4-D [batch, seq, heads, head_dim] bfloat16 CUDA tensor, "
                         f"got {t.dtype} {tuple(t.shape)} {t.device}")
    Bt, S, H, D = t.shape
    if (D > 1 and t.stride(3) != 1) or (H > 1 and t.stride(2) != D):
        raise ValueError(f"{name} must have dense heads x head_dim rows")
    # token row b * S + i at pitch ld; with one token per sequence the rows are
    # the batches (a size-1 dimension's stride says nothing about memory)
    if S > 1:
        ld = t.stride(1)
        if Bt > 1 and t.stride(0) != S * ld:
            raise ValueError(f"{name} must have batches of whole rows")
    elif Bt > 1:
        ld = t.stride(0)
    else:
        ld = H * D
    if ld < H * D:  # overlapping or broadcast rows: not a token-major layout
        raise ValueError(f"{name} token rows overlap (pitch {ld} < {H * D} elements)")
    return t.data_ptr(), ld


def attention_bf16(Q, K, V, O=None, causal: bool = False, scale: float | None = None, stream=None,
                   path: int = PATH_AUTO):
    """O = softmax(scale Q K^T, causal mask) V per head for Q [B, Sq, H, 128] and
    K, V [B, Sk, Hkv, 128] (bfloat16); returns O [B, Sq, H, 128].  ``path``:
    PATH_AUTO, PATH_TENSOR_CORE (the tcgen05 kernel) or PATH_CUDA_CORE (the
    decode kernel, Sq x H / Hkv <= 4)."""
    torch = _torch()
    q_ptr, ldq = _tokens_heads(Q, "Q")
    k_ptr, ldk = _tokens_heads(K, "K")
    v_ptr, ldv = _tokens_heads(V, "V")
    Bt, Sq, H, D = Q.shape
    Sk, Hkv = K.shape[1], K.shape[2]
    if tuple(K.shape) != (Bt, Sk, Hkv, D) or tuple(V.shape) != tuple(K.shape):
        raise ValueError(f"K and V must be [{Bt}, seq_k, kv_heads, {D}], got {tuple(K.shape)} and {tuple(V.shape)}")
    if O is None:
        O = torch.empty((Bt, Sq, H, D), dtype=torch.bfloat16, device=Q.device)
    if tuple(O.shape) != (Bt, Sq, H, D):
        raise ValueError(f"O must be [{Bt}, {Sq}, {H}, {D}]")
    o_ptr, ldo = _tokens_heads(O, "O")
    scale = D ** -0.5 if scale is None else float(scale)
    with torch.cuda.device(Q.device):
        st = load().attention_bf16_path(q_ptr, k_ptr, v_ptr, o_ptr, Bt, Sq, Sk, H, Hkv, D, ldq, ldk, ldv, ldo,
                                        1 if causal else 0, scale, path, _stream_handle(stream))
    _check(st, "attention_bf16_path")
    return O


# ------------------------------------------------------------------ paged NVFP4 KV cache
# These calls are short on the GPU (2 to 5 us for a decode step), so their checks read
# each tensor attribute once.  Every entry point calls _torch() first.
def _on_device(t, fn, args, stream, where: str) -> None:
    """fn(*args, stream handle) with t's device current; raises on a status."""
    if _get_device() == t.get_device():
        st = fn(*args, _raw_stream(t.get_device()) if stream is None else _stream_handle(stream))
    else:
        with _torch().cuda.device(t.device):
            st = fn(*args, _stream_handle(stream))
    if st != SG_OK:
        raise SgError(st, where, load())


def _int32s(t, name: str, size: int | None = None):
    if t.dtype is not _i32 or not t.is_cuda or t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 1-D int32 CUDA tensor, got {t.dtype} {tuple(t.shape)} {t.device}")
    if size is not None and t.numel() != size:
        raise ValueError(f"{name} must hold {size} values, got {t.numel()}")
    return t.data_ptr()


def _rows2d(t, name: str, dtype, what: str):
    """(pointer, rows, columns, pitch) of a 2-D CUDA tensor with unit stride along its columns."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or len(shape) != 2 or not t.is_cuda or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name} must be a 2-D {what} CUDA tensor with unit stride along its last dimension, got "
                         f"{t.dtype} {tuple(shape)} {t.device}")
    rows, cols = shape
    pitch = stride[0] if rows > 1 else cols
    if pitch < cols:
        raise ValueError(f"{name} rows overlap (pitch {pitch} < {cols})")
    return t.data_ptr(), rows, cols, pitch


def _block_table(t):
    return _rows2d(t, "block_table", _i32, "int32 [requests, pages]")


def _kv_cache(cache, kv_heads: int, page_size: int):
    """(pointer, pages, pitch) of a cache tensor: uint8 [pages, >= kv_nvfp4_page_bytes]."""
    ptr, pages, size, pitch = _rows2d(cache, "cache", _u8, "uint8 [pages, bytes]")
    need = kv_nvfp4_page_bytes(kv_heads, page_size)
    if size < need:
        raise ValueError(f"a page of {page_size} tokens and {kv_heads} kv heads is {need} bytes, got {size}")
    return ptr, pages, pitch


def _rows_heads(t, name: str, want=None):
    """A [tokens, heads, head_dim] bfloat16 CUDA tensor with dense rows (of shape `want`,
    if given): (pointer, pitch)."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _bf16 or len(shape) != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a 3-D [tokens, heads, head_dim] bfloat16 CUDA tensor, got {t.dtype} "
                         f"{tuple(shape)} {t.device}")
    if want is not None and shape != want:
        raise ValueError(f"{name} must be {list(want)}, got {tuple(shape)}")
    T, H, D = shape
    if (stride[2] != 1 and D > 1) or (stride[1] != D and H > 1):
        raise ValueError(f"{name} must have dense heads x head_dim rows")
    pitch = stride[0] if T > 1 else H * D
    if pitch < H * D:
        raise ValueError(f"{name} token rows overlap (pitch {pitch} < {H * D} elements)")
    return t.data_ptr(), pitch


def kv_nvfp4_page_bytes(kv_heads: int, page_size: int) -> int:
    """Bytes of one page of a paged NVFP4 KV cache (page_size a multiple of 16)."""
    n = load().kv_nvfp4_page_bytes(kv_heads, page_size)
    if n < 0:
        raise ValueError(f"page_size must be a positive multiple of 16 (at most 65536), got {page_size}")
    return n


def kv_pages_assign(seq_lens, new_lens, free_pages, free_head, block_table, page_size: int, tokens: int | None = None,
                    slots=None, positions=None, cu_new=None, total_lens=None, free_head_out=None, unserved=None,
                    stream=None):
    """Pages, slots and positions of a step's new tokens, on the device (int32
    tensors): request b grows from seq_lens[b] by new_lens[b], new pages come from
    free_pages[free_head:], block_table [requests, max_pages] is extended in place.
    ``tokens`` is the number of rows of slots and positions (needed when they are
    not given).  Returns (slots, positions, cu_new, total_lens, free_head_out,
    unserved); total_lens may be seq_lens and free_head_out free_head."""
    torch = _torch()
    n = seq_lens.numel()
    sl, nl = _int32s(seq_lens, "seq_lens"), _int32s(new_lens, "new_lens", n)
    fp, fh = _int32s(free_pages, "free_pages"), _int32s(free_head, "free_head", 1)
    tab, rows, max_pages, pitch = _block_table(block_table)
    if rows != n:
        raise ValueError(f"block_table must have {n} rows, got {tuple(block_table.shape)}")
    if tokens is None:
        given = slots if slots is not None else positions
        if given is None:
            raise ValueError("tokens (the rows of slots and positions) is needed")
        tokens = given.numel()
    dev = seq_lens.device

    def out(t, name, size):
        t = torch.empty(size, dtype=torch.int32, device=dev) if t is None else t
        return t, _int32s(t, name, size)

    slots, sp = out(slots, "slots", tokens)
    positions, pp = out(positions, "positions", tokens)
    cu_new, cp = out(cu_new, "cu_new", n + 1)
    total_lens, tp = out(total_lens, "total_lens", n)
    free_head_out, hp = out(free_head_out, "free_head_out", 1)
    unserved, up = out(unserved, "unserved", 1)
    _on_device(seq_lens, load().kv_pages_assign,
               (sl, nl, n, fp, free_pages.numel(), fh, tab, pitch, max_pages, page_size, sp, pp, tokens, cp, tp, hp, up),
               stream, "kv_pages_assign")
    return slots, positions, cu_new, total_lens, free_head_out, unserved


def _norm_weight(w, name: str, D: int):
    if w.dtype is not _bf16 or w.shape != (D,) or not w.is_cuda or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{D}] bfloat16 CUDA tensor")
    return w.data_ptr()


def qk_norm_rope_bf16(Q, K, cos_sin, positions, wq=None, wk=None, eps: float = 1e-6, neighbours: bool = False,
                      Q_out=None, K_out=None, stream=None):
    """RMS norm of every head of Q [T, H, D] and K [T, Hkv, D] (with the bfloat16
    weights wq, wk [D]; None: no norm) and the position rotation by the float32
    table cos_sin [max_pos, rot_dim] (cosines, then sines) at positions [T]; pairs
    are (i, i + rot_dim / 2), or neighbours (2i, 2i + 1).  Q_out and K_out may be Q
    and K.  Returns (Q_out, K_out)."""
    torch = _torch()
    q_ptr, ldq = _rows_heads(Q, "Q")
    k_ptr, ldk = _rows_heads(K, "K")
    q_shape, k_shape = Q.shape, K.shape
    T, H, D = q_shape
    Hkv = k_shape[1]
    if k_shape[0] != T or k_shape[2] != D:
        raise ValueError(f"Q and K must share tokens and head_dim: {tuple(q_shape)} and {tuple(k_shape)}")
    if cos_sin.dtype is not _f32 or cos_sin.dim() != 2 or not cos_sin.is_cuda or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be a contiguous [max_pos, rot_dim] float32 CUDA tensor, got {cos_sin.dtype} "
                         f"{tuple(cos_sin.shape)} {cos_sin.device}")
    max_pos, rot = cos_sin.shape
    wq_ptr = None if wq is None else _norm_weight(wq, "wq", D)
    wk_ptr = None if wk is None else _norm_weight(wk, "wk", D)
    if Q_out is None:
        Q_out = torch.empty(q_shape, dtype=torch.bfloat16, device=Q.device)
    if K_out is None:
        K_out = torch.empty(k_shape, dtype=torch.bfloat16, device=K.device)
    qo_ptr, ldqo = (q_ptr, ldq) if Q_out is Q else _rows_heads(Q_out, "Q_out", q_shape)
    ko_ptr, ldko = (k_ptr, ldk) if K_out is K else _rows_heads(K_out, "K_out", k_shape)
    _on_device(Q, load().qk_norm_rope_bf16,
               (q_ptr, k_ptr, qo_ptr, ko_ptr, T, H, Hkv, D, ldq, ldk, ldqo, ldko, wq_ptr, wk_ptr, eps,
                cos_sin.data_ptr(), max_pos, rot, _int32s(positions, "positions", T), 1 if neighbours else 0),
               stream, "qk_norm_rope_bf16")
    return Q_out, K_out


def kv_append_nvfp4(K, V, cache, slots, page_size: int, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Quantises K and V [T, Hkv, 128] (bfloat16) into the slots [T] (int32; negative:
    skipped) of the paged NVFP4 cache (uint8 [pages, kv_nvfp4_page_bytes]); the
    scales are powers of two.  Returns the cache."""
    torch = _torch()
    k_ptr, ldk = _rows_heads(K, "K")
    shape = K.shape
    T, Hkv, D = shape
    v_ptr, ldv = _rows_heads(V, "V", shape)
    c_ptr, pages, pitch = _kv_cache(cache, Hkv, page_size)
    _on_device(K, load().kv_append_nvfp4,
               (k_ptr, v_ptr, T, Hkv, D, ldk, ldv, c_ptr, pages, pitch, page_size, _int32s(slots, "slots", T), k_scale,
                v_scale), stream, "kv_append_nvfp4")
    return cache


def kv_read_nvfp4(cache, slots, kv_heads: int, page_size: int, k_scale: float = 1.0, v_scale: float = 1.0, K=None,
                  V=None, stream=None):
    """The rows of the paged NVFP4 cache at slots [T] as bfloat16 K, V [T, kv_heads,
    128] (exact; a negative slot gives zeros)."""
    torch = _torch()
    T = slots.numel()
    shape = (T, kv_heads, 128)
    K = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if K is None else K
    V = torch.empty(shape, dtype=torch.bfloat16, device=cache.device) if V is None else V
    k_ptr, ldk = _rows_heads(K, "K", shape)
    v_ptr, ldv = _rows_heads(V, "V", shape)
    c_ptr, pages, pitch = _kv_cache(cache, kv_heads, page_size)
    _on_device(cache, load().kv_read_nvfp4,
               (c_ptr, pages, pitch, page_size, _int32s(slots, "slots"), T, kv_heads, 128, k_ptr, v_ptr, ldk, ldv,
                k_scale, v_scale), stream, "kv_read_nvfp4")
    return K, V


def attention_kv_nvfp4(Q, cache, block_table, seq_lens, cu_q, kv_heads: int, page_size: int, max_q: int, O=None,
                       causal: bool = True, scale: float | None = None, k_scale: float = 1.0, v_scale: float = 1.0,
                       stream=None, path: int = PATH_AUTO):
    """Attention of Q [T, H, 128] over the paged NVFP4 cache: request b's queries are
    rows cu_q[b] .. cu_q[b + 1] (at most max_q), its keys the seq_lens[b] tokens of
    block_table[b] (queries last, causal).  ``path``: PATH_AUTO, PATH_STREAM (decode)
    or PATH_TENSOR_CORE (prefill).  Returns O [T, H, 128]."""
    torch = _torch()
    q_ptr, ldq = _rows_heads(Q, "Q")
    shape = Q.shape
    T, H, D = shape
    c_ptr, pages, pitch = _kv_cache(cache, kv_heads, page_size)
    tab, n, max_pages, tpitch = _block_table(block_table)
    if O is None:
        O = torch.empty(shape, dtype=torch.bfloat16, device=Q.device)
    o_ptr, ldo = _rows_heads(O, "O", shape)
    _on_device(Q, load().attention_kv_nvfp4_path,
               (q_ptr, c_ptr, o_ptr, tab, tpitch, max_pages, _int32s(seq_lens, "seq_lens", n),
                _int32s(cu_q, "cu_q", n + 1), n, T, max_q, H, kv_heads, D, ldq, ldo, pages, pitch, page_size,
                1 if causal else 0, D ** -0.5 if scale is None else float(scale), k_scale, v_scale, path),
               stream, "attention_kv_nvfp4")
    return O


def gemv_bf16_batched(A, Bs, Cs=None, stream=None, path: int = PATH_AUTO):
    """C_i = A @ B_i^T for every weight B_i (all [N_i, K]) in one launch; returns
    the list of C_i."""
    torch = _torch()
    a_ptr, lda = _operand(A, "A")
    M, K = A.shape
    n = len(Bs)
    if Cs is None:
        Cs = []
        for B in Bs:
            ld = -(-B.shape[0] // 8) * 8
            Cs.append(torch.empty((M, ld), dtype=torch.bfloat16, device=A.device)[:, :B.shape[0]])
    if len(Cs) != n:
        raise ValueError("one output per weight")
    bp, nn, lb, cp, lc = ((ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int64 * n)(),
                          (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)())
    for i, (B, C) in enumerate(zip(Bs, Cs)):
        b_ptr, ldb = _operand(B, f"B[{i}]")
        c_ptr, ldc = _operand(C, f"C[{i}]")
        if B.shape[1] != K or tuple(C.shape) != (M, B.shape[0]):
            raise ValueError(f"shapes of B[{i}] {tuple(B.shape)} / C[{i}] {tuple(C.shape)}")
        bp[i], nn[i], lb[i], cp[i], lc[i] = b_ptr, B.shape[0], ldb, c_ptr, ldc
    with torch.cuda.device(A.device):
        st = load().gemv_bf16_batched(a_ptr, M, K, lda, bp, nn, lb, cp, lc, n, path, _stream_handle(stream))
    _check(st, "gemv_bf16_batched")
    return Cs


def gemv_bf16(A, B, C=None, stream=None, path: int = PATH_AUTO):
    """The skinny path (1 <= M <= 64); ``path`` picks the kernel (PATH_*)."""
    return _call("gemv_bf16", A, B, C, stream, path)


def gemv_bf16_noalloc(A, B, C=None, stream=None):
    """The CUDA-core skinny path with its scratch in the library's fixed device
    array instead of an allocated workspace (for callers that cannot allocate)."""
    return _call("gemv_bf16_noalloc", A, B, C, stream)


# ------------------------------------------------------------------ host-only helpers
def plan(M: int, N: int, K: int, num_sms: int, entry: int = 0) -> dict:
    info = PlanInfo()
    _check(load().sg_plan(M, N, K, num_sms, entry, ctypes.byref(info)), "sg_plan")
    d = info.as_dict()
    d["_struct"] = info
    return d


def plan_nvfp4(M: int, N: int, K: int, num_sms: int, path: int = PATH_AUTO) -> dict:
    info = PlanInfo()
    _check(load().sg_plan_nvfp4(M, N, K, num_sms, path, ctypes.byref(info)), "sg_plan_nvfp4")
    d = info.as_dict()
    d["_struct"] = info
    return d


def plan_swiglu(M: int, N: int, K: int, num_sms: int, entry: int = 0) -> dict:
    info = PlanInfo()
    _check(load().sg_plan_swiglu(M, N, K, num_sms, entry, ctypes.byref(info)), "sg_plan_swiglu")
    d = info.as_dict()
    d["_struct"] = info
    return d


def plan_items(info: dict) -> list[list[tuple]]:
    """All work items of a tcgen05 plan, per CTA: (tile, k0, k1, piece, npieces, slot, sk_index, tm, tn)."""
    lib = load()
    out = (ctypes.c_int32 * 9)()
    st = info["_struct"]
    items = []
    for cta in range(info["grid"]):
        row = []
        n = lib.sg_plan_item(ctypes.byref(st), cta, 0, out)
        for i in range(max(n, 0)):
            lib.sg_plan_item(ctypes.byref(st), cta, i, out)
            row.append(tuple(out))
        items.append(row)
    return items


def wave_efficiency(ctas: int, slots: int) -> float:
    return load().sg_wave_efficiency(ctas, slots)


def set_wait_timeout_ns(ns: int) -> None:
    load().sg_set_wait_timeout_ns(ns)


def check_device_errors(stream=None):
    """Synchronises the stream; returns (status, detail[4]) of kernel wait timeouts and
    indices out of range, a timeout first (the other kind by the next call)."""
    detail = (ctypes.c_uint32 * 4)()
    st = load().sg_check_device_errors(_stream_handle(stream), detail)
    return st, list(detail)


def device_query() -> dict:
    info = DeviceInfo()
    _check(load().sg_device_query(ctypes.byref(info)), "sg_device_query")
    return {name: getattr(info, name) for name, _ in info._fields_}


def bench_tcgen05_peak(iters: int, stream=None) -> tuple[float, float]:
    tf, mhz = ctypes.c_double(), ctypes.c_double()
    _check(load().sg_bench_tcgen05_peak(iters, ctypes.byref(tf), ctypes.byref(mhz), _stream_handle(stream)),
           "sg_bench_tcgen05_peak")
    return tf.value, mhz.value


def bench_copy(dst, src, reps: int = 20, stream=None) -> float:
    g = ctypes.c_double()
    nbytes = src.numel() * src.element_size()
    _check(load().sg_bench_copy(dst.data_ptr(), src.data_ptr(), nbytes, reps, ctypes.byref(g),
                                _stream_handle(stream)), "sg_bench_copy")
    return g.value


def bench_read(src, sink, reps: int = 20, stream=None) -> float:
    g = ctypes.c_double()
    nbytes = src.numel() * src.element_size()
    _check(load().sg_bench_read(src.data_ptr(), nbytes, reps, sink.data_ptr(), ctypes.byref(g),
                                _stream_handle(stream)), "sg_bench_read")
    return g.value
