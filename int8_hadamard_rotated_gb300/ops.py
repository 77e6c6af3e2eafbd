"""Thin Python binding of libconvrot.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks dtypes/devices, allocates outputs and
workspace with PyTorch when the caller does not pass them, and hands raw
device pointers plus the current CUDA stream to the library. All compute runs
in the library's sm_103a kernels; if the library is missing this module
raises, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import List, Optional, Sequence, Tuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libconvrot.so")

# status codes (include/convrot.h)
OK = 0
ERR_ARG = 1
ERR_GROUP = 2
ERR_ALIGN = 3
ERR_OVERFLOW = 4
ERR_ALIAS = 5
ERR_WORKSPACE = 6
ERR_UNSUPPORTED = 7
ERR_TIMEOUT = 8
ERR_CUDA = 9
ERR_DEVICE = 10
ERR_SCRATCH = 11

ACT_NONE = 0
ACT_GELU = 1
ACT_SWIGLU = 2

NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2

F32 = 0
F16 = 1
BF16 = 2
MAX_LINEARS = 8
PACK_MAX_K = 32768
MAX_K = 133144
W4_MAX_K = 16384
CHUNK_ROWS = 128
NOALLOC_SCRATCH_BYTES = 32 << 20
GEMM_SYNC_BYTES = 4096
NORM_MAX_K = 32768
FP8_BLOCK = 128

MOE_SOFTMAX = 0
MOE_SIGMOID = 1
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOP_K = 32
MOE_MAX_GROUPS = 32


class ConvrotError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _lib_or_none()
        msg = lib.convrot_strerror(status).decode() if lib else str(status)
        if status == ERR_CUDA and lib:
            msg += f" (cudaError {lib.convrot_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [status {status}]")
        self.status = status


class convrot_prologue(ctypes.Structure):
    _fields_ = [("rmsnorm", ctypes.c_int), ("eps", ctypes.c_float), ("weight", ctypes.c_void_p),
                ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p)]


class convrot_weight(ctypes.Structure):
    _fields_ = [("q16", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("Y", ctypes.c_void_p), ("kchunk", ctypes.c_void_p),
                ("q4", ctypes.c_void_p)]


class convrot_block_norm_args(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int), ("u_dtype", ctypes.c_int),
                ("H", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("residual_scale", ctypes.c_float), ("block_scale", ctypes.c_float),
                ("post_norm", ctypes.c_int), ("pre_norm", ctypes.c_int),
                ("post_eps", ctypes.c_float), ("pre_eps", ctypes.c_float),
                ("post_weight", ctypes.c_void_p), ("post_bias", ctypes.c_void_p),
                ("pre_weight", ctypes.c_void_p), ("pre_bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("shift", ctypes.c_void_p),
                ("ld_gate", ctypes.c_int64), ("ld_mod", ctypes.c_int64), ("n_samples", ctypes.c_int64),
                ("row_sample", ctypes.c_void_p), ("rows_per_sample", ctypes.c_int64),
                ("H_out", ctypes.c_void_p), ("U", ctypes.c_void_p), ("ldho", ctypes.c_int64), ("ldu", ctypes.c_int64),
                ("Q", ctypes.c_void_p), ("s", ctypes.c_void_p)]


class convrot_fp8_weight(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class convrot_moe_route_args(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("n_experts", ctypes.c_int), ("top_k", ctypes.c_int), ("dtype", ctypes.c_int),
                ("score", ctypes.c_int), ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("bias", ctypes.c_void_p), ("n_groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("group_top", ctypes.c_int), ("renormalise", ctypes.c_int), ("scale", ctypes.c_float),
                ("experts", ctypes.c_void_p), ("weights", ctypes.c_void_p)]


class convrot_experts(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64), ("bias_stride", ctypes.c_int64)]


class convrot_moe_args(ctypes.Structure):
    _fields_ = [("X", ctypes.c_void_p), ("x_dtype", ctypes.c_int), ("T", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("experts", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("top_k", ctypes.c_int), ("n_experts", ctypes.c_int), ("gate", ctypes.c_void_p),
                ("up", ctypes.c_void_p), ("down", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("ld_res", ctypes.c_int64), ("Y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("y_dtype", ctypes.c_int)]


_LIB = None

_VP, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
SIGNATURES = {
    "convrot_version": (_I, []),
    "convrot_strerror": (ctypes.c_char_p, [_I]),
    "convrot_last_cuda_error": (_I, []),
    "convrot_prepare_weight": (_I, [_VP, _I64, _I64, _I, _VP, _VP, _VP, _VP]),
    "convrot_pack_activations": (_I, [_VP, _I, _I64, _I64, _I, _VP, _VP, _VP]),
    "int8_linear_workspace_size": (_SZ, [_I64, _I64, _I64, _I]),
    "int8_linear": (_I, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _VP, _I64, _VP, _VP, _SZ, _VP]),
    "convrot_linear_workspace_size": (_SZ, [_I64, _I64]),
    "convrot_linear": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _I, _VP, _SZ, _VP]),
    "convrot_pack_prologue": (_I, [_VP, _I64, _I64, _I, ctypes.POINTER(convrot_prologue), _VP, _VP, _VP]),
    "convrot_linear_prologue": (_I, [_VP, _I64, _I64, _I, ctypes.POINTER(convrot_prologue),
                                     ctypes.POINTER(convrot_weight), _I, _VP, _SZ, _VP]),
    "convrot_linear_scaled": (_I, [_VP, _I, _I64, _I64, _I, ctypes.c_float, ctypes.POINTER(convrot_weight), _I,
                                   _VP, _SZ, _VP]),
    "int8_gemm_s32": (_I, [_VP, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _VP, _SZ, _VP]),
    "int8_gemm_s32_w4_workspace_size": (_SZ, [_I64, _I64]),
    "int8_gemm_s32_w4": (_I, [_VP, _I64, _I64, _VP, _I64, _VP, _VP, _SZ, _VP]),
    "convrot_weight_chunks": (_I, [_VP, _I64, _I64, _VP, _VP]),
    "convrot_w4_expand": (_I, [_VP, _I64, _I64, _VP, _VP, _VP]),
    "convrot_pack_activations_f16": (_I, [_VP, _I, _I64, _I64, _I, _VP, _VP, _VP]),
    "convrot_linear_packed": (_I, [_VP, _VP, _I64, _I64, ctypes.POINTER(convrot_weight), _I, _VP, _SZ, _VP]),
    "convrot_pack_gelu_f16": (_I, [_VP, _I64, _I64, _I, _VP, _VP, _VP]),
    "convrot_linear_packed_act": (_I, [_VP, _VP, _I64, _I64, ctypes.POINTER(convrot_weight), _I, _I, _VP, _SZ,
                                       _VP]),
    "convrot_linear_host_workspace_size": (_SZ, [_I64, _I64, _I, _I64, _I64]),
    "convrot_linear_host": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _I, _I64, _VP, _SZ,
                                 _VP, _VP, _VP]),
    "convrot_mlp_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "convrot_mlp_host_workspace_size": (_SZ, [_I64, _I64, _I, _I64, _I64, _I64]),
    "convrot_mlp_host": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _I, _I,
                              ctypes.POINTER(convrot_weight), _VP, _I64, _VP, _SZ, _VP, _VP, _VP]),
    "convrot_mlp": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _I, _I,
                         ctypes.POINTER(convrot_weight), _VP, _SZ, _VP]),
    "convrot_linear_noalloc": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _I, _VP]),
    "convrot_linear_swiglu": (_I, [_VP, _I, _I64, _I64, _I, ctypes.POINTER(convrot_weight), _VP, _SZ, _VP]),
    "convrot_block_norm": (_I, [_VP, _VP]),
    "fp8_pack_activations": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _VP, _VP]),
    "fp8_prepare_weight": (_I, [_VP, _I, _I64, _I64, _VP, _VP, _VP]),
    "fp8_linear_workspace_size": (_SZ, [_I64, _I64]),
    "fp8_linear_packed": (_I, [_VP, _VP, _I64, _I64, _VP, _I, _I, _VP]),
    "fp8_linear": (_I, [_VP, _I, _I64, _I64, _I64, _VP, _I, _I, _VP, _SZ, _VP]),
    "moe_route": (_I, [_VP, _VP]),
    "moe_plan_workspace_size": (_SZ, [_I64, _I]),
    "moe_plan": (_I, [_VP, _I64, _I, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fp8_expert_linear": (_I, [_VP, _VP, _I64, _I64, _VP, _VP, _I64, _I, _I, _VP, _VP, _I64, _I, _VP, _SZ,
                               _VP]),
    "fp8_expert_swiglu": (_I, [_VP, _VP, _I64, _I64, _VP, _VP, _I64, _I, _I, _VP, _VP, _VP, _VP, _VP, _SZ, _VP]),
    "fp8_expert_workspace_size": (_SZ, [_I64, _I64, _I]),
    "moe_combine": (_I, [_VP, _I, _I64, _I64, _VP, _VP, _I64, _I, _I64, _VP, _I64, _VP, _I64, _I, _VP]),
    "fp8_moe_workspace_size": (_SZ, [_I64, _I64, _I64, _I64, _I, _I, _I]),
    "fp8_moe": (_I, [_VP, _VP, _SZ, _VP]),
    "convrot_device_status": (_I, [_VP]),
    "convrot_test_block_norm_timeout": (_I, [_VP, _I64, ctypes.c_uint64, _VP]),
    "fp8_test_linear_timeout": (_I, [_VP, _VP, _I64, _I64, _VP, _I, _I, ctypes.c_uint64, _VP]),
    "fp8_test_expert_timeout": (_I, [_VP, _VP, _I64, _I64, _VP, _I, _VP, _VP, _VP, _VP, _I64, _I, ctypes.c_uint64,
                                     _VP]),
    "convrot_test_handover_timeout": (_I, [_VP, _VP, _I64, _I64, ctypes.POINTER(convrot_weight), _I, _VP, _SZ,
                                           ctypes.c_uint64, _VP]),
    "convrot_test_unscale_sweep": (_I, [_VP, _I, _I, _VP, _VP, _VP]),
}


def _lib_or_none():
    return _LIB


def lib() -> ctypes.CDLL:
    """Load libconvrot.so (once). Raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m int8_hadamard_rotated_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int, where: str):
    if status != OK:
        raise ConvrotError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _need(t: torch.Tensor, dtype, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _xdtype(X: torch.Tensor) -> int:
    if X.dtype == torch.float32:
        return F32
    if X.dtype == torch.float16:
        return F16
    raise ValueError("X must be float32 or float16")


# ---------------------------------------------------------------------------

def convrot_pack_activations(X: torch.Tensor, G: int, Q_x: Optional[torch.Tensor] = None,
                             s_x: Optional[torch.Tensor] = None, stream=None
                             ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rotate and quantize the rows of X [M,K] -> (Q_x int8 [M,K], s_x f32 [M])."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    if Q_x is None:
        Q_x = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if s_x is None:
        s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _need(Q_x, torch.int8, "Q_x")
    _need(s_x, torch.float32, "s_x")
    _check(lib().convrot_pack_activations(_ptr(X), xd, M, K, G, _ptr(Q_x), _ptr(s_x), _stream(stream)),
           "convrot_pack_activations")
    return Q_x, s_x


def convrot_prepare_weight(W: torch.Tensor, G: int, with_f16: bool = True, stream=None):
    """Offline weight path: W [N,K] f32 -> (Q_w int8, s_w f32, Q_w16 fp16 codes or None)."""
    _need(W, torch.float32, "W")
    N, K = W.shape
    Q_w = torch.empty((N, K), dtype=torch.int8, device=W.device)
    s_w = torch.empty((N,), dtype=torch.float32, device=W.device)
    Q_w16 = torch.empty((N, K), dtype=torch.float16, device=W.device) if with_f16 else None
    _check(lib().convrot_prepare_weight(_ptr(W), N, K, G, _ptr(Q_w), _ptr(s_w), _ptr(Q_w16), _stream(stream)),
           "convrot_prepare_weight")
    return Q_w, s_w, Q_w16


def int8_linear_workspace_size(M: int, N: int, K: int, have_q_w16: bool) -> int:
    return int(lib().int8_linear_workspace_size(M, N, K, 1 if have_q_w16 else 0))


def convrot_linear_workspace_size(M: int, K: int) -> int:
    return int(lib().convrot_linear_workspace_size(M, K))


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is None:
        return torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError("workspace too small")
    return workspace


def int8_linear(Q_x, s_x, Q_w=None, Q_w16=None, s_w=None, bias=None, Y=None,
                workspace=None, stream=None) -> torch.Tensor:
    """Y = float(Q_x Q_w^T) * s_x * s_w + bias, fp32 [M,N]."""
    _need(Q_x, torch.int8, "Q_x")
    _need(s_x, torch.float32, "s_x")
    ref = Q_w16 if Q_w16 is not None else Q_w
    if ref is None:
        raise ValueError("Q_w or Q_w16 is required")
    M, K = Q_x.shape
    N = ref.shape[0]
    if Q_w is not None:
        _need(Q_w, torch.int8, "Q_w")
    if Q_w16 is not None:
        _need(Q_w16, torch.float16, "Q_w16")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.float32, device=Q_x.device)
    ws = _workspace(int8_linear_workspace_size(M, N, K, Q_w16 is not None), Q_x.device, workspace)
    _check(lib().int8_linear(_ptr(Q_x), _ptr(s_x), M, K, _ptr(Q_w), _ptr(Q_w16), _ptr(s_w), _ptr(bias),
                             N, _ptr(Y), _ptr(ws), ws.numel(), _stream(stream)), "int8_linear")
    return Y


def convrot_weight_chunks(Q_w: torch.Tensor, kchunk: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Exact-chunk plan of int8 weight codes [N,K]: int32 [ceil(N/128)]."""
    _need(Q_w, torch.int8, "Q_w")
    N, K = Q_w.shape
    if kchunk is None:
        kchunk = torch.empty(((N + CHUNK_ROWS - 1) // CHUNK_ROWS,), dtype=torch.int32, device=Q_w.device)
    _check(lib().convrot_weight_chunks(_ptr(Q_w), N, K, _ptr(kchunk), _stream(stream)), "convrot_weight_chunks")
    return kchunk


def convrot_w4_expand(Q_w4: torch.Tensor, K: int, with_int8: bool = True, stream=None):
    """Packed signed 4-bit weights [N, K/2] (uint8, low nibble first) ->
    (int8 codes or None, binary16 codes) [N, K]."""
    _need(Q_w4, torch.uint8, "Q_w4")
    N = Q_w4.shape[0]
    if Q_w4.shape[1] * 2 != K:
        raise ValueError("Q_w4 must be [N, K/2]")
    q8 = torch.empty((N, K), dtype=torch.int8, device=Q_w4.device) if with_int8 else None
    q16 = torch.empty((N, K), dtype=torch.float16, device=Q_w4.device)
    _check(lib().convrot_w4_expand(_ptr(Q_w4), N, K, _ptr(q8), _ptr(q16), _stream(stream)), "convrot_w4_expand")
    return q8, q16


def int8_gemm_s32(Q_x, Q_w=None, Q_w16=None, A=None, workspace=None, stream=None, kchunk=None) -> torch.Tensor:
    """Raw int32 A = Q_x Q_w^T through the tensor-core GEMM (optionally with
    the weight's exact-chunk plan)."""
    _need(Q_x, torch.int8, "Q_x")
    ref = Q_w16 if Q_w16 is not None else Q_w
    M, K = Q_x.shape
    N = ref.shape[0]
    if A is None:
        A = torch.empty((M, N), dtype=torch.int32, device=Q_x.device)
    ws = _workspace(int8_linear_workspace_size(M, N, K, Q_w16 is not None), Q_x.device, workspace)
    _check(lib().int8_gemm_s32(_ptr(Q_x), M, K, _ptr(Q_w), _ptr(Q_w16), _ptr(kchunk), N, _ptr(A), _ptr(ws),
                               ws.numel(), _stream(stream)), "int8_gemm_s32")
    return A


def int8_gemm_s32_w4(Q_x, Q_w4, A=None, workspace=None, stream=None) -> torch.Tensor:
    """Raw int32 A = Q_x Q_w^T with packed signed 4-bit weights Q_w4 [N, K/2]
    (uint8, low nibble first), through the S8 x S4 GEMM."""
    _need(Q_x, torch.int8, "Q_x")
    _need(Q_w4, torch.uint8, "Q_w4")
    M, K = Q_x.shape
    N = Q_w4.shape[0]
    if Q_w4.shape[1] * 2 != K:
        raise ValueError("Q_w4 must be [N, K/2]")
    if A is None:
        A = torch.empty((M, N), dtype=torch.int32, device=Q_x.device)
    ws = _workspace(int(lib().int8_gemm_s32_w4_workspace_size(M, K)), Q_x.device, workspace)
    _check(lib().int8_gemm_s32_w4(_ptr(Q_x), M, K, _ptr(Q_w4), N, _ptr(A), _ptr(ws), ws.numel(), _stream(stream)),
           "int8_gemm_s32_w4")
    return A


def make_weights(q16s: Sequence[torch.Tensor], scales: Sequence[Optional[torch.Tensor]],
                 biases: Sequence[Optional[torch.Tensor]], Ys: Sequence[torch.Tensor],
                 kchunks: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """The convrot_weight descriptors (kchunks: optional exact-chunk plans).
    Each weight is binary16 codes [N, K] (float16) or packed signed 4-bit
    weights [N, K/2] (uint8, low nibble first), which the S8 x S4 GEMM reads
    as they are."""
    arr = (convrot_weight * len(q16s))()
    if kchunks is None:
        kchunks = [None] * len(q16s)
    for j, (q, s, b, y, kc) in enumerate(zip(q16s, scales, biases, Ys, kchunks)):
        if q.dtype == torch.uint8:
            arr[j] = convrot_weight(None, _ptr(s), _ptr(b), q.shape[0], _ptr(y), None, _ptr(q))
        else:
            arr[j] = convrot_weight(_ptr(q), _ptr(s), _ptr(b), q.shape[0], _ptr(y), _ptr(kc), None)
    return arr


def convrot_linear(X: torch.Tensor, G: int, q16s: Sequence[torch.Tensor],
                   scales: Sequence[Optional[torch.Tensor]], biases: Sequence[Optional[torch.Tensor]],
                   Ys: Optional[List[torch.Tensor]] = None, workspace=None, stream=None,
                   weights=None, kchunks=None) -> List[torch.Tensor]:
    """Pack X once, then every Y_j = float(Q_x Q_wj^T) * s_x * s_wj + b_j."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=X.device) for q in q16s]
    ws = _workspace(convrot_linear_workspace_size(M, K), X.device, workspace)
    if weights is None:
        weights = make_weights(q16s, scales, biases, Ys, kchunks)
    _check(lib().convrot_linear(_ptr(X), xd, M, K, G, weights, len(q16s), _ptr(ws), ws.numel(),
                                _stream(stream)), "convrot_linear")
    return Ys


def convrot_linear_scaled(X: torch.Tensor, G: int, input_scale: float, q16s: Sequence[torch.Tensor],
                          scales: Sequence[Optional[torch.Tensor]], biases: Sequence[Optional[torch.Tensor]],
                          Ys: Optional[List[torch.Tensor]] = None, workspace=None, stream=None,
                          kchunks=None, weights=None) -> List[torch.Tensor]:
    """convrot_linear with an input scale: X is scaled before the pack and
    every output unscaled before its bias."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=X.device) for q in q16s]
    ws = _workspace(convrot_linear_workspace_size(M, K), X.device, workspace)
    if weights is None:
        weights = make_weights(q16s, scales, biases, Ys, kchunks)
    _check(lib().convrot_linear_scaled(_ptr(X), xd, M, K, G, float(input_scale), weights, len(q16s), _ptr(ws),
                                       ws.numel(), _stream(stream)), "convrot_linear_scaled")
    return Ys


def _prologue(rmsnorm=False, eps=1e-6, weight=None, scale=None, shift=None):
    for name, t in (("weight", weight), ("scale", scale), ("shift", shift)):
        if t is not None:
            _need(t, torch.float32, name)
    return convrot_prologue(1 if rmsnorm else 0, float(eps), _ptr(weight), _ptr(scale), _ptr(shift))


def convrot_pack_prologue(X: torch.Tensor, G: int, rmsnorm=False, eps=1e-6, weight=None, scale=None, shift=None,
                          Q_x=None, s_x=None, stream=None):
    """Pack of the modulated X (RMS norm, per-channel weight, modulation) into
    int8 codes and row scales, without materializing the modulated X."""
    _need(X, torch.float32, "X")
    M, K = X.shape
    if Q_x is None:
        Q_x = torch.empty((M, K), dtype=torch.int8, device=X.device)
    if s_x is None:
        s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    pro = _prologue(rmsnorm, eps, weight, scale, shift)
    _check(lib().convrot_pack_prologue(_ptr(X), M, K, G, ctypes.byref(pro), _ptr(Q_x), _ptr(s_x), _stream(stream)),
           "convrot_pack_prologue")
    return Q_x, s_x


def convrot_linear_prologue(X: torch.Tensor, G: int, q16s, scales, biases, rmsnorm=False, eps=1e-6,
                            weight=None, scale=None, shift=None, Ys=None, workspace=None, stream=None,
                            kchunks=None):
    """convrot_linear of the modulated X."""
    _need(X, torch.float32, "X")
    M, K = X.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=X.device) for q in q16s]
    ws = _workspace(convrot_linear_workspace_size(M, K), X.device, workspace)
    pro = _prologue(rmsnorm, eps, weight, scale, shift)
    weights = make_weights(q16s, scales, biases, Ys, kchunks)
    _check(lib().convrot_linear_prologue(_ptr(X), M, K, G, ctypes.byref(pro), weights, len(q16s), _ptr(ws),
                                         ws.numel(), _stream(stream)), "convrot_linear_prologue")
    return Ys


def convrot_pack_activations_f16(X: torch.Tensor, G: int, Q_x16: Optional[torch.Tensor] = None,
                                 s_x: Optional[torch.Tensor] = None, stream=None):
    """Pack X into the GEMM operand form: (Q_x16 fp16 codes [M,K], s_x f32 [M])."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    if Q_x16 is None:
        Q_x16 = torch.empty((M, K), dtype=torch.float16, device=X.device)
    if s_x is None:
        s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _need(Q_x16, torch.float16, "Q_x16")
    _need(s_x, torch.float32, "s_x")
    _check(lib().convrot_pack_activations_f16(_ptr(X), xd, M, K, G, _ptr(Q_x16), _ptr(s_x), _stream(stream)),
           "convrot_pack_activations_f16")
    return Q_x16, s_x


def convrot_linear_packed(Q_x16: torch.Tensor, s_x: torch.Tensor, q16s, scales, biases,
                          Ys=None, stream=None, weights=None, kchunks=None, workspace=None,
                          split_tail: bool = True):
    """Grouped GEMM on an already packed activation (fp16 codes + row scales).
    With split_tail (the default) the GEMM gets GEMM_SYNC_BYTES of scratch
    (`workspace`, or a fresh buffer) and may split its last wave of tiles by K;
    split_tail=False passes none (whole tiles only; same results)."""
    _need(Q_x16, torch.float16, "Q_x16")
    _need(s_x, torch.float32, "s_x")
    M, K = Q_x16.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=Q_x16.device) for q in q16s]
    if weights is None:
        weights = make_weights(q16s, scales, biases, Ys, kchunks)
    ws_ptr, ws_bytes = None, 0
    if split_tail:
        ws = _workspace(GEMM_SYNC_BYTES, Q_x16.device, workspace)
        ws_ptr, ws_bytes = _ptr(ws), ws.numel() * ws.element_size()
    _check(lib().convrot_linear_packed(_ptr(Q_x16), _ptr(s_x), M, K, weights, len(q16s), ws_ptr, ws_bytes,
                                       _stream(stream)),
           "convrot_linear_packed")
    return Ys


def convrot_linear_packed_act(Q_x16: torch.Tensor, s_x: torch.Tensor, q16s, scales, biases, activation: int,
                              Ys=None, stream=None, kchunks=None, workspace=None):
    """convrot_linear_packed with an activation in the GEMM's epilogue: GELU
    on every output, or split SwiGLU of q16s = [gate, up] (returns [h])."""
    _need(Q_x16, torch.float16, "Q_x16")
    _need(s_x, torch.float32, "s_x")
    M, K = Q_x16.shape
    if Ys is None:
        n_out = 1 if activation == ACT_SWIGLU else len(q16s)
        Ys = [torch.empty((M, q16s[j].shape[0]), dtype=torch.float32, device=Q_x16.device) for j in range(n_out)]
    outs = [Ys[0], Ys[0]] if activation == ACT_SWIGLU else Ys
    weights = make_weights(q16s, scales, biases, outs, kchunks)
    ws = _workspace(GEMM_SYNC_BYTES, Q_x16.device, workspace)
    _check(lib().convrot_linear_packed_act(_ptr(Q_x16), _ptr(s_x), M, K, weights, len(q16s), activation, _ptr(ws),
                                           ws.numel() * ws.element_size(), _stream(stream)),
           "convrot_linear_packed_act")
    return Ys


def convrot_pack_gelu_f16(X: torch.Tensor, G: int, Q_x16: Optional[torch.Tensor] = None,
                          s_x: Optional[torch.Tensor] = None, stream=None):
    """The MLP's repack: GELU applied to fp32 X as it is loaded, then the pack
    into binary16 codes and row scales."""
    _need(X, torch.float32, "X")
    M, K = X.shape
    if Q_x16 is None:
        Q_x16 = torch.empty((M, K), dtype=torch.float16, device=X.device)
    if s_x is None:
        s_x = torch.empty((M,), dtype=torch.float32, device=X.device)
    _check(lib().convrot_pack_gelu_f16(_ptr(X), M, K, G, _ptr(Q_x16), _ptr(s_x), _stream(stream)),
           "convrot_pack_gelu_f16")
    return Q_x16, s_x


def convrot_linear_host_workspace_size(M: int, K: int, x_dtype: int, n_total: int, chunk_rows: int = 0) -> int:
    return int(lib().convrot_linear_host_workspace_size(M, K, x_dtype, n_total, chunk_rows))


def convrot_linear_host(X: torch.Tensor, G: int, q16s: Sequence[torch.Tensor],
                        scales: Sequence[Optional[torch.Tensor]], biases: Sequence[Optional[torch.Tensor]],
                        Ys: Optional[List[torch.Tensor]] = None, chunk_rows: int = 0, workspace=None,
                        stream=None, copy_in_stream=None, copy_out_stream=None, weights=None,
                        kchunks=None) -> List[torch.Tensor]:
    """convrot_linear on host arrays: X [M,K] and the outputs live in (pinned)
    host memory, the weights on the device; transfers of row chunks overlap
    compute on the given copy streams."""
    xd = _xdtype(X)
    if X.is_cuda or not X.is_contiguous():
        raise ValueError("X must be a contiguous host tensor")
    M, K = X.shape
    dev = q16s[0].device
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, pin_memory=True) for q in q16s]
    for y in Ys:
        if y.is_cuda or y.dtype != torch.float32 or not y.is_contiguous():
            raise ValueError("every Y must be a contiguous float32 host tensor")
    n_total = sum(q.shape[0] for q in q16s)
    ws = _workspace(convrot_linear_host_workspace_size(M, K, xd, n_total, chunk_rows), dev, workspace)
    if weights is None:
        weights = make_weights(q16s, scales, biases, Ys, kchunks)
    _check(lib().convrot_linear_host(X.data_ptr(), xd, M, K, G, weights, len(q16s), chunk_rows, _ptr(ws),
                                     ws.numel(), _stream(stream), _stream(copy_in_stream) if copy_in_stream else None,
                                     _stream(copy_out_stream) if copy_out_stream else None),
           "convrot_linear_host")
    return Ys


def convrot_mlp_workspace_size(M: int, K: int, N_up: int) -> int:
    return int(lib().convrot_mlp_workspace_size(M, K, N_up))


def convrot_mlp(X: torch.Tensor, G_up: int, up: Tuple, activation: int, G_down: int, down: Tuple,
                Y: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None, workspace=None,
                stream=None) -> torch.Tensor:
    """Up linear, activation, down linear on the device. `up` and `down` are
    (weight codes, scale, bias, kchunk) tuples, the codes binary16 [N, K] or
    packed 4-bit [N, K/2] (uint8); with ACT_SWIGLU `up` is a pair of such
    tuples, (gate, up). H (optional, fp32 [M, N_up]) receives the activated
    up output that the down linear packs (GELU(Y_up), or with ACT_SWIGLU
    h = silu(gate) * up)."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    ups = list(up) if activation == ACT_SWIGLU else [up]
    dq, ds, db, dk = down
    N_up, N_down = ups[0][0].shape[0], dq.shape[0]
    if Y is None:
        Y = torch.empty((M, N_down), dtype=torch.float32, device=X.device)
    if H is not None:
        _need(H, torch.float32, "H")
    wu = make_weights([u[0] for u in ups], [u[1] for u in ups], [u[2] for u in ups], [H] * len(ups),
                      [u[3] for u in ups])
    wd = make_weights([dq], [ds], [db], [Y], [dk])
    ws = _workspace(convrot_mlp_workspace_size(M, K, N_up), X.device, workspace)
    _check(lib().convrot_mlp(_ptr(X), xd, M, K, G_up, wu, activation, G_down, wd, _ptr(ws), ws.numel(),
                             _stream(stream)), "convrot_mlp")
    return Y


def convrot_mlp_host_workspace_size(M: int, K: int, x_dtype: int, N_up: int, N_down: int,
                                    chunk_rows: int = 0) -> int:
    return int(lib().convrot_mlp_host_workspace_size(M, K, x_dtype, N_up, N_down, chunk_rows))


def convrot_mlp_host(X: torch.Tensor, G_up: int, up: Tuple, activation: int, G_down: int, down: Tuple,
                     Y: Optional[torch.Tensor] = None, chunk_rows: int = 0, workspace=None, stream=None,
                     copy_in_stream=None, copy_out_stream=None) -> torch.Tensor:
    """convrot_mlp on host arrays: X [M,K] and Y [M,N_down] live in (pinned)
    host memory, the weights on the device; row chunks are copied in, run
    and copied out on three streams so that transfers overlap compute. `up`
    and `down` as in convrot_mlp."""
    xd = _xdtype(X)
    if X.is_cuda or not X.is_contiguous():
        raise ValueError("X must be a contiguous host tensor")
    M, K = X.shape
    ups = list(up) if activation == ACT_SWIGLU else [up]
    dq, ds, db, dk = down
    N_up, N_down = ups[0][0].shape[0], dq.shape[0]
    dev = dq.device
    if Y is None:
        Y = torch.empty((M, N_down), dtype=torch.float32, pin_memory=True)
    if Y.is_cuda or Y.dtype != torch.float32 or not Y.is_contiguous():
        raise ValueError("Y must be a contiguous float32 host tensor")
    wu = make_weights([u[0] for u in ups], [u[1] for u in ups], [u[2] for u in ups], [None] * len(ups),
                      [u[3] for u in ups])
    wd = make_weights([dq], [ds], [db], [None], [dk])
    ws = _workspace(convrot_mlp_host_workspace_size(M, K, xd, N_up, N_down, chunk_rows), dev, workspace)
    _check(lib().convrot_mlp_host(X.data_ptr(), xd, M, K, G_up, wu, activation, G_down, wd, Y.data_ptr(),
                                  chunk_rows, _ptr(ws), ws.numel(), _stream(stream),
                                  _stream(copy_in_stream) if copy_in_stream else None,
                                  _stream(copy_out_stream) if copy_out_stream else None), "convrot_mlp_host")
    return Y


def convrot_linear_noalloc(X: torch.Tensor, G: int, q16s: Sequence[torch.Tensor],
                           scales: Sequence[Optional[torch.Tensor]],
                           biases: Sequence[Optional[torch.Tensor]],
                           Ys: Optional[List[torch.Tensor]] = None, stream=None,
                           weights=None, kchunks=None) -> List[torch.Tensor]:
    """convrot_linear without a workspace, for callers that cannot allocate
    device memory: the packed activation lives in the library's fixed device
    array (NOALLOC_SCRATCH_BYTES per GPU). Pass preallocated Ys to make the
    whole call allocation-free; calls that overlap on the GPU race."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=X.device) for q in q16s]
    if weights is None:
        weights = make_weights(q16s, scales, biases, Ys, kchunks)
    _check(lib().convrot_linear_noalloc(_ptr(X), xd, M, K, G, weights, len(q16s), _stream(stream)),
           "convrot_linear_noalloc")
    return Ys


def convrot_device_status(stream=None) -> int:
    return int(lib().convrot_device_status(_stream(stream)))


def convrot_test_unscale_sweep(divisors: torch.Tensor, y_exp: int, stream=None) -> Tuple[int, Optional[Tuple[float, float]]]:
    """Test-only: the GEMM epilogue's unscaling step against the IEEE division
    for every divisor in `divisors` (fp32, on the device) and all 2^23 values
    y = 1.m * 2^y_exp. Returns (count of results that differ, (divisor, y) of
    the first of them or None)."""
    _need(divisors, torch.float32, "divisors")
    out = torch.tensor([0, -1], dtype=torch.int64, device=divisors.device)  # count, first (~0)
    _check(lib().convrot_test_unscale_sweep(_ptr(divisors), divisors.numel(), int(y_exp), _ptr(out),
                                            out.data_ptr() + 8, _stream(stream)),
           "convrot_test_unscale_sweep")
    n, first = (int(v) for v in out.cpu())
    if n == 0:
        return 0, None
    first &= (1 << 64) - 1
    d = float(divisors[first >> 32].item())
    y = struct.unpack("<f", struct.pack("<I", first & 0xffffffff))[0]
    return n, (d, y)


def convrot_test_handover_timeout(Q_x16: torch.Tensor, s_x: torch.Tensor, q16s, scales, biases, wait_ns: int,
                                  workspace: torch.Tensor, Ys=None, stream=None):
    """Test-only GEMM launch whose split-tile hand-over waits can never be
    satisfied and give up after wait_ns: the kernel records CONVROT_ERR_TIMEOUT
    (read it with convrot_device_status) and exits, leaving those tiles of Ys
    unfinished. Returns Ys."""
    _need(Q_x16, torch.float16, "Q_x16")
    _need(s_x, torch.float32, "s_x")
    M, K = Q_x16.shape
    if Ys is None:
        Ys = [torch.empty((M, q.shape[0]), dtype=torch.float32, device=Q_x16.device) for q in q16s]
    weights = make_weights(q16s, scales, biases, Ys)
    _check(lib().convrot_test_handover_timeout(_ptr(Q_x16), _ptr(s_x), M, K, weights, len(q16s), _ptr(workspace),
                                               workspace.numel() * workspace.element_size(), int(wait_ns),
                                               _stream(stream)),
           "convrot_test_handover_timeout")
    return Ys


def convrot_linear_swiglu(X: torch.Tensor, G: int, gate: Tuple, up: Tuple, H: Optional[torch.Tensor] = None,
                          workspace=None, stream=None) -> torch.Tensor:
    """Split SwiGLU of two linears sharing X: h = silu(gate) * up, where gate
    and up are (q16, scale, bias, kchunk) tuples with the same N; one pack and
    one GEMM whose epilogue writes only h (fp32 [M, N])."""
    xd = _xdtype(X)
    _need(X, X.dtype, "X")
    M, K = X.shape
    N = gate[0].shape[0]
    if H is None:
        H = torch.empty((M, N), dtype=torch.float32, device=X.device)
    _need(H, torch.float32, "H")
    w = make_weights([gate[0], up[0]], [gate[1], up[1]], [gate[2], up[2]], [H, H], [gate[3], up[3]])
    ws = _workspace(convrot_linear_workspace_size(M, K), X.device, workspace)
    _check(lib().convrot_linear_swiglu(_ptr(X), xd, M, K, G, w, _ptr(ws), ws.numel(), _stream(stream)),
           "convrot_linear_swiglu")
    return H


# ---------------------------------------------------------------------------
# block norms and 8-bit floating-point linears
#
# A single token's calls take a few microseconds on the GPU, so the checks
# here are written to cost little: one condition per tensor, its description
# formed only for a refusal, and the argument structs packed in one go.
# ---------------------------------------------------------------------------

_DTYPES = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_E4M3 = torch.float8_e4m3fn
_F32 = torch.float32
# convrot_block_norm_args and convrot_fp8_weight as the C compiler lays them out
_NORM_ARGS = struct.Struct("@qqiiPPqqffiiffPPPPPPPqqqPqPPqqPP")
_FP8_WEIGHTS = [None] + [struct.Struct("@" + "PPPqPq" * n) for n in range(1, MAX_LINEARS + 1)]
assert _NORM_ARGS.size == ctypes.sizeof(convrot_block_norm_args)
assert _FP8_WEIGHTS[2].size == 2 * ctypes.sizeof(convrot_fp8_weight)


def _start(t: torch.Tensor, stream):
    """(device, stream handle) of a call whose first input is t."""
    device = t.get_device()
    if device < 0:
        raise ValueError("the inputs must be CUDA tensors")
    if device != torch.cuda.current_device():
        raise ValueError("the inputs must be on the current CUDA device")
    if stream is None:
        return device, torch._C._cuda_getCurrentRawStream(device)
    return device, stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _empty(shape, dtype, device: int, stream) -> torch.Tensor:
    """Memory that belongs to the call's stream, so that neither its earlier
    nor its later use elsewhere overlaps the call."""
    dev = torch.device("cuda", device)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream, dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _rows(t: torch.Tensor, name: str, device: int, shape, dtype=None) -> int:
    """Checks a matrix whose rows are contiguous (of a float type, or dtype);
    the distance between them."""
    if t.get_device() != device or t.shape != shape or (t.dtype not in _DTYPES if dtype is None else t.dtype is not dtype):
        raise ValueError(f"{name} must be a {dtype or 'float32, float16 or bfloat16'} matrix of shape {tuple(shape)} "
                         f"on the device of the other tensors, got {t.dtype} {tuple(t.shape)}")
    M, K = shape
    if t.is_contiguous():
        return K
    ld, inner = t.stride()
    if inner != 1 and K > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if M <= 1 or K == 0:
        return K
    if ld < K:
        raise ValueError(f"the rows of {name} overlap")
    return ld


def _dense(t: torch.Tensor, name: str, device: int, shape, dtype) -> int:
    """Checks a contiguous array of a given shape and type; its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the device of the "
                         f"other tensors, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _matrix(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    return t.shape


def _n_blocks(n: int) -> int:
    return (n + FP8_BLOCK - 1) // FP8_BLOCK


def fp8_pack_activations(X: torch.Tensor, Q_x: Optional[torch.Tensor] = None, s_x: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """X [M,K] (float32, float16 or bfloat16, rows contiguous) -> (Q_x
    float8_e4m3fn [M,K], s_x float32 [M, ceil(K/128)])."""
    device, handle = _start(X, stream)
    M, K = shape = _matrix(X, "X")
    ldx = _rows(X, "X", device, shape)
    kb = (M, _n_blocks(K))
    if Q_x is None:
        Q_x = _empty(shape, _E4M3, device, stream)
    if s_x is None:
        s_x = _empty(kb, _F32, device, stream)
    _check(lib().fp8_pack_activations(X.data_ptr(), _DTYPES[X.dtype], M, K, ldx,
                                      _dense(Q_x, "Q_x", device, shape, _E4M3), _dense(s_x, "s_x", device, kb, _F32),
                                      handle), "fp8_pack_activations")
    return Q_x, s_x


def fp8_prepare_weight(W: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Offline weight path: W [N,K] (float32, float16 or bfloat16) -> (Q_w
    float8_e4m3fn [N,K], s_w float32 [ceil(N/128), ceil(K/128)])."""
    device, handle = _start(W, stream)
    N, K = shape = _matrix(W, "W")
    if _rows(W, "W", device, shape) != K:
        raise ValueError("W must be contiguous")
    Q_w = _empty(shape, _E4M3, device, stream)
    s_w = _empty((_n_blocks(N), _n_blocks(K)), _F32, device, stream)
    _check(lib().fp8_prepare_weight(W.data_ptr(), _DTYPES[W.dtype], N, K, Q_w.data_ptr(), s_w.data_ptr(), handle),
           "fp8_prepare_weight")
    return Q_w, s_w


def _fp8_weights(device: int, stream, M: int, K: int, qs, scales, biases, Ys, out_dtype):
    """(descriptors, outputs, y_dtype) of an fp8 linear call."""
    n = len(qs)
    if not 1 <= n <= MAX_LINEARS or len(scales) != n or (biases is not None and len(biases) != n) or \
            (Ys is not None and len(Ys) != n):
        raise ValueError(f"1 to {MAX_LINEARS} weights, with as many scales, biases and outputs")
    if Ys is None:
        Ys = [_empty((M, q.shape[0]), out_dtype, device, stream) for q in qs]
    y_dtype = Ys[0].dtype
    kb = _n_blocks(K)
    d = []
    for j in range(n):
        q, b, y = qs[j], None if biases is None else biases[j], Ys[j]
        N = q.shape[0]
        d += (_dense(q, "a weight", device, (N, K), _E4M3),
              _dense(scales[j], "a weight's scales", device, (_n_blocks(N), kb), _F32),
              0 if b is None else _dense(b, "a bias", device, (N,), _F32), N, y.data_ptr(),
              _rows(y, "an output", device, (M, N)))
        if y.dtype is not y_dtype:
            raise ValueError("the outputs of one call have one type")
    return _FP8_WEIGHTS[n].pack(*d), Ys, _DTYPES[y_dtype]


def fp8_linear_packed(Q_x: torch.Tensor, s_x: torch.Tensor, qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
                      biases: Optional[Sequence[Optional[torch.Tensor]]] = None,
                      Ys: Optional[List[torch.Tensor]] = None, out_dtype: torch.dtype = torch.bfloat16,
                      stream=None) -> List[torch.Tensor]:
    """Every Y_j = X W_j^T + b_j on an activation packed by
    fp8_pack_activations or convrot_block_norm_fp8; weights (codes `qs`,
    `scales`) from fp8_prepare_weight. Ys: outputs to write (float32, float16
    or bfloat16, rows contiguous), or new ones of out_dtype."""
    device, handle = _start(Q_x, stream)
    M, K = shape = _matrix(Q_x, "Q_x")
    q_ptr = _dense(Q_x, "Q_x", device, shape, _E4M3)
    s_ptr = _dense(s_x, "s_x", device, (M, _n_blocks(K)), _F32)
    weights, Ys, y_dtype = _fp8_weights(device, stream, M, K, qs, scales, biases, Ys, out_dtype)
    _check(lib().fp8_linear_packed(q_ptr, s_ptr, M, K, weights, len(Ys), y_dtype, handle), "fp8_linear_packed")
    return Ys


def fp8_linear_workspace_size(M: int, K: int) -> int:
    return int(lib().fp8_linear_workspace_size(M, K))


def fp8_linear(X: torch.Tensor, qs: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
               biases: Optional[Sequence[Optional[torch.Tensor]]] = None, Ys: Optional[List[torch.Tensor]] = None,
               out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> List[torch.Tensor]:
    """Pack X once (fp8_pack_activations), then every Y_j = X W_j^T + b_j as
    fp8_linear_packed. New outputs are of out_dtype (X's own by default)."""
    device, handle = _start(X, stream)
    M, K = shape = _matrix(X, "X")
    ldx = _rows(X, "X", device, shape)
    weights, Ys, y_dtype = _fp8_weights(device, stream, M, K, qs, scales, biases, Ys,
                                        X.dtype if out_dtype is None else out_dtype)
    ws = workspace
    if ws is None:
        ws = _empty((max(fp8_linear_workspace_size(M, K), 1),), torch.uint8, device, stream)
    elif ws.get_device() != device or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    _check(lib().fp8_linear(X.data_ptr(), _DTYPES[X.dtype], M, K, ldx, weights, len(Ys), y_dtype, ws.data_ptr(),
                            ws.numel() * ws.element_size(), handle), "fp8_linear")
    return Ys


def _n_samples(t: torch.Tensor, name: str, M: int) -> int:
    """The samples that a matrix of gates, scales or shifts is for: its rows.
    None for some rows of H would have no address, which says "absent"."""
    if t.dim() != 2 or (M and not t.shape[0]):
        raise ValueError(f"{name} must be a matrix with a row per sample, got {tuple(t.shape)}")
    return t.shape[0]


def _block_norm(H, Y, residual_scale, block_scale, post_norm, post_eps, post_weight, post_bias, gate, pre_norm,
                pre_eps, pre_weight, pre_bias, scale, shift, row_sample, rows_per_sample, H_out, U, u_dtype, ldu, Q, s,
                device, handle):
    """Checks what both forms of the block norm share and calls the library."""
    M, K = shape = H.shape
    dtype = H.dtype
    ldh = _rows(H, "H", device, shape)
    ldy = 0 if Y is None else _rows(Y, "Y", device, shape, dtype)
    ldho = 0 if H_out is None else _rows(H_out, "H_out", device, shape, dtype)
    vec = (K,)
    samples = ld_gate = ld_mod = 0
    if gate is not None:
        samples = _n_samples(gate, "gate", M)
        ld_gate = _rows(gate, "gate", device, (samples, K), _F32)
    if scale is not None:
        samples = samples or _n_samples(scale, "scale", M)
        ld_mod = _rows(scale, "scale", device, (samples, K), _F32)
    if shift is not None:
        samples = samples or _n_samples(shift, "shift", M)
        ld = _rows(shift, "shift", device, (samples, K), _F32)
        if scale is not None and ld != ld_mod:
            raise ValueError("scale and shift must have the same distance between rows")
        ld_mod = ld
    rows = 0
    if samples:
        if row_sample is not None:
            rows = _dense(row_sample, "row_sample", device, (M,), torch.int32)
        elif rows_per_sample == 0 and samples > 1:
            raise ValueError("several samples need row_sample or rows_per_sample")
    args = _NORM_ARGS.pack(
        M, K, _DTYPES[dtype], u_dtype, H.data_ptr(), 0 if Y is None else Y.data_ptr(), ldh, ldy, residual_scale,
        block_scale, post_norm, pre_norm, post_eps, pre_eps,
        0 if post_weight is None else _dense(post_weight, "post_weight", device, vec, _F32),
        0 if post_bias is None else _dense(post_bias, "post_bias", device, vec, _F32),
        0 if pre_weight is None else _dense(pre_weight, "pre_weight", device, vec, _F32),
        0 if pre_bias is None else _dense(pre_bias, "pre_bias", device, vec, _F32),
        0 if gate is None else gate.data_ptr(), 0 if scale is None else scale.data_ptr(),
        0 if shift is None else shift.data_ptr(), ld_gate, ld_mod, samples, rows, rows_per_sample,
        0 if H_out is None else H_out.data_ptr(), U, ldho, ldu, Q, s)
    _check(lib().convrot_block_norm(args, handle), "convrot_block_norm")


def convrot_block_norm(H: torch.Tensor, Y: Optional[torch.Tensor] = None, *, residual_scale: float = 1.0,
                       block_scale: float = 1.0, post_norm: int = NORM_NONE, post_eps: float = 1e-6, post_weight=None,
                       post_bias=None, gate=None, pre_norm: int = NORM_RMS, pre_eps: float = 1e-6, pre_weight=None,
                       pre_bias=None, scale=None, shift=None, row_sample=None, rows_per_sample: int = 0,
                       H_out: Optional[torch.Tensor] = None, U: Optional[torch.Tensor] = None,
                       u_dtype: Optional[torch.dtype] = None, want_h: bool = True, want_u: bool = True, stream=None):
    """The norms before and after a block with its gate and residual, one pass:
        h' = residual_scale H + gate * block_scale * post(Y),
        u = modulate(pre(h')),  modulate(u) = u + u * scale + shift.
    H, Y [M,K] (one type, rows contiguous); weights and biases float32 [K];
    gate, scale, shift float32 [samples, K], the row m taking the sample
    row_sample[m] (int32) or m // rows_per_sample. Returns (h', u): H_out and U
    where given (H_out may be H), new tensors where not (u of u_dtype, H's own
    by default), None for what want_h or want_u leaves out. The INT8 linears
    take a u of float16 or float32, the fp8 linears any."""
    device, handle = _start(H, stream)
    shape = _matrix(H, "H")
    if H_out is None and want_h:
        H_out = _empty(shape, H.dtype, device, stream)
    if U is None and want_u:
        U = _empty(shape, H.dtype if u_dtype is None else u_dtype, device, stream)
    ldu = 0 if U is None else _rows(U, "U", device, shape)
    _block_norm(H, Y, residual_scale, block_scale, post_norm, post_eps, post_weight, post_bias, gate, pre_norm,
                pre_eps, pre_weight, pre_bias, scale, shift, row_sample, rows_per_sample, H_out,
                0 if U is None else U.data_ptr(), 0 if U is None else _DTYPES[U.dtype], ldu, 0, 0, device, handle)
    return H_out, U


def convrot_block_norm_fp8(H: torch.Tensor, Y: Optional[torch.Tensor] = None, *, residual_scale: float = 1.0,
                           block_scale: float = 1.0, post_norm: int = NORM_NONE, post_eps: float = 1e-6,
                           post_weight=None, post_bias=None, gate=None, pre_norm: int = NORM_RMS,
                           pre_eps: float = 1e-6, pre_weight=None, pre_bias=None, scale=None, shift=None,
                           row_sample=None, rows_per_sample: int = 0, H_out: Optional[torch.Tensor] = None,
                           Q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None, want_h: bool = True,
                           stream=None):
    """convrot_block_norm with u quantized as it is formed: returns (h', Q, s),
    Q float8_e4m3fn [M,K] and s float32 [M, ceil(K/128)] as
    fp8_pack_activations gives them, for fp8_linear_packed."""
    device, handle = _start(H, stream)
    M, K = shape = _matrix(H, "H")
    kb = (M, _n_blocks(K))
    if H_out is None and want_h:
        H_out = _empty(shape, H.dtype, device, stream)
    if Q is None:
        Q = _empty(shape, _E4M3, device, stream)
    if s is None:
        s = _empty(kb, _F32, device, stream)
    _block_norm(H, Y, residual_scale, block_scale, post_norm, post_eps, post_weight, post_bias, gate, pre_norm,
                pre_eps, pre_weight, pre_bias, scale, shift, row_sample, rows_per_sample, H_out, 0, 0, 0,
                _dense(Q, "Q", device, shape, _E4M3), _dense(s, "s", device, kb, _F32), device, handle)
    return H_out, Q, s


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

_ROUTE_ARGS = struct.Struct("@qiiiiPqPiiiifPP")
_EXPERTS = struct.Struct("@PPPqqqq")
_MOE_ARGS = struct.Struct("@PiqqqPPiiPPPPqPqi0q")
assert _ROUTE_ARGS.size == ctypes.sizeof(convrot_moe_route_args)
assert _EXPERTS.size == ctypes.sizeof(convrot_experts)
assert _MOE_ARGS.size == ctypes.sizeof(convrot_moe_args)


def moe_route(logits: torch.Tensor, top_k: int, *, score: int = MOE_SOFTMAX, bias: Optional[torch.Tensor] = None,
              n_groups: int = 1, top_groups: int = 1, group_top: int = 2, renormalise: bool = True,
              scale: float = 1.0, experts: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
              stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Router logits [T,E] (float32, float16 or bfloat16, rows contiguous) ->
    (experts int32 [T,top_k], weights float32 [T,top_k]): the top_k largest of
    score(logits) + bias in the best top_groups of n_groups groups of experts,
    equal ones in the order of their index, weighted by their scores (without
    the bias). Logits of -inf close an expert; slots that no open expert fills
    get expert -1 and weight 0."""
    device, handle = _start(logits, stream)
    T, E = shape = _matrix(logits, "logits")
    ld = _rows(logits, "logits", device, shape)
    out = (T, top_k)
    if experts is None:
        experts = _empty(out, torch.int32, device, stream)
    if weights is None:
        weights = _empty(out, _F32, device, stream)
    args = _ROUTE_ARGS.pack(T, E, top_k, _DTYPES[logits.dtype], score, logits.data_ptr(), ld,
                            0 if bias is None else _dense(bias, "bias", device, (E,), _F32), n_groups, top_groups,
                            group_top, 1 if renormalise else 0, scale,
                            _dense(experts, "experts", device, out, torch.int32),
                            _dense(weights, "weights", device, out, _F32))
    _check(lib().moe_route(args, handle), "moe_route")
    return experts, weights


def moe_plan_workspace_size(n: int, n_experts: int) -> int:
    return int(lib().moe_plan_workspace_size(n, n_experts))


def _bytes(workspace, size: int, device: int, stream):
    """(address, size) of a workspace of at least `size` bytes: the given one, or
    a new one where some is needed (returned third, to be kept for the call)."""
    if workspace is not None:
        if workspace.get_device() != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the device of the other tensors")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if size == 0:
        return 0, 0, None
    ws = _empty(size, torch.uint8, device, stream)
    return ws.data_ptr(), size, ws


def moe_plan(experts: torch.Tensor, n_experts: int, order: Optional[torch.Tensor] = None,
             place: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None):
    """The choices (int32, of any shape) sorted by expert: (order, place,
    offsets), int32. order[i] is the choice of row i (-1 behind the last one),
    place[c] the row of choice c (-1 for none), and expert e has the rows from
    offsets[e] to offsets[e + 1]."""
    device, handle = _start(experts, stream)
    n, i32 = experts.numel(), torch.int32
    if order is None:
        order = _empty((n,), i32, device, stream)
    if place is None:
        place = _empty((n,), i32, device, stream)
    if offsets is None:
        offsets = _empty((n_experts + 1,), i32, device, stream)
    ws, size, keep = _bytes(workspace, moe_plan_workspace_size(n, n_experts), device, stream)
    _check(lib().moe_plan(_dense(experts, "experts", device, experts.shape, i32), n, n_experts,
                          _dense(order, "order", device, (n,), i32), _dense(place, "place", device, (n,), i32),
                          _dense(offsets, "offsets", device, (n_experts + 1,), i32), ws, size, handle), "moe_plan")
    return order, place, offsets


def fp8_prepare_experts(W: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """fp8_prepare_weight of every expert's matrix W[e], W [E,N,K]: (Q
    float8_e4m3fn [E,N,K], s float32 [E, ceil(N/128), ceil(K/128)])."""
    device, handle = _start(W, stream)
    if W.dim() != 3 or W.dtype not in _DTYPES or not W.is_contiguous():
        raise ValueError("W must be a contiguous float32, float16 or bfloat16 tensor [experts, N, K]")
    E, N, K = W.shape
    Q = _empty((E, N, K), _E4M3, device, stream)
    s = _empty((E, _n_blocks(N), _n_blocks(K)), _F32, device, stream)
    for e in range(E):
        _check(lib().fp8_prepare_weight(W[e].data_ptr(), _DTYPES[W.dtype], N, K, Q[e].data_ptr(), s[e].data_ptr(),
                                        handle), "fp8_prepare_weight")
    return Q, s


def _per_expert(t: torch.Tensor, name: str, what: str, device: int, shape, dtype) -> Tuple[int, int]:
    """(address, distance between experts) of an array whose part of every
    expert is dense."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device:
        step = 1
        for s in shape[1:]:
            step *= s
        if t.is_contiguous():
            return t.data_ptr(), step
        if shape[0] == 0 or t[0].is_contiguous():
            return t.data_ptr(), t.stride(0) if shape[0] > 1 else step
    raise ValueError(f"{name}: {what} must be {dtype} of shape {tuple(shape)} on the device of the other tensors, dense "
                     f"for every expert, got {t.dtype} {tuple(t.shape)}")


def _experts(w, name: str, device: int, K: int, E: Optional[int] = None):
    """(descriptor, E, N) of a set of experts' matrices: a tuple of codes
    [E,N,K], scales [E, ceil(N/128), ceil(K/128)] and, or None, biases [E,N].
    An expert's own part is dense; the experts may be further apart."""
    q, s, b = w if len(w) == 3 else (*w, None)
    if q.dim() != 3:
        raise ValueError(f"{name}: the codes must have the shape (experts, N, K)")
    n, N, _ = q.shape
    if E is not None and n != E:
        raise ValueError(f"{name}: {n} experts, and {E} elsewhere in the call")
    q_ptr, q_stride = _per_expert(q, name, "codes", device, (n, N, K), _E4M3)
    s_ptr, s_stride = _per_expert(s, name, "scales", device, (n, _n_blocks(N), _n_blocks(K)), _F32)
    b_ptr, b_stride = (0, N) if b is None else _per_expert(b, name, "biases", device, (n, N), _F32)
    return _EXPERTS.pack(q_ptr, s_ptr, b_ptr, N, q_stride, s_stride, b_stride), n, N


def _plan_of(Q_x, s_x, order, offsets, E: int, device: int):
    """(T, K, n, addresses of Q_x, s_x, order and offsets) of an expert linear."""
    T, K = shape = _matrix(Q_x, "Q_x")
    n = T if order is None else order.numel()
    return (T, K, n, _dense(Q_x, "Q_x", device, shape, _E4M3), _dense(s_x, "s_x", device, (T, _n_blocks(K)), _F32),
            0 if order is None else _dense(order, "order", device, (n,), torch.int32),
            _dense(offsets, "offsets", device, (E + 1,), torch.int32))


def fp8_expert_workspace_size(n: int, K: int, n_experts: int) -> int:
    return int(lib().fp8_expert_workspace_size(n, K, n_experts))


def fp8_expert_linear(Q_x: torch.Tensor, s_x: torch.Tensor, offsets: torch.Tensor, weight,
                      order: Optional[torch.Tensor] = None, top_k: int = 1, Y: Optional[torch.Tensor] = None,
                      out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Rows in the order of a moe_plan, each through its expert's matrix:
    Y[i] = X[m] W_e^T + b_e, with m = i, or, given the plan's order,
    m = order[i] // top_k (an order of more than T * top_k rows is refused).
    weight: (codes [E,N,K], scales, biases or None) as fp8_prepare_experts gives
    them. Rows from offsets[E] on are left as they are (in a new Y:
    uninitialised)."""
    device, handle = _start(Q_x, stream)
    w, E, N = _experts(weight, "weight", device, _matrix(Q_x, "Q_x")[1])
    T, K, n, q, s, o, f = _plan_of(Q_x, s_x, order, offsets, E, device)
    if Y is None:
        Y = _empty((n, N), out_dtype, device, stream)
    ldy = _rows(Y, "Y", device, (n, N))
    ws, size, keep = _bytes(workspace, 0 if order is None else fp8_expert_workspace_size(n, K, E), device, stream)
    _check(lib().fp8_expert_linear(q, s, T, K, o, f, n, E, top_k, w, Y.data_ptr(), ldy, _DTYPES[Y.dtype], ws, size,
                                   handle), "fp8_expert_linear")
    return Y


def fp8_expert_swiglu(Q_x: torch.Tensor, s_x: torch.Tensor, order: Optional[torch.Tensor], offsets: torch.Tensor,
                      top_k: int, gate, up, Q_h: Optional[torch.Tensor] = None, s_h: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The rows of a moe_plan through their expert's gate and up matrices (as
    fp8_expert_linear, order and top_k included): h = silu(gate) * up, quantized
    as it leaves to (Q_h float8_e4m3fn [n,N], s_h float32 [n, ceil(N/128)]),
    which an fp8_expert_linear without order reads."""
    device, handle = _start(Q_x, stream)
    K = _matrix(Q_x, "Q_x")[1]
    g, E, N = _experts(gate, "gate", device, K)
    u, _, N_up = _experts(up, "up", device, K, E)
    if N_up != N:
        raise ValueError("gate and up must have the same output features")
    T, K, n, q, s, o, f = _plan_of(Q_x, s_x, order, offsets, E, device)
    if Q_h is None:
        Q_h = _empty((n, N), _E4M3, device, stream)
    if s_h is None:
        s_h = _empty((n, _n_blocks(N)), _F32, device, stream)
    ws, size, keep = _bytes(workspace, 0 if order is None else fp8_expert_workspace_size(n, K, E), device, stream)
    _check(lib().fp8_expert_swiglu(q, s, T, K, o, f, n, E, top_k, g, u, _dense(Q_h, "Q_h", device, (n, N), _E4M3),
                                   _dense(s_h, "s_h", device, (n, _n_blocks(N)), _F32), ws, size, handle),
           "fp8_expert_swiglu")
    return Q_h, s_h


def fp8_test_expert_timeout(Q_x: torch.Tensor, s_x: torch.Tensor, offsets: torch.Tensor, weight, wait_ns: int,
                            Y: torch.Tensor, up=None, s_h: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Test-only launch of an expert linear (SwiGLU with `up`: Y are codes, s_h
    their scales) on rows in the plan's order, whose last tile is not loaded to its
    end: the kernel's waits give up after wait_ns, it records ERR_TIMEOUT (read it
    with convrot_device_status) and leaves that tile unwritten."""
    device, handle = _start(Q_x, stream)
    w, E, N = _experts(weight, "weight", device, _matrix(Q_x, "Q_x")[1])
    n, K, _, q, s, _, f = _plan_of(Q_x, s_x, None, offsets, E, device)
    u = None if up is None else _experts(up, "up", device, K, E)[0]
    y = _dense(Y, "Y", device, (n, N), Y.dtype if up is None else _E4M3)
    _check(lib().fp8_test_expert_timeout(q, s, n, K, f, E, w, u, y,
                                         0 if s_h is None else _dense(s_h, "s_h", device, (n, _n_blocks(N)), _F32), N,
                                         F32 if up is not None else _DTYPES[Y.dtype], int(wait_ns), handle),
           "fp8_test_expert_timeout")
    return Y


def moe_combine(rows: torch.Tensor, place: torch.Tensor, weights: torch.Tensor,
                residual: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """Y[t] = residual[t] + sum_j weights[t,j] rows[place[t,j]]: rows [n,N],
    place int32 and weights float32 [T,top_k] (place of any shape with as many
    elements). New outputs are of out_dtype (rows' own by default; a residual
    has the type of Y, and may be Y)."""
    device, handle = _start(rows, stream)
    n, N = shape = _matrix(rows, "rows")
    T, top_k = _matrix(weights, "weights")
    if place.numel() != T * top_k:
        raise ValueError(f"place must have {T * top_k} elements, got {place.numel()}")
    if Y is None:
        Y = _empty((T, N), out_dtype or (rows.dtype if residual is None else residual.dtype), device, stream)
    ldr = _rows(rows, "rows", device, shape)
    ldy = _rows(Y, "Y", device, (T, N))
    res, ld_res = (0, N) if residual is None else (residual.data_ptr(),
                                                   _rows(residual, "residual", device, (T, N), Y.dtype))
    _check(lib().moe_combine(rows.data_ptr(), _DTYPES[rows.dtype], ldr, n,
                             _dense(place, "place", device, place.shape, torch.int32),
                             _dense(weights, "weights", device, (T, top_k), _F32), T, top_k, N, res, ld_res,
                             Y.data_ptr(), ldy, _DTYPES[Y.dtype], handle), "moe_combine")
    return Y


def fp8_moe_workspace_size(T: int, K: int, inner: int, N: int, top_k: int, n_experts: int,
                           out_dtype: torch.dtype = torch.bfloat16) -> int:
    return int(lib().fp8_moe_workspace_size(T, K, inner, N, top_k, n_experts, _DTYPES[out_dtype]))


def fp8_moe(X: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor, gate, up, down,
            residual: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
            out_dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """Y[t] = residual[t] + sum_j weights[t,j] down_e(silu(gate_e(x_t)) * up_e(x_t)),
    e = experts[t,j] (moe_route's results; -1 adds nothing): X [T,K] (float32,
    float16 or bfloat16, rows contiguous) is packed, the choices are sorted by
    expert, and the experts' linears, SwiGLU and the weighted sum follow. gate,
    up, down: (codes, scales, biases or None) as fp8_prepare_experts gives them,
    of matrices [I,K], [I,K] and [N,I]. New outputs are of out_dtype (X's own by
    default); a residual has the type of Y, and may be Y. For a bfloat16 Y the
    experts' rows pass to the sum in binary16, scaled per 128 features."""
    device, handle = _start(X, stream)
    T, K = shape = _matrix(X, "X")
    ldx = _rows(X, "X", device, shape)
    g, E, inner = _experts(gate, "gate", device, K)
    u, _, inner_up = _experts(up, "up", device, K, E)
    if inner_up != inner:
        raise ValueError("gate and up must have the same output features")
    d, _, N = _experts(down, "down", device, inner, E)
    top_k = _matrix(experts, "experts")[1]
    if Y is None:
        Y = _empty((T, N), out_dtype or (X.dtype if residual is None else residual.dtype), device, stream)
    ldy = _rows(Y, "Y", device, (T, N))
    res, ld_res = (0, N) if residual is None else (residual.data_ptr(),
                                                   _rows(residual, "residual", device, (T, N), Y.dtype))
    ws, size, keep = _bytes(workspace, fp8_moe_workspace_size(T, K, inner, N, top_k, E, Y.dtype), device, stream)
    sets = ctypes.create_string_buffer(g + u + d)
    at = ctypes.addressof(sets)
    args = _MOE_ARGS.pack(X.data_ptr(), _DTYPES[X.dtype], T, K, ldx,
                          _dense(experts, "experts", device, (T, top_k), torch.int32),
                          _dense(weights, "weights", device, (T, top_k), _F32), top_k, E, at, at + _EXPERTS.size,
                          at + 2 * _EXPERTS.size, res, ld_res, Y.data_ptr(), ldy, _DTYPES[Y.dtype])
    _check(lib().fp8_moe(args, ws, size, handle), "fp8_moe")
    return Y
