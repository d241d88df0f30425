"""Norm-compensated 2:4 activation-sparse linear layer with a low-rank branch, on MI355X.

Thin Python binding of the C ABI in ``include/rtl.h`` (``librtl.so``, gfx950 HIP
kernels).  Every function here only marshals arguments: tensors stay on the GPU, the
work runs in the library's kernels on the current torch stream, and nothing falls back
to the CPU.  If the library is missing the import fails loudly; build it with
``python activation_sparse_gemm_amd/build.py``.  No call records an autograd graph, whatever its
inputs require: gradients are the ``_backward`` calls' and the caller's to chain.

Method: "RT-Lynx: Putting the GEMM Sparsity In a Right Way for Diffusion Models"
(summary page, method steps 1, 2 and 4):
    X~ = top-2-of-4 magnitudes of X,  s = ||X|| / (||X~|| + eps),
    Y  = s * (X~ W^T) + (X L_B^T) L_A^T.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

try:  # the allocation alone, without torch.empty_strided's parsing of arguments and dispatch (half the
    # time): every element of these tensors is written, so deterministic mode's fill is not missed
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_cuda
except ImportError:
    def _empty_cuda(shape, stride, dtype):
        return torch.empty_strided(shape, stride, dtype=dtype, device="cuda")

__all__ = [
    "RTL_F32", "RTL_BF16", "RTL_TIE_LOWER_INDEX", "EPS", "RtlError", "lib", "library_path",
    "rtl_sparsify", "rtl_linear_fused", "rtl_linear_fused_workspace_bytes", "rtl_linear_fused_ex",
    "rtl_linear_fused_prep", "rtl_linear_fused_main", "rtl_linear_fused_noalloc", "rtl_linear_dense_ref",
    "RTL_NOALLOC_SCRATCH_BYTES", "rtl_mlp_fused", "rtl_mlp_fused_workspace_bytes", "RTL_MLP_AUTO",
    "RTL_MLP_PRODUCER", "RTL_MLP_CONSUMER", "RTL_VARIANT_AUTO", "RTL_VARIANT_PROLOGUE", "RTL_VARIANT_PRECOMPRESSED",
    "RTL_VARIANT_STREAM_K",
    "rtl_status_string", "rtl_version",
    "rtl_quantize_weight_fp8", "rtl_linear_fused_fp8", "rtl_linear_fused_fp8_workspace_bytes",
    "RTL_ROPE_ADJACENT", "RTL_ROPE_HALVES", "rtl_rope_axes", "rtl_qk_norm_rope", "rtl_qk_norm_rope_backward",
    "rtl_qk_norm_rope_backward_workspace_bytes",
    "RTL_ACT_SILU", "RTL_ACT_GELU", "rtl_glu_fused", "rtl_glu_backward", "rtl_glu_backward_workspace_bytes",
    "RTL_REST_KEPT", "RTL_REST_ZEROS", "rtl_layer_norm", "rtl_layer_norm_backward",
    "rtl_layer_norm_backward_workspace_bytes",
    "rtl_adapters_plan", "rtl_adapters_plan_bytes", "rtl_adapters", "rtl_adapters_workspace_bytes",
    "rtl_adapters_backward", "rtl_adapters_backward_workspace_bytes",
    "RTL_STATES_8", "RTL_STATES_32", "AdamWTensors", "rtl_adamw_tensors", "rtl_adamw",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# RTL_LIBRARY selects another build of the same library (e.g. one with sanitized host code).
library_path = os.environ.get("RTL_LIBRARY") or os.path.join(_PKG, "librtl.so")

RTL_F32, RTL_BF16 = 0, 1
RTL_TIE_LOWER_INDEX = 0
RTL_VARIANT_AUTO, RTL_VARIANT_PROLOGUE, RTL_VARIANT_PRECOMPRESSED, RTL_VARIANT_STREAM_K = 0, 1, 2, 3
EPS = 1e-8
RTL_NOALLOC_SCRATCH_BYTES = 192 << 20  # include/rtl.h
RTL_MLP_AUTO, RTL_MLP_PRODUCER, RTL_MLP_CONSUMER = 0, 1, 2
RTL_ROPE_ADJACENT, RTL_ROPE_HALVES = 0, 1
RTL_ACT_SILU, RTL_ACT_GELU = 0, 1
RTL_STATES_8, RTL_STATES_32 = 8, 32
RTL_REST_KEPT, RTL_REST_ZEROS = 0, 1
STATUS = {0: "RTL_OK", 1: "RTL_ERR_NULL", 2: "RTL_ERR_SHAPE", 3: "RTL_ERR_ALIGN", 4: "RTL_ERR_UNSUPPORTED",
          5: "RTL_ERR_ARG", 6: "RTL_ERR_WORKSPACE", 7: "RTL_ERR_HIP"}

# Every entry point include/rtl.h declares.
EXPORTS = ["rtl_sparsify", "rtl_linear_fused_workspace_bytes", "rtl_linear_fused", "rtl_linear_fused_ex",
           "rtl_linear_fused_prep", "rtl_linear_fused_main", "rtl_linear_fused_noalloc", "rtl_linear_dense_ref",
           "rtl_mlp_fused_workspace_bytes", "rtl_mlp_fused", "rtl_quantize_weight_fp8",
           "rtl_linear_fused_fp8_workspace_bytes", "rtl_linear_fused_fp8", "rtl_rope_axes", "rtl_qk_norm_rope",
           "rtl_qk_norm_rope_backward_workspace_bytes", "rtl_qk_norm_rope_backward", "rtl_glu_fused",
           "rtl_glu_backward_workspace_bytes", "rtl_glu_backward", "rtl_layer_norm", "rtl_layer_norm_ex",
           "rtl_layer_norm_backward_workspace_bytes", "rtl_layer_norm_backward", "rtl_layer_norm_backward_ex",
           "rtl_adapters_plan_bytes",
           "rtl_adapters_plan", "rtl_adapters_workspace_bytes", "rtl_adapters",
           "rtl_adapters_backward_workspace_bytes", "rtl_adapters_backward", "rtl_adamw", "rtl_status_string",
           "rtl_last_error", "rtl_version"]


class RtlError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class _AdamWTensor(ctypes.Structure):
    """rtl_adamw_tensor of include/rtl.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "master", "m", "v", "m_scale", "v_scale")] + [("n", ctypes.c_int64)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(library_path):
        raise ImportError(f"{library_path} is missing: build it with `python activation_sparse_gemm_amd/build.py`")
    L = ctypes.CDLL(library_path)
    p, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.rtl_sparsify.argtypes = [i32, i64, i64, p, i32, f32, p, p, p, p]
    L.rtl_sparsify.restype = i32
    L.rtl_linear_fused_workspace_bytes.argtypes = [i32, i64, i64, i64, i64]
    L.rtl_linear_fused_workspace_bytes.restype = sz
    L.rtl_linear_fused.argtypes = [i32, i64, i64, i64, i64, p, p, p, p, i32, f32, p, p, sz, p, p, p]
    L.rtl_linear_fused.restype = i32
    L.rtl_linear_fused_ex.argtypes = [i32, i32, i64, i64, i64, i64, p, p, p, p, i32, f32, p, p, sz, p, p, p]
    L.rtl_linear_fused_ex.restype = i32
    L.rtl_linear_fused_prep.argtypes = [i32, i32, i64, i64, i64, i64, p, p, i32, f32, p, sz, p, p, p]
    L.rtl_linear_fused_prep.restype = i32
    L.rtl_linear_fused_main.argtypes = [i32, i32, i64, i64, i64, i64, p, p, p, i32, f32, p, p, sz, p, p, p]
    L.rtl_linear_fused_main.restype = i32
    L.rtl_linear_fused_noalloc.argtypes = [i32, i64, i64, i64, i64, p, p, p, p, i32, f32, p, p, p, p]
    L.rtl_linear_fused_noalloc.restype = i32
    L.rtl_mlp_fused_workspace_bytes.argtypes = [i64, i64, i64, i64, i64, i64]
    L.rtl_mlp_fused_workspace_bytes.restype = sz
    L.rtl_mlp_fused.argtypes = [i32, i32, i64, i64, i64, i64, i64, i64, p, p, p, p, p, p, p, i32, f32, p, p, sz, p, p,
                                p, p]
    L.rtl_mlp_fused.restype = i32
    L.rtl_linear_dense_ref.argtypes = [i32, i64, i64, i64, p, p, p, p]
    L.rtl_linear_dense_ref.restype = i32
    L.rtl_quantize_weight_fp8.argtypes = [i64, i64, p, p, p, p]
    L.rtl_quantize_weight_fp8.restype = i32
    L.rtl_linear_fused_fp8_workspace_bytes.argtypes = [i64, i64, i64, i64]
    L.rtl_linear_fused_fp8_workspace_bytes.restype = sz
    L.rtl_linear_fused_fp8.argtypes = [i64, i64, i64, i64, p, p, p, p, p, i32, f32, p, p, sz, p, p, p]
    L.rtl_linear_fused_fp8.restype = i32
    f64, dims = ctypes.c_double, ctypes.POINTER(ctypes.c_int32)
    heads = [p, i64, i64]  # pointer, row stride, head stride
    rope = [p, i32, dims, f64, i32]  # pos, n_axes, axis_dims, theta, pairs
    L.rtl_rope_axes.argtypes = [i32, i64, i64, i64, *heads, *rope, i32, *heads, p]
    L.rtl_rope_axes.restype = i32
    L.rtl_qk_norm_rope.argtypes = [i32, i64, i64, i64, i64, *heads, *heads, p, p, f32, *rope, *heads, *heads, p]
    L.rtl_qk_norm_rope.restype = i32
    L.rtl_qk_norm_rope_backward_workspace_bytes.argtypes = [i64]
    L.rtl_qk_norm_rope_backward_workspace_bytes.restype = sz
    L.rtl_qk_norm_rope_backward.argtypes = [i32, i64, i64, i64, i64, *heads, *heads, p, p, f32, *rope, *heads, *heads,
                                            *heads, *heads, p, p, p, sz, p]
    L.rtl_qk_norm_rope_backward.restype = i32
    L.rtl_glu_fused.argtypes = [i32, i32, i64, i64, i64, p, p, p, p, p, p, p]
    L.rtl_glu_fused.restype = i32
    L.rtl_glu_backward_workspace_bytes.argtypes = [i64, i64, i64]
    L.rtl_glu_backward_workspace_bytes.restype = sz
    L.rtl_glu_backward.argtypes = [i32, i32, i64, i64, i64, p, p, p, p, p, p, p, p, p, p, sz, p]
    L.rtl_glu_backward.restype = i32
    rows = [p, i64]  # pointer, row stride
    L.rtl_layer_norm.argtypes = [i32, i64, i64, *rows, p, p, i64, p, *rows, *rows, f32, *rows, p, p]
    L.rtl_layer_norm_ex.argtypes = [i32, *L.rtl_layer_norm.argtypes]
    L.rtl_layer_norm.restype = L.rtl_layer_norm_ex.restype = i32
    L.rtl_layer_norm_backward_workspace_bytes.argtypes = [i64, i64, i64]
    L.rtl_layer_norm_backward_workspace_bytes.restype = sz
    L.rtl_layer_norm_backward.argtypes = [i32, i64, i64, *rows, p, *rows, p, p, i64, p, *rows, *rows, p, p, p, p, p, sz, p]
    L.rtl_layer_norm_backward_ex.argtypes = [i32, *L.rtl_layer_norm_backward.argtypes]
    L.rtl_layer_norm_backward.restype = L.rtl_layer_norm_backward_ex.restype = i32
    L.rtl_adapters_plan_bytes.argtypes = [i64, i64]
    L.rtl_adapters_plan_bytes.restype = sz
    L.rtl_adapters_plan.argtypes = [i64, i64, p, p, sz, p]
    L.rtl_adapters_plan.restype = i32
    for name in ("rtl_adapters_workspace_bytes", "rtl_adapters_backward_workspace_bytes"):
        getattr(L, name).argtypes = [i64] * 5
        getattr(L, name).restype = sz
    L.rtl_adapters.argtypes = [i32, i64, i64, i64, i64, i64, *rows, p, p, p, p, sz, *rows, *rows, p, p, sz, p]
    L.rtl_adapters.restype = i32
    L.rtl_adapters_backward.argtypes = [i32, i64, i64, i64, i64, i64, *rows, p, p, p, p, sz, p, *rows, *rows, *rows, p, p, p, sz,
                                        p]
    L.rtl_adapters_backward.restype = i32
    L.rtl_adamw.argtypes = [i32, i32, i32, i64, ctypes.POINTER(_AdamWTensor), i64, p, f64, p, f64, f64, f64, f64, p, p]
    L.rtl_adamw.restype = i32
    L.rtl_status_string.argtypes = [i32]
    L.rtl_status_string.restype = ctypes.c_char_p
    L.rtl_last_error.argtypes = []
    L.rtl_last_error.restype = ctypes.c_char_p
    L.rtl_version.argtypes = []
    L.rtl_version.restype = i32
    return L


lib = _load()


def rtl_status_string(status: int) -> str:
    return lib.rtl_status_string(status).decode()


def rtl_version() -> int:
    return lib.rtl_version()


def _check(status: int):
    if status != 0:
        raise RtlError(status, lib.rtl_last_error().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return RTL_F32
    if t.dtype == torch.bfloat16:
        return RTL_BF16
    raise TypeError(f"tensors must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _torch_stream(stream):
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream))


def _empty(shape, dtype, device, stream):
    """A tensor allocated on the stream the call runs on (torch's current stream when
    `stream` is None), so that torch's caching allocator does not give its memory to other
    work before that stream is done with it."""
    ts = _torch_stream(stream)
    if ts is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(ts):
        return torch.empty(shape, dtype=dtype, device=device)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def rtl_sparsify(X: torch.Tensor, tie: int = RTL_TIE_LOWER_INDEX, eps: float = EPS, vals=None, idx=None, s=None,
                 stream=None):
    """Selection, compression and rescale factor of every row of X [M,K].

    Returns (vals [M,K/2] X.dtype, idx [M,K/4] uint8, s [M] float32); outputs given by
    the caller are written in place."""
    M, K = X.shape
    if vals is None:
        vals = _empty((M, K // 2), X.dtype, X.device, stream)
    if idx is None:
        idx = _empty((M, K // 4), torch.uint8, X.device, stream)
    if s is None:
        s = _empty((M,), torch.float32, X.device, stream)
    _check(lib.rtl_sparsify(_dt(X), M, K, _ptr(X), tie, eps, _ptr(vals), _ptr(idx), _ptr(s), _stream(stream)))
    return vals, idx, s


def rtl_linear_fused_workspace_bytes(dtype: int, M: int, N: int, K: int, R: int) -> int:
    return int(lib.rtl_linear_fused_workspace_bytes(dtype, M, N, K, R))


def _workspace(dt, M, N, K, R, workspace, device, stream=None):
    need = rtl_linear_fused_workspace_bytes(dt, M, N, K, R)
    if workspace is None and need > 0:
        workspace = _empty((need,), torch.uint8, device, stream)
    return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())


def rtl_linear_fused(X: torch.Tensor, W: torch.Tensor, LA, LB, tie: int = RTL_TIE_LOWER_INDEX, eps: float = EPS,
                     Y=None, workspace=None, dbg_idx=None, dbg_s=None, stream=None,
                     variant: int = RTL_VARIANT_AUTO) -> torch.Tensor:
    """Y = s * (X~ W^T) + (X L_B^T) L_A^T.  X [M,K], W [N,K], LA [N,R], LB [R,K] (LA/LB None: R = 0).

    ``workspace`` (a uint8 tensor) is allocated when not given; pass one to keep the call
    free of allocations.  ``dbg_idx`` [M,K/4] uint8 and ``dbg_s`` [M] float32 receive the
    selection codes and s computed inside the kernels.  ``variant`` picks where the bf16
    path selects (RTL_VARIANT_*; rtl_linear_fused_ex in the C ABI)."""
    M, K = X.shape
    N = W.shape[0]
    R = 0 if LB is None else LB.shape[0]
    dt = _dt(X)
    if Y is None:
        Y = _empty((M, N), X.dtype, X.device, stream)
    workspace, ws_bytes = _workspace(dt, M, N, K, R, workspace, X.device, stream)
    _check(lib.rtl_linear_fused_ex(variant, dt, M, N, K, R, _ptr(X), _ptr(W), _ptr(LA), _ptr(LB), tie, eps, _ptr(Y),
                                   _ptr(workspace), ws_bytes, _ptr(dbg_idx), _ptr(dbg_s), _stream(stream)))
    return Y


def rtl_linear_fused_prep(X: torch.Tensor, LB, N: int, workspace: torch.Tensor, variant: int = RTL_VARIANT_AUTO,
                          tie: int = RTL_TIE_LOWER_INDEX, eps: float = EPS, dbg_idx=None, dbg_s=None, stream=None):
    """First launch of the bf16 layer: the pre-pass over X into ``workspace``."""
    M, K = X.shape
    R = 0 if LB is None else LB.shape[0]
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.rtl_linear_fused_prep(variant, _dt(X), M, N, K, R, _ptr(X), _ptr(LB), tie, eps, _ptr(workspace),
                                     ws_bytes, _ptr(dbg_idx), _ptr(dbg_s), _stream(stream)))


def rtl_linear_fused_main(X: torch.Tensor, W: torch.Tensor, LA, R: int, workspace: torch.Tensor,
                          variant: int = RTL_VARIANT_AUTO, tie: int = RTL_TIE_LOWER_INDEX, eps: float = EPS, Y=None,
                          dbg_idx=None, dbg_s=None, stream=None) -> torch.Tensor:
    """Second launch of the bf16 layer: the sparse-MFMA GEMM and its epilogue."""
    M, K = X.shape
    N = W.shape[0]
    if Y is None:
        Y = _empty((M, N), X.dtype, X.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.rtl_linear_fused_main(variant, _dt(X), M, N, K, R, _ptr(X), _ptr(W), _ptr(LA), tie, eps, _ptr(Y),
                                     _ptr(workspace), ws_bytes, _ptr(dbg_idx), _ptr(dbg_s), _stream(stream)))
    return Y


def rtl_linear_fused_noalloc(X: torch.Tensor, W: torch.Tensor, LA, LB, tie: int = RTL_TIE_LOWER_INDEX,
                             eps: float = EPS, Y=None, dbg_idx=None, dbg_s=None, stream=None) -> torch.Tensor:
    """rtl_linear_fused with the library's own per-GPU workspace (no allocation in the
    call; pass ``Y`` to keep the whole call allocation-free).  Calls that overlap on one
    GPU share that workspace and must be serialised by the caller."""
    M, K = X.shape
    N = W.shape[0]
    R = 0 if LB is None else LB.shape[0]
    if Y is None:
        Y = _empty((M, N), X.dtype, X.device, stream)
    _check(lib.rtl_linear_fused_noalloc(_dt(X), M, N, K, R, _ptr(X), _ptr(W), _ptr(LA), _ptr(LB), tie, eps, _ptr(Y),
                                        _ptr(dbg_idx), _ptr(dbg_s), _stream(stream)))
    return Y


def rtl_mlp_fused_workspace_bytes(M: int, K: int, H: int, N: int, Ru: int, Rd: int) -> int:
    return int(lib.rtl_mlp_fused_workspace_bytes(M, K, H, N, Ru, Rd))


def rtl_mlp_fused(X: torch.Tensor, Wu: torch.Tensor, LAu, LBu, Wd: torch.Tensor, LAd, LBd,
                  tie: int = RTL_TIE_LOWER_INDEX, eps: float = EPS, Y=None, workspace=None, dbg_xd=None,
                  dbg_idx=None, dbg_s=None, stream=None, variant: int = RTL_MLP_AUTO) -> torch.Tensor:
    """The MLP pair Y = layer_down(bf16(GELU(bf16(layer_up(X))))) in one call (bf16).

    X [M,K], Wu [H,K], LAu [H,Ru], LBu [Ru,K], Wd [N,H], LAd [N,Rd], LBd [Rd,H] (a layer's
    LA/LB None: rank 0).  ``dbg_xd`` [M,H] bf16, ``dbg_idx`` [M,H/4] uint8 and ``dbg_s`` [M]
    float32 receive the down layer's input, selection codes and s as the kernels formed them.
    ``variant``: RTL_MLP_PRODUCER (down operand from the up GEMM's epilogue), RTL_MLP_CONSUMER
    (GELU in the down layer's pre-pass) or RTL_MLP_AUTO."""
    M, K = X.shape
    H, N = Wu.shape[0], Wd.shape[0]
    Ru = 0 if LBu is None else LBu.shape[0]
    Rd = 0 if LBd is None else LBd.shape[0]
    if X.dtype != torch.bfloat16:
        raise TypeError("the MLP pair takes bf16 tensors")
    if Y is None:
        Y = _empty((M, N), X.dtype, X.device, stream)
    need = rtl_mlp_fused_workspace_bytes(M, K, H, N, Ru, Rd)
    if workspace is None:
        workspace = _empty((max(need, 1),), torch.uint8, X.device, stream)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check(lib.rtl_mlp_fused(variant, RTL_BF16, M, K, H, N, Ru, Rd, _ptr(X), _ptr(Wu), _ptr(LAu), _ptr(LBu), _ptr(Wd),
                             _ptr(LAd), _ptr(LBd), tie, eps, _ptr(Y), _ptr(workspace), ws_bytes, _ptr(dbg_xd),
                             _ptr(dbg_idx), _ptr(dbg_s), _stream(stream)))
    return Y


def rtl_linear_dense_ref(X: torch.Tensor, W: torch.Tensor, Y=None, stream=None) -> torch.Tensor:
    """Dense Y = X W^T with the fused kernel's tiling (the comparison layer)."""
    M, K = X.shape
    N = W.shape[0]
    if Y is None:
        Y = _empty((M, N), X.dtype, X.device, stream)
    _check(lib.rtl_linear_dense_ref(_dt(X), M, N, K, _ptr(X), _ptr(W), _ptr(Y), _stream(stream)))
    return Y


def rtl_quantize_weight_fp8(W: torch.Tensor, Wq=None, sw=None, stream=None):
    """E4M3 codes Wq [N,K] uint8 and per-output-row scales sw [N] float32 of bf16 W [N,K]."""
    N, K = W.shape
    if W.dtype != torch.bfloat16:
        raise TypeError("the FP8 layer takes bf16 weights")
    if Wq is None:
        Wq = _empty((N, K), torch.uint8, W.device, stream)
    if sw is None:
        sw = _empty((N,), torch.float32, W.device, stream)
    _check(lib.rtl_quantize_weight_fp8(N, K, _ptr(W), _ptr(Wq), _ptr(sw), _stream(stream)))
    return Wq, sw


def rtl_linear_fused_fp8_workspace_bytes(M: int, N: int, K: int, R: int) -> int:
    return int(lib.rtl_linear_fused_fp8_workspace_bytes(M, N, K, R))


def rtl_linear_fused_fp8(X: torch.Tensor, Wq: torch.Tensor, sw: torch.Tensor, LA, LB, tie: int = RTL_TIE_LOWER_INDEX,
                         eps: float = EPS, Y=None, workspace=None, dbg_xq=None, dbg_sx=None, stream=None) -> torch.Tensor:
    """FP8 layer Y = s sx sw (Xq~ Wq^T) + (X L_B^T) L_A^T.  X [M,K], LA [N,R], LB [R,K] bf16
    (LA/LB None: R = 0); Wq, sw from rtl_quantize_weight_fp8.  ``dbg_xq`` [M,K/2] uint8 and
    ``dbg_sx`` [M] float32 receive the activation codes and scales the kernels computed."""
    M, K = X.shape
    N = Wq.shape[0]
    R = 0 if LB is None else LB.shape[0]
    if X.dtype != torch.bfloat16:
        raise TypeError("the FP8 layer takes bf16 activations")
    if Y is None:
        Y = _empty((M, N), torch.bfloat16, X.device, stream)
    need = rtl_linear_fused_fp8_workspace_bytes(M, N, K, R)
    if workspace is None and need > 0:
        workspace = _empty((need,), torch.uint8, X.device, stream)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.rtl_linear_fused_fp8(M, N, K, R, _ptr(X), _ptr(Wq), _ptr(sw), _ptr(LA), _ptr(LB), tie, eps, _ptr(Y),
                                    _ptr(workspace), ws_bytes, _ptr(dbg_xq), _ptr(dbg_sx), _stream(stream)))
    return Y


def _elsewhere(first, *rest):
    """None if every given tensor is on the current GPU; if they are on another one, the context in
    which that is the current device, so that a call without ``stream`` runs on its current stream."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on one GPU, got {first.device} and {t.device}")
    if dev < 0:
        raise ValueError(f"tensors must be on one GPU, got {first.device}")
    return None if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _mismatch(name, t, shape, dtype):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _flat(name, t, shape, dtype):
    """Address of a contiguous tensor of `shape` and `dtype` (None: null)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype:
        _mismatch(name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


_NO_HEADS = None, 0, 0


def _heads(name, t, shape, dtype):
    """Address, row stride and head stride of a tensor of `shape` [M, H, D] and `dtype` whose
    channels are contiguous (None: null)."""
    if t is None:
        return _NO_HEADS
    if t.shape != shape or t.dtype is not dtype:
        _mismatch(name, t, shape, dtype)
    row, head, channel = t.stride()
    if channel != 1 and shape[2] > 1:
        raise ValueError("the channels of a head must be contiguous")
    return t.data_ptr(), row, head


def _space(t):
    """Address and bytes of a workspace."""
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _new(stream, like, shape, dtype):
    """A tensor on `like`'s device (the current one), as _empty allocates it."""
    if stream is not None:
        return _empty(shape, dtype, like.device, stream)
    n = len(shape)
    return _empty_cuda(shape, (shape[1] * shape[2], shape[2], 1) if n == 3 else (shape[1], 1) if n == 2 else (1,), dtype)


def _queue(stream, like):
    """The hipStream_t of `stream`, or of the current stream of `like`'s device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(like.get_device())
    return _stream(stream)


def _changed(given):
    """Counts outputs that the caller gave as changed (torch's in-place operations do), so that autograd
    refuses to use one that it kept for a backward pass."""
    for t in given:
        if t is not None:
            return torch.autograd.graph.increment_version([t for t in given if t is not None])


@functools.lru_cache(maxsize=64)
def _dims(axis_dims):
    if any(not 0 <= d < 2 ** 31 for d in axis_dims):
        raise ValueError(f"axis_dims must be whole numbers of channels, got {axis_dims}")
    return (ctypes.c_int32 * max(len(axis_dims), 1))(*axis_dims)


def _rope_args(pos, axis_dims, theta, pairs, M):
    dims = tuple(axis_dims)
    if not dims:
        return None, 0, _dims(dims), theta, pairs
    return _flat("pos", pos, (M, len(dims)), torch.float32), len(dims), _dims(dims), theta, pairs


def rtl_rope_axes(X: torch.Tensor, pos: torch.Tensor, axis_dims, theta: float = 10000.0,
                  pairs: int = RTL_ROPE_ADJACENT, inverse: bool = False, Y=None, stream=None) -> torch.Tensor:
    """X [M,H,D] (any row and head strides) turned by the positions ``pos`` [M, axes] float32.

    ``axis_dims`` holds the channels that each axis turns (even; their sum a multiple of 8, at
    most D).  ``pairs``: RTL_ROPE_ADJACENT pairs channels 2p and 2p + 1, RTL_ROPE_HALVES p and
    p + sum / 2.  ``inverse`` turns back, which is also the gradient.  ``Y`` may be X."""
    M, H, D = X.shape
    shape, dt = (M, H, D), X.dtype
    there = _elsewhere(X, pos, Y)
    if there is not None:
        with there:
            return rtl_rope_axes(X, pos, axis_dims, theta, pairs, inverse, Y, stream)
    given = (Y,)
    if Y is None:
        Y = _new(stream, X, shape, dt)
    _check(lib.rtl_rope_axes(_dt(X), M, H, D, *_heads("X", X, shape, dt),
                             *_rope_args(pos, axis_dims, theta, pairs, M), bool(inverse),
                             *_heads("Y", Y, shape, dt), _queue(stream, X)))
    _changed(given)
    return Y


def rtl_qk_norm_rope(Q: torch.Tensor, K, qw, kw, pos, axis_dims, theta: float = 10000.0, eps: float = 1e-6,
                     pairs: int = RTL_ROPE_ADJACENT, Qo=None, Ko=None, stream=None):
    """RMS norm of every head of Q [M,Hq,D] and K [M,Hk,D] (weights ``qw`` and ``kw`` [D], None:
    ones), then the rotation of rtl_rope_axes (``axis_dims`` empty: none), in one pass.  K None:
    queries only (``kw`` is not read).  Q and K may be views of a packed projection.  Returns (Qo, Ko); outputs given
    by the caller are written in place and may be Q and K."""
    M, Hq, D = Q.shape
    dt = Q.dtype
    qs, ks, ws = (M, Hq, D), (M, 0 if K is None else K.shape[1], D), (D,)
    there = _elsewhere(Q, K, qw, kw, pos if len(axis_dims) else None, Qo, Ko)
    if there is not None:
        with there:
            return rtl_qk_norm_rope(Q, K, qw, kw, pos, axis_dims, theta, eps, pairs, Qo, Ko, stream)
    given = Qo, Ko
    if Qo is None:
        Qo = _new(stream, Q, qs, dt)
    keys, keys_out, kw_at = _NO_HEADS, _NO_HEADS, None
    if K is not None:
        if Ko is None:
            Ko = _new(stream, Q, ks, dt)
        keys, keys_out, kw_at = _heads("K", K, ks, dt), _heads("Ko", Ko, ks, dt), _flat("kw", kw, ws, dt)
    elif Ko is not None:
        raise ValueError("Ko without K")
    _check(lib.rtl_qk_norm_rope(_dt(Q), M, Hq, ks[1], D, *_heads("Q", Q, qs, dt), *keys,
                                _flat("qw", qw, ws, dt), kw_at, eps,
                                *_rope_args(pos, axis_dims, theta, pairs, M), *_heads("Qo", Qo, qs, dt), *keys_out,
                                _queue(stream, Q)))
    _changed(given)
    return Qo, Ko


@functools.lru_cache(maxsize=64)
def rtl_qk_norm_rope_backward_workspace_bytes(D: int) -> int:
    return int(lib.rtl_qk_norm_rope_backward_workspace_bytes(D))


def rtl_qk_norm_rope_backward(Q: torch.Tensor, K, qw, kw, pos, axis_dims, dQo: torch.Tensor, dKo,
                              theta: float = 10000.0, eps: float = 1e-6, pairs: int = RTL_ROPE_ADJACENT, dQ=None,
                              dK=None, dqw=None, dkw=None, workspace=None, stream=None):
    """Gradient of rtl_qk_norm_rope: (dQ, dK, dqw, dkw) from its inputs and the gradients of its
    outputs; dqw and dkw [D] are float32 sums over all tokens and heads (zeros for a K of no heads).
    Outputs given by the caller are written in place; dQ and dK may be dQo and dKo, or Q and K."""
    M, Hq, D = Q.shape
    dt = Q.dtype
    qs, ks, ws = (M, Hq, D), (M, 0 if K is None else K.shape[1], D), (D,)
    there = _elsewhere(Q, K, qw, kw, pos if len(axis_dims) else None, dQo, dKo, dQ, dK, dqw, dkw, workspace)
    if there is not None:
        with there:
            return rtl_qk_norm_rope_backward(Q, K, qw, kw, pos, axis_dims, dQo, dKo, theta, eps, pairs, dQ, dK, dqw, dkw,
                                             workspace, stream)
    given = dQ, dK, dqw, dkw
    if dQ is None:
        dQ = _new(stream, Q, qs, dt)
    if dqw is None:
        dqw = _new(stream, Q, (D,), torch.float32)
    keys, grads, grads_out, kw_at, dkw_at = _NO_HEADS, _NO_HEADS, _NO_HEADS, None, None
    if K is not None:
        if dK is None:
            dK = _new(stream, Q, ks, dt)
        if dkw is None:
            dkw = _new(stream, Q, (D,), torch.float32)
        keys, grads, grads_out = _heads("K", K, ks, dt), _heads("dKo", dKo, ks, dt), _heads("dK", dK, ks, dt)
        kw_at, dkw_at = _flat("kw", kw, ws, dt), _flat("dkw", dkw, ws, torch.float32)
    elif dKo is not None or dK is not None or dkw is not None:
        raise ValueError("dKo, dK or dkw without K")
    if workspace is None:
        workspace = _new(stream, Q, (max(rtl_qk_norm_rope_backward_workspace_bytes(D), 1),), torch.uint8)
    _check(lib.rtl_qk_norm_rope_backward(_dt(Q), M, Hq, ks[1], D, *_heads("Q", Q, qs, dt), *keys,
                                         _flat("qw", qw, ws, dt), kw_at, eps,
                                         *_rope_args(pos, axis_dims, theta, pairs, M),
                                         *_heads("dQo", dQo, qs, dt), *grads, *_heads("dQ", dQ, qs, dt), *grads_out,
                                         _flat("dqw", dqw, ws, torch.float32), dkw_at, *_space(workspace),
                                         _queue(stream, Q)))
    if K is not None and ks[1] == 0:  # to the library, no K: an empty sum is not written
        with torch.cuda.stream(_torch_stream(stream)):
            dkw.zero_()
    _changed(given)
    return dQ, dK, dqw, dkw


def rtl_glu_fused(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, act: int = RTL_ACT_SILU, Y=None, G=None, U=None,
                  stream=None) -> torch.Tensor:
    """Y = act(X Wg^T) * (X Wu^T) in one kernel (bf16).  X [M,K], Wg and Wu [H,K], Y [M,H].
    ``G`` and ``U`` [M,H], when given, receive the two products (rtl_glu_backward takes them)."""
    M, K = X.shape
    H = Wg.shape[0]
    xs, ws, ys, bf16 = (M, K), (H, K), (M, H), torch.bfloat16
    there = _elsewhere(X, Wg, Wu, Y, G, U)
    if there is not None:
        with there:
            return rtl_glu_fused(X, Wg, Wu, act, Y, G, U, stream)
    given = Y, G, U
    if Y is None:
        Y = _new(stream, X, ys, bf16)
    _check(lib.rtl_glu_fused(act, RTL_BF16, M, K, H, _flat("X", X, xs, bf16), _flat("Wg", Wg, ws, bf16),
                             _flat("Wu", Wu, ws, bf16), _flat("Y", Y, ys, bf16), _flat("G", G, ys, bf16),
                             _flat("U", U, ys, bf16), _queue(stream, X)))
    _changed(given)
    return Y


def rtl_glu_backward_workspace_bytes(M: int, K: int, H: int) -> int:
    return int(lib.rtl_glu_backward_workspace_bytes(M, K, H))


def rtl_glu_backward(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, G: torch.Tensor, U: torch.Tensor,
                     dY: torch.Tensor, act: int = RTL_ACT_SILU, dX=None, dWg=None, dWu=None, workspace=None,
                     need_dx: bool = True, need_dw: bool = True, stream=None):
    """Gradient of rtl_glu_fused: (dX, dWg, dWu) from its inputs, G and U as it left them, and dY
    [M,H] (bf16).  ``need_dx`` or ``need_dw`` False leaves those out (None).  Outputs given by the
    caller are written in place; pass ``workspace`` (uint8) to keep the call free of allocations."""
    M, K = X.shape
    H = Wg.shape[0]
    xs, ws, ys, bf16 = (M, K), (H, K), (M, H), torch.bfloat16
    there = _elsewhere(X, Wg, Wu, G, U, dY, dX, dWg, dWu, workspace)
    if there is not None:
        with there:
            return rtl_glu_backward(X, Wg, Wu, G, U, dY, act, dX, dWg, dWu, workspace, need_dx, need_dw, stream)
    if not need_dx:
        dX = None
    if not need_dw:
        dWg = dWu = None
    given = dX, dWg, dWu
    if need_dx and dX is None:
        dX = _new(stream, X, xs, bf16)
    if need_dw:
        dWg = _new(stream, X, ws, bf16) if dWg is None else dWg
        dWu = _new(stream, X, ws, bf16) if dWu is None else dWu
    if workspace is None:
        workspace = _new(stream, X, (max(rtl_glu_backward_workspace_bytes(M, K, H), 1),), torch.uint8)
    _check(lib.rtl_glu_backward(act, RTL_BF16, M, K, H, _flat("X", X, xs, bf16), _flat("Wg", Wg, ws, bf16),
                                _flat("Wu", Wu, ws, bf16), _flat("G", G, ys, bf16), _flat("U", U, ys, bf16),
                                _flat("dY", dY, ys, bf16), _flat("dX", dX, xs, bf16), _flat("dWg", dWg, ws, bf16),
                                _flat("dWu", dWu, ws, bf16), *_space(workspace), _queue(stream, X)))
    _changed(given)
    return dX, dWg, dWu


_NO_ROWS = None, 0


def _rows(name, t, shape, dtype):
    """Address and row stride of a tensor of `shape` [M, C] and `dtype` whose channels are contiguous
    (None: null)."""
    if t is None:
        return _NO_ROWS
    if t.shape != shape or t.dtype is not dtype:
        _mismatch(name, t, shape, dtype)
    row, channel = t.stride()
    if channel != 1 and shape[1] > 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return t.data_ptr(), row


def _groups(groups, scale):
    """Number of groups, and the address of their offsets."""
    if groups is None:
        return (0 if scale is None else scale.shape[0]), None
    if groups.dim() != 1 or groups.numel() < 2:
        raise ValueError(f"groups must hold G + 1 offsets, got shape {tuple(groups.shape)}")
    return groups.numel() - 1, _flat("groups", groups, groups.shape, torch.int32)


def rtl_layer_norm(X: torch.Tensor, weight=None, bias=None, scale=None, shift=None, groups=None, eps: float = 1e-6,
                   Y=None, stats=None, stream=None) -> torch.Tensor:
    """Layer norm of every row of X [M,D] (any row stride): y = (n weight + bias) (1 + scale_g) + shift_g.

    ``weight`` and ``bias`` [D] (None: ones, zeros).  ``scale`` and ``shift`` [G,D] (any row stride; both or
    neither) belong to groups of rows: ``groups`` int32 [G+1] on the GPU holds ascending offsets, rows outside
    them are left as they were in a ``Y`` that is given, zeros in a new one; None: all rows are one group.  ``stats`` [M,2] float32, when given, receives
    each row's mean and 1 / deviation (rtl_layer_norm_backward takes them).  ``Y`` may be X."""
    M, D = X.shape
    shape, dt, ws = (M, D), X.dtype, (D,)
    there = _elsewhere(X, weight, bias, scale, shift, groups, Y, stats)
    if there is not None:
        with there:
            return rtl_layer_norm(X, weight, bias, scale, shift, groups, eps, Y, stats, stream)
    given, rest = (Y, stats), RTL_REST_KEPT
    if Y is None:
        Y, rest = _new(stream, X, shape, dt), RTL_REST_ZEROS
    G, at = _groups(groups, scale)
    _check(lib.rtl_layer_norm_ex(rest, _dt(X), M, D, *_rows("X", X, shape, dt), _flat("weight", weight, ws, dt),
                                 _flat("bias", bias, ws, dt), G, at, *_rows("scale", scale, (G, D), dt),
                                 *_rows("shift", shift, (G, D), dt), eps, *_rows("Y", Y, shape, dt),
                                 _flat("stats", stats, (M, 2), torch.float32), _queue(stream, X)))
    _changed(given)
    return Y


@functools.lru_cache(maxsize=64)
def rtl_layer_norm_backward_workspace_bytes(M: int, D: int, G: int) -> int:
    return int(lib.rtl_layer_norm_backward_workspace_bytes(M, D, G))


def rtl_layer_norm_backward(X: torch.Tensor, stats: torch.Tensor, dY: torch.Tensor, weight=None, bias=None, scale=None,
                            groups=None, dX=None, dweight=None, dbias=None, dscale=None, dshift=None, workspace=None,
                            need_dw: bool = True, stream=None):
    """Gradient of rtl_layer_norm: (dX, dweight, dbias, dscale, dshift) from its inputs, the ``stats`` it
    left and dY.  The sums are float32, dweight and dbias [D] for a weight or bias that is given, dscale and
    dshift [G,D] for a scale that is (else None; all None with ``need_dw`` False).  Rows outside the groups
    count in no sum; in a dX that is given they are left as they were, in a new one they are zeros.  Outputs given by the caller are written in place; dX may be dY or X."""
    M, D = X.shape
    shape, dt, ws, f32 = (M, D), X.dtype, (D,), torch.float32
    there = _elsewhere(X, stats, dY, weight, bias, scale, groups, dX, dweight, dbias, dscale, dshift, workspace)
    if there is not None:
        with there:
            return rtl_layer_norm_backward(X, stats, dY, weight, bias, scale, groups, dX, dweight, dbias, dscale, dshift,
                                           workspace, need_dw, stream)
    G, at = _groups(groups, scale)
    if not need_dw:
        dweight = dbias = dscale = dshift = None
    if scale is None and (dscale is not None or dshift is not None):
        raise ValueError("dscale or dshift without scale")
    given, rest = (dX, dweight, dbias, dscale, dshift), RTL_REST_KEPT
    if dX is None:
        dX, rest = _new(stream, X, shape, dt), RTL_REST_ZEROS
    if need_dw:
        if weight is not None and dweight is None:
            dweight = _new(stream, X, ws, f32)
        if bias is not None and dbias is None:
            dbias = _new(stream, X, ws, f32)
        if scale is not None:
            dscale = _new(stream, X, (G, D), f32) if dscale is None else dscale
            dshift = _new(stream, X, (G, D), f32) if dshift is None else dshift
    if workspace is None:
        workspace = _new(stream, X, (max(rtl_layer_norm_backward_workspace_bytes(M, D, G), 1),), torch.uint8)
    _check(lib.rtl_layer_norm_backward_ex(
        rest, _dt(X), M, D, *_rows("X", X, shape, dt), _flat("stats", stats, (M, 2), f32), *_rows("dY", dY, shape, dt),
        _flat("weight", weight, ws, dt), _flat("bias", bias, ws, dt), G, at, *_rows("scale", scale, (G, D), dt),
        *_rows("dX", dX, shape, dt), _flat("dweight", dweight, ws, f32), _flat("dbias", dbias, ws, f32),
        _flat("dscale", dscale, (G, D), f32), _flat("dshift", dshift, (G, D), f32), *_space(workspace), _queue(stream, X)))
    _changed(given)
    return dX, dweight, dbias, dscale, dshift


@functools.lru_cache(maxsize=64)
def rtl_adapters_plan_bytes(M: int, A: int) -> int:
    return int(lib.rtl_adapters_plan_bytes(M, A))


def rtl_adapters_plan(ids: torch.Tensor, A: int, plan=None, stream=None) -> torch.Tensor:
    """The plan of a batch whose row m has adapter ids[m] (int32 [M] on the GPU; outside 0..A-1: none), for
    rtl_adapters and rtl_adapters_backward: a uint8 tensor, written in place when given (a captured call
    then takes the next batch of M rows)."""
    M, = ids.shape
    there = _elsewhere(ids, plan)
    if there is not None:
        with there:
            return rtl_adapters_plan(ids, A, plan, stream)
    given = (plan,)
    if plan is None:
        plan = _new(stream, ids, (max(rtl_adapters_plan_bytes(M, A), 1),), torch.uint8)
    _check(lib.rtl_adapters_plan(M, A, _flat("ids", ids, (M,), torch.int32), *_space(plan), _queue(stream, ids)))
    _changed(given)
    return plan


@functools.lru_cache(maxsize=64)
def rtl_adapters_workspace_bytes(M: int, N: int, K: int, R: int, A: int) -> int:
    return int(lib.rtl_adapters_workspace_bytes(M, N, K, R, A))


def _factors(LA, LB):
    """A, N, R and K of LA [A,N,R] and LB [A,R,K]."""
    if LA.dim() != 3 or LB.dim() != 3 or LA.shape[0] != LB.shape[0] or LA.shape[2] != LB.shape[1]:
        raise ValueError(f"LA and LB must be [A,N,R] and [A,R,K], got {tuple(LA.shape)} and {tuple(LB.shape)}")
    return *LA.shape, LB.shape[2]


def rtl_adapters(X: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor, plan: torch.Tensor, alpha=None, Y0=None, Y=None,
                 T=None, workspace=None, stream=None) -> torch.Tensor:
    """Y = Y0 + alpha_a (X LB_a^T) LA_a^T, each row with its own adapter a of LA [A,N,R] and LB [A,R,K] (bf16).

    X [M,K] and Y0 [M,N] (what the shared projection made of X; None: zeros) may be parts of wider rows.
    ``plan`` is rtl_adapters_plan's of the batch, ``alpha`` [A] float32 (None: ones).  ``Y`` may be Y0, and then
    rows without an adapter are not touched.  ``T`` [M,R] float32, when given, receives X LB_a^T
    (rtl_adapters_backward takes it)."""
    M = X.shape[0]
    A, N, R, K = _factors(LA, LB)
    bf16 = torch.bfloat16
    there = _elsewhere(X, LA, LB, plan, alpha, Y0, Y, T, workspace)
    if there is not None:
        with there:
            return rtl_adapters(X, LA, LB, plan, alpha, Y0, Y, T, workspace, stream)
    given = Y, T
    if Y is None:
        Y = _new(stream, X, (M, N), bf16)
    if workspace is None:
        workspace = _new(stream, X, (max(rtl_adapters_workspace_bytes(M, N, K, R, A), 1),), torch.uint8)
    _check(lib.rtl_adapters(RTL_BF16, M, N, K, R, A, *_rows("X", X, (M, K), bf16), _flat("LA", LA, (A, N, R), bf16),
                            _flat("LB", LB, (A, R, K), bf16), _flat("alpha", alpha, (A,), torch.float32), *_space(plan),
                            *_rows("Y0", Y0, (M, N), bf16), *_rows("Y", Y, (M, N), bf16),
                            _flat("T", T, (M, R), torch.float32), *_space(workspace), _queue(stream, X)))
    _changed(given)
    return Y


@functools.lru_cache(maxsize=64)
def rtl_adapters_backward_workspace_bytes(M: int, N: int, K: int, R: int, A: int) -> int:
    return int(lib.rtl_adapters_backward_workspace_bytes(M, N, K, R, A))


def rtl_adapters_backward(X: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor, plan: torch.Tensor, T, dY: torch.Tensor,
                          alpha=None, dX0=None, dX=None, dLA=None, dLB=None, workspace=None, need_dx: bool = True,
                          need_dw: bool = True, stream=None):
    """Gradient of rtl_adapters: (dX, dLA, dLB) from its inputs, the ``T`` it left and dY [M,N].

    dX = dX0 + alpha_a (dY LA_a) LB_a [M,K] (``dX0``: what came through the shared projection, None: zeros;
    ``dX`` may be dX0); dLA [A,N,R] and dLB [A,R,K] are float32, zeros for an adapter without rows.
    ``need_dx`` or ``need_dw`` False leaves those out (None).  Outputs given by the caller are written in place."""
    M = X.shape[0]
    A, N, R, K = _factors(LA, LB)
    bf16, f32 = torch.bfloat16, torch.float32
    there = _elsewhere(X, LA, LB, plan, T, dY, alpha, dX0, dX, dLA, dLB, workspace)
    if there is not None:
        with there:
            return rtl_adapters_backward(X, LA, LB, plan, T, dY, alpha, dX0, dX, dLA, dLB, workspace, need_dx, need_dw,
                                         stream)
    if not need_dx:
        dX = None
    if not need_dw:
        dLA = dLB = None
    given = dX, dLA, dLB
    if need_dx and dX is None:
        dX = _new(stream, X, (M, K), bf16)
    if need_dw:
        dLA = _new(stream, X, (A, N, R), f32) if dLA is None else dLA
        dLB = _new(stream, X, (A, R, K), f32) if dLB is None else dLB
    if workspace is None:
        workspace = _new(stream, X, (max(rtl_adapters_backward_workspace_bytes(M, N, K, R, A), 1),), torch.uint8)
    _check(lib.rtl_adapters_backward(
        RTL_BF16, M, N, K, R, A, *_rows("X", X, (M, K), bf16), _flat("LA", LA, (A, N, R), bf16),
        _flat("LB", LB, (A, R, K), bf16), _flat("alpha", alpha, (A,), f32), *_space(plan), _flat("T", T, (M, R), f32),
        *_rows("dY", dY, (M, N), bf16), *_rows("dX0", dX0, (M, K), bf16), *_rows("dX", dX, (M, K), bf16),
        _flat("dLA", dLA, (A, N, R), f32), _flat("dLB", dLB, (A, R, K), f32), *_space(workspace), _queue(stream, X)))
    _changed(given)
    return dX, dLA, dLB


class AdamWTensors:
    """The tensors that an rtl_adamw call steps, checked and listed once (rtl_adamw_tensors).  It holds
    them: their memory stays as long as it does, and a tensor that is replaced needs a new list."""

    def __init__(self, params, grads, m, v, masters, m_scales, v_scales):
        kinds = dict(p=params, g=grads, master=masters, m=m, v=v, m_scale=m_scales, v_scale=v_scales)
        kinds = {n: [t.detach() for t in ts] for n, ts in kinds.items() if ts is not None}
        if not kinds["p"]:
            raise ValueError("no tensors")
        if any(len(ts) != len(kinds["p"]) for ts in kinds.values()):
            raise ValueError("the lists differ in length: " + ", ".join(f"{n} {len(ts)}" for n, ts in kinds.items()))
        self.p_dt, self.g_dt = _dt(kinds["p"][0]), _dt(kinds["g"][0])
        self.states = RTL_STATES_32 if kinds["m"][0].dtype is torch.float32 else RTL_STATES_8
        if (self.p_dt == RTL_BF16) != ("master" in kinds):
            raise ValueError("bf16 parameters need fp32 masters, fp32 ones take none")
        if any((self.states == RTL_STATES_8) != (n in kinds) for n in ("m_scale", "v_scale")):
            raise ValueError("8-bit states need m_scales and v_scales, 32-bit ones take none")
        state = torch.float32 if self.states == RTL_STATES_32 else torch.float8_e4m3fn
        types = dict(p=kinds["p"][0].dtype, g=kinds["g"][0].dtype, master=torch.float32, m=state, v=state,
                     m_scale=torch.float32, v_scale=torch.float32)
        self.like = kinds["p"][0]
        _elsewhere(self.like, *(t for ts in kinds.values() for t in ts))
        self.array = (_AdamWTensor * len(kinds["p"]))()
        for i, entry in enumerate(self.array):
            shape = kinds["p"][i].shape
            entry.n = kinds["p"][i].numel()
            blocks = ((entry.n + 255) // 256,)
            for n, ts in kinds.items():
                setattr(entry, n, _flat(f"{n}[{i}]", ts[i], blocks if n.endswith("scale") else shape, types[n]))
        self.held = kinds
        self.changed = [t for n, ts in kinds.items() if n != "g" for t in ts]


def rtl_adamw_tensors(params, grads, m, v, masters=None, m_scales=None, v_scales=None) -> AdamWTensors:
    """The list that rtl_adamw steps: tensors of equal shapes at equal places of ``params``, ``grads``, ``m``, ``v`` and,
    where ``params`` are bf16, ``masters`` (float32).  m and v are float32, or torch.float8_e4m3fn with
    ``m_scales`` and ``v_scales`` float32 [(n + 255) // 256] (all zeros to start)."""
    return AdamWTensors(params, grads, m, v, masters, m_scales, v_scales)


def _number(name, x, dtype, like):
    """A number, or the address of one on the GPU: (number, address)."""
    if not isinstance(x, torch.Tensor):
        return x, None
    if x.numel() != 1 or x.dtype is not dtype:
        raise ValueError(f"{name} must be one {dtype}, got {x.dtype} of shape {tuple(x.shape)}")
    _elsewhere(like, x)
    return 1, x.data_ptr()


def rtl_adamw(tensors: AdamWTensors, step, lr, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.01, grad_scale=None, stream=None) -> None:
    """One AdamW step of all ``tensors`` in place (rtl_adamw_tensors), on the gradients they hold then:
    m += (1 - beta1) (g - m), v = beta2 v + (1 - beta2) g^2, and the parameters (their masters, where bf16) less
    lr (m / (1 - beta1^step) / (sqrt(v / (1 - beta2^step)) + eps) + weight_decay p).

    ``step`` counts from 1.  ``step`` (int64) and ``lr`` (float32) may be tensors of one element on the GPU, which a captured
    call reads anew with every replay; so is ``grad_scale`` (float32, None: 1), a factor of the gradients."""
    like = tensors.like
    there = _elsewhere(like)
    if there is not None:
        with there:
            return rtl_adamw(tensors, step, lr, beta1, beta2, eps, weight_decay, grad_scale, stream)
    step, step_at = _number("step", step, torch.int64, like)
    lr, lr_at = _number("lr", lr, torch.float32, like)
    if grad_scale is not None and not isinstance(grad_scale, torch.Tensor):
        raise ValueError("grad_scale must be a tensor on the GPU")
    scale_at = None if grad_scale is None else _number("grad_scale", grad_scale, torch.float32, like)[1]
    _check(lib.rtl_adamw(tensors.p_dt, tensors.g_dt, tensors.states, len(tensors.array), tensors.array, step, step_at, lr,
                         lr_at, beta1, beta2, eps, weight_decay, scale_at, _queue(stream, like)))
    _changed(tensors.changed)
