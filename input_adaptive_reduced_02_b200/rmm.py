"""Python binding for librmm, the B200 Reduced Matrix Multiplication library.

Argument marshalling only: every step of score -> select -> pack -> gemm runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. There is no fallback: if librmm.so is missing, loading fails loudly.

Method (gist.science summary of "Reduced Matrix Multiplication: Input-Adaptive
Matrix-Product Reduction for LLM Inference", Resumo Técnico › Metodologia):
score every contraction slice k of A·B, keep the top ceil(rho·K), and compute
A[:, I]·B[I, :]. The default score is ||A[:,k]||·||B[k,:]|| ("product"); the
pages' activation-only column norm is mode "a_only".
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librmm.so")

RMM_OK, RMM_ERR_INVALID, RMM_ERR_NONFINITE, RMM_ERR_CUDA, RMM_ERR_TIMEOUT, RMM_ERR_UNSUPPORTED = range(6)
RMM_BF16, RMM_F32 = 0, 1
SCORE_MODES = {"product": 0, "a_only": 1}
STATUS_NAMES = {0: "RMM_OK", 1: "RMM_ERR_INVALID", 2: "RMM_ERR_NONFINITE", 3: "RMM_ERR_CUDA",
                4: "RMM_ERR_TIMEOUT", 5: "RMM_ERR_UNSUPPORTED"}


class RMMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None

_vp, _i64, _f64, _i32, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_double, ctypes.c_int, ctypes.c_uint64
_SIGS = {
    "rmm_keep_count": (_i64, [_f64, _i64]),
    "rmm_padded_keep": (_i64, [_i64]),
    "rmm_packed_b_ld": (_i64, [_i64]),
    "rmm_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64, _i32]),
    "rmm_workspace_size_for": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64, _i32, _i32]),
    "rmm_score": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _i64, _i32, _i32, _vp, _vp,
                         _vp]),
    "rmm_select": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "rmm_pack": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _vp,
                        _vp, _vp]),
    "rmm_gemm": (_i32, [_vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32, _vp, _i64, _i64, _i32, _vp, _vp]),
    "rmm_matmul_reduced": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _f64, _i32, _i32, _vp, _i64, _i32, _vp,
                                  _vp, ctypes.c_size_t, _vp]),
    "rmm_matmul_reduced_batched": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _i64, _i64, _i64, _i64, _f64,
                                          _i32, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.c_size_t, _vp]),
    "rmm_qk_reduced": (_i32, [_vp, _vp, _i64, _i64, _i64, _i64, _f64, _i32, _i32, _vp, _i32, _vp, _vp,
                              ctypes.c_size_t, _vp]),
    "rmm_pv_reduced": (_i32, [_vp, _vp, _i64, _i64, _i64, _i64, _f64, _i32, _i32, _vp, _i32, _vp, _vp,
                              ctypes.c_size_t, _vp]),
    "rmm_matmul_reduced_noalloc": (_i32, [_vp, _i64, _vp, _i64, _i64, _i64, _i64, _f64, _i32, _i32, _vp, _i64, _i32,
                                          _vp, _vp, _vp]),
    "rmm_b_norms": (_i32, [_vp, _i64, _i64, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp]),
    "rmm_score_b_norms": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i32, _vp, _vp, _vp]),
    "rmm_matmul_reduced_b_norms": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i32, _vp, _i64, _i64, _i64, _i64,
                                          _i64, _f64, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.c_size_t,
                                          _vp]),
    "rmm_gemv_gather": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i32, _vp,
                               _i64, _i64, _i32, _vp]),
    "rmm_b_norms_w8": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp]),
    "rmm_pack_w8": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp,
                           _vp, _vp, _vp]),
    "rmm_matmul_reduced_w8": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64,
                                     _i64, _f64, _i32, _i32, _vp, _i64, _i64, _i32, _vp, _vp, ctypes.c_size_t,
                                     _vp]),
    "rmm_gemv_gather_w8": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64,
                                  _vp, _i64, _i64, _i32, _vp]),
    "rmm_mask_rows": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i32, _vp, _vp]),
    "rmm_gemm_full": (_i32, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _i32, _vp, _i64, _i64, _i32, _vp,
                             _vp]),
    "rmm_fused_route": (_i32, [_i64, _i64, _i64, _i32, _i32, _vp, _i64, _i64]),
    "rmm_softmax_row_stats": (_i32, [_vp, _i32, ctypes.c_float, _i32, _i64, _i64, _i64, _vp, _vp, _vp]),
    "rmm_softmax_score": (_i32, [_vp, _i32, ctypes.c_float, _i32, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp,
                                 _vp]),
    "rmm_pv_softmax_workspace_size": (ctypes.c_size_t, [_i64, _i64, _i64, _i64, _i64]),
    "rmm_pv_softmax_reduced": (_i32, [_vp, _i32, ctypes.c_float, _i32, _vp, _i64, _i64, _i64, _i64, _f64, _i32, _vp,
                                      _vp, _i32, _vp, _vp, ctypes.c_size_t, _vp]),
    "rmm_attn_prompt": (_i32, [_vp, _i64, _i64] * 3 + [_vp, _vp] + [_i64] * 6 + [ctypes.c_float, _i32, _i32, _vp,
                                                                                 _i64, _i64, _i32, _vp, _vp, _vp]),
    "rmm_attn_key_weights": (_i32, [_vp, _i64, _i64] * 2 + [_vp, _vp] + [_i64] * 6 + [ctypes.c_float, _i32, _i32] +
                             [_vp] * 5),
    "rmm_kv4_store": (_i32, [_vp, _i64, _i64] * 2 + [_i32, _vp, _vp] + [_i64] * 5 + [_vp] * 8),
    "rmm_kv4_attn_workspace_size": (ctypes.c_size_t, [_i64] * 5 + [_i32]),
    "rmm_kv4_attn": (_i32, [_vp, _i64, _i64] + [_vp] * 5 + [_i64] * 5 + [ctypes.c_float, _i32, _vp, _i64, _i64, _i32] +
                     [_vp] * 4 + [ctypes.c_size_t, _vp]),
    "rmm_cache_evict_workspace_size": (ctypes.c_size_t, [_i64] * 3),
    "rmm_cache_evict": (_i32, [_vp, _vp] + [_i64] * 6 + [_vp, _i64, _i64] + [_vp] * 3 + [ctypes.c_size_t, _vp]),
    "rmm_check": (_i32, [_vp, _vp]),
    "rmm_last_error_string": (ctypes.c_char_p, []),
    "rmm_set_wait_limit_ns": (None, [_u64]),
    "rmm_set_stall_producer_for_test": (None, [_i32]),
    "rmm_set_gemm_cta_group": (_i32, [_i32]),
    "rmm_launch_count": (_u64, []),
    "rmm_set_debug": (_i32, [_i32]),
    "rmm_set_gemm_events": (None, [ctypes.c_void_p, ctypes.c_void_p]),
}


def lib() -> ctypes.CDLL:
    """The loaded librmm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(f"librmm.so not found at {_LIB_PATH}; build it with "
                              "`python -m input_adaptive_reduced_02_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def library_path() -> str:
    return _LIB_PATH


def _check(status: int):
    if status != RMM_OK:
        raise RMMError(status, lib().rmm_last_error_string().decode(errors="replace"))


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return RMM_BF16
    if t.dtype == torch.float32:
        return RMM_F32
    raise TypeError(f"unsupported dtype {t.dtype}; librmm takes bfloat16 or float32")


def _out_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return RMM_BF16
    if dt == torch.float32:
        return RMM_F32
    raise TypeError(f"unsupported output dtype {dt}")


def _stream(t: torch.Tensor) -> int:
    """The handle of the current stream of t's device (a small call's time is the host's, so no Stream object is made)."""
    device = t.get_device()
    if device < 0:  # which the lookup would take for the current device
        raise ValueError("expected a CUDA tensor")
    return torch._C._cuda_getCurrentRawStream(device)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _status_ptr(status: torch.Tensor | None, device):
    """The address of a status word (status_word()) on the call's device."""
    if status is None:
        return None
    if status.dtype not in (torch.int32, torch.uint32) or status.numel() < 1 or status.device != device:
        raise ValueError(f"status must be a 32-bit integer tensor on {device} (status_word())")
    return status.data_ptr()


def _mat(t: torch.Tensor, name: str):
    """(batch, rows, cols, ld, batch_stride) of a 2-D or 3-D CUDA tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() == 2:
        t3 = t.unsqueeze(0)
    elif t.dim() == 3:
        t3 = t
    else:
        raise ValueError(f"{name} must be 2-D or 3-D")
    if t3.stride(2) != 1 and t3.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    b, r, c = t3.shape
    ld = t3.stride(1) if r > 1 else c
    bs = t3.stride(0) if b > 1 else r * ld
    return b, r, c, ld, bs


def keep_count(rho: float, K: int) -> int:
    k = lib().rmm_keep_count(float(rho), int(K))
    if k < 1:
        raise ValueError(f"rho must lie in (0, 1] and K >= 1 (rho={rho}, K={K})")
    return int(k)


def padded_keep(k_keep: int) -> int:
    return int(lib().rmm_padded_keep(int(k_keep)))


def workspace_size(batch: int, M: int, K: int, N: int, k_keep: int, dtype: torch.dtype) -> int:
    """Workspace bytes of a fused call on any route."""
    return int(lib().rmm_workspace_size(batch, M, K, N, k_keep, _out_code(dtype)))


def workspace_size_for(batch: int, M: int, K: int, N: int, k_keep: int, dtype: torch.dtype,
                       b_kmajor: bool = False) -> int:
    """Workspace bytes of a fused call on the route it takes (no packed operands when M <= 16 and B is row-major)."""
    return int(lib().rmm_workspace_size_for(batch, M, K, N, k_keep, _out_code(dtype), int(b_kmajor)))


class Workspace:
    """A 1 KiB-aligned device workspace carved from one torch allocation."""

    def __init__(self, nbytes: int, device):
        self.nbytes = int(nbytes)
        self._buf = torch.empty(self.nbytes + 1024, dtype=torch.uint8, device=device)
        self.device = self._buf.device
        base = self._buf.data_ptr()
        self.offset = (-base) % 1024
        self.ptr = base + self.offset

    @property
    def status_ptr(self) -> int:
        return self.ptr


def _ensure_ws(ws, nbytes, device):
    if ws is not None and ws.device != device:
        raise ValueError(f"the workspace is on {ws.device}, the call on {device}")
    if ws is None or ws.nbytes < nbytes:
        return Workspace(nbytes, device)
    return ws


def status_word(device="cuda") -> torch.Tensor:
    """A zeroed device u32 (as int32 storage) for the stage calls' status bits."""
    return torch.zeros(1, dtype=torch.int32, device=device)


def check(status, stream_tensor: torch.Tensor | None = None):
    """Read and clear a device status word (a tensor from status_word(), or a
    Workspace); raise RMMError on NaN/Inf scores, a pipeline timeout or a token
    outside its cache."""
    if isinstance(status, Workspace):
        ptr, dev = status.ptr, status._buf.device
    else:
        ptr, dev = status.data_ptr(), status.device
    st = ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)
    _check(lib().rmm_check(ctypes.c_void_p(ptr), st))


# ---------------------------------------------------------------- stage calls
def score(A: torch.Tensor, B: torch.Tensor | None, mode: str = "product", b_kmajor: bool = False,
          out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """Slice scores s [batch][K] (f32). A [b][M][K]; B [b][K][N] (or [b][N][K] with b_kmajor)."""
    ba, M, K, lda, sA = _mat(A, "A")
    if B is not None:
        bb, r, c, ldb, sB = _mat(B, "B")
        N = r if b_kmajor else c
        if (c if b_kmajor else r) != K or bb != ba:
            raise ValueError("A and B disagree on the contraction dimension or batch")
    else:
        if SCORE_MODES[mode] != 1:
            raise ValueError("B is required in product mode")
        N, ldb, sB = 0, 0, 0
    if out is None:
        out = torch.empty((ba, K) if A.dim() == 3 else (K,), dtype=torch.float32, device=A.device)
    _check(lib().rmm_score(_ptr(A), lda, sA, _ptr(B), ldb, sB, int(b_kmajor), ba, M, K, N, _dtype(A),
                           SCORE_MODES[mode], _ptr(out), _ptr(status), _stream(A)))
    return out


def b_norms(B: torch.Tensor, b_kmajor: bool = False, out: torch.Tensor | None = None,
            status: torch.Tensor | None = None) -> torch.Tensor:
    """B's factor of the product score, ||B[k,:]||_2 per slice k (f32 [batch][K] or [K]),
    for reuse across calls while B is unchanged. B [b][K][N] (or Kmat [b][N][K] with b_kmajor)."""
    bb, r, c, ldb, sB = _mat(B, "B")
    K, N = (c, r) if b_kmajor else (r, c)
    if out is None:
        out = torch.empty((bb, K) if B.dim() == 3 else (K,), dtype=torch.float32, device=B.device)
    _check(lib().rmm_b_norms(_ptr(B), ldb, sB, int(b_kmajor), bb, K, N, _dtype(B), _ptr(out), _ptr(status),
                             _stream(B)))
    return out


def _bn_stride(b_norm: torch.Tensor, batch: int, K: int) -> int:
    if b_norm.dtype != torch.float32 or not b_norm.is_cuda or not b_norm.is_contiguous():
        raise ValueError("b_norm must be a contiguous float32 CUDA tensor")
    if b_norm.dim() == 1:
        if b_norm.shape[0] != K:
            raise ValueError("b_norm must hold K values")
        return 0  # one vector shared by every batch item
    if tuple(b_norm.shape) != (batch, K):
        raise ValueError("b_norm must be [K] or [batch][K]")
    return K


def score_b_norms(A: torch.Tensor, b_norm: torch.Tensor, out: torch.Tensor | None = None,
                  status: torch.Tensor | None = None) -> torch.Tensor:
    """Product-form slice scores with B's norms given: s[k] = ||A[:,k]||_2 · b_norm[k]."""
    ba, M, K, lda, sA = _mat(A, "A")
    stride = _bn_stride(b_norm, ba, K)
    if out is None:
        out = torch.empty((ba, K) if A.dim() == 3 else (K,), dtype=torch.float32, device=A.device)
    _check(lib().rmm_score_b_norms(_ptr(A), lda, sA, _ptr(b_norm), stride, ba, M, K, _dtype(A), _ptr(out),
                                   _ptr(status), _stream(A)))
    return out


def select(s: torch.Tensor, k_keep: int, out: torch.Tensor | None = None,
           status: torch.Tensor | None = None) -> torch.Tensor:
    """Ascending int32 indices of the k_keep largest scores per row of s (ties -> lower index)."""
    if s.dtype != torch.float32 or not s.is_cuda or not s.is_contiguous():
        raise ValueError("s must be a contiguous float32 CUDA tensor")
    batch, K = (1, s.shape[0]) if s.dim() == 1 else s.shape
    if out is None:
        out = torch.empty((k_keep,) if s.dim() == 1 else (batch, k_keep), dtype=torch.int32, device=s.device)
    _check(lib().rmm_select(_ptr(s), batch, K, k_keep, _ptr(out), _ptr(status), _stream(s)))
    return out


def packed_b_ld(N: int) -> int:
    return int(lib().rmm_packed_b_ld(int(N)))


def packed_b_shape(batched: bool, batch: int, N: int, k_pad: int, b_kmajor: bool):
    """Shape of the packed B operand: [(b)][N][k_pad] (b_kmajor) or [(b)][k_pad][packed_b_ld(N)]."""
    shp = (N, k_pad) if b_kmajor else (k_pad, packed_b_ld(N))
    return (batch, *shp) if batched else shp


def pack(A: torch.Tensor, B: torch.Tensor, idx: torch.Tensor, b_kmajor: bool = False, out=None,
         status: torch.Tensor | None = None):
    """A_S [b][M][k_pad] (kept columns of A, zero padded) and the packed B
    operand: the kept rows of B ([b][k_pad][packed_b_ld(N)]) or, with b_kmajor,
    the kept columns of Kmat ([b][N][k_pad]). `out` may supply the pair."""
    ba, M, K, lda, sA = _mat(A, "A")
    bb, r, c, ldb, sB = _mat(B, "B")
    N = r if b_kmajor else c
    k_keep = idx.shape[-1]
    kp = padded_keep(k_keep)
    bshape = packed_b_shape(A.dim() == 3, ba, N, kp, b_kmajor)
    if out is None:
        A_S = torch.empty((ba, M, kp) if A.dim() == 3 else (M, kp), dtype=A.dtype, device=A.device)
        B_S = torch.empty(bshape, dtype=A.dtype, device=A.device)
    else:
        A_S, B_S = out
        if A_S.numel() != ba * M * kp or B_S.numel() != int(torch.tensor(bshape).prod()):
            raise ValueError("pack: output buffers have the wrong size")
    _check(lib().rmm_pack(_ptr(A), lda, sA, _ptr(B), ldb, sB, int(b_kmajor), ba, M, K, N, _ptr(idx), k_keep,
                          _dtype(A), _ptr(A_S), _ptr(B_S), _ptr(status), _stream(A)))
    return A_S, B_S


def gemm(A_S: torch.Tensor, B_S: torch.Tensor, k_keep: int, out_dtype=torch.float32, b_kmajor: bool = False,
         N: int | None = None, out: torch.Tensor | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """C = A_S · B_S over the first k_keep (of k_pad) slices; B_S as written by pack()."""
    ba, M, kp, _, _ = _mat(A_S, "A_S")
    if b_kmajor:
        N = B_S.shape[-2]
    elif N is None:
        N = B_S.shape[-1]
    if out is None:
        out = torch.empty((ba, M, N) if A_S.dim() == 3 else (M, N), dtype=out_dtype, device=A_S.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_gemm(_ptr(A_S), _ptr(B_S), int(b_kmajor), ba, M, N, k_keep, _dtype(A_S), _ptr(out), ldc, sC,
                          _out_code(out.dtype), _ptr(status), _stream(A_S)))
    return out


def gemv_gather(A: torch.Tensor, B: torch.Tensor, idx: torch.Tensor, out_dtype=torch.float32,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A[:, idx] · B[idx, :] straight from A (M <= 16 rows) and row-major B, no packing."""
    ba, M, K, lda, sA = _mat(A, "A")
    bb, r, N, ldb, sB = _mat(B, "B")
    if r != K or bb != ba:
        raise ValueError("A and B disagree on the contraction dimension or batch")
    k = idx.shape[-1]
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_gemv_gather(_ptr(A), lda, sA, _ptr(B), ldb, sB, ba, M, K, N, _ptr(idx), k, _dtype(A),
                                 _ptr(out), ldc, sC, _out_code(out.dtype), _stream(A)))
    return out


ROUTE_PACK, ROUTE_STREAM, ROUTE_GEMV = 0, 1, 2


def fused_route(A: torch.Tensor, N: int, b_kmajor: bool = False) -> int:
    """Route a fused call takes for A (2-D or 3-D) and N: ROUTE_PACK,
    ROUTE_STREAM (B's dropped rows zeroed, A streamed whole) or ROUTE_GEMV."""
    ba, M, K, lda, sA = _mat(A, "A")
    return int(lib().rmm_fused_route(ba, M, N, int(b_kmajor), _dtype(A), _ptr(A), lda, sA))


def _fused_ws_bytes(A: torch.Tensor, N: int, k: int, b_kmajor: bool) -> int:
    """Workspace of a fused call on the route it takes for this A."""
    ba, M, K, _, _ = _mat(A, "A")
    if fused_route(A, N, b_kmajor) == ROUTE_PACK:
        return workspace_size(ba, M, K, N, k, A.dtype)
    return workspace_size_for(ba, M, K, N, k, A.dtype, b_kmajor)


def mask_rows(B: torch.Tensor, idx: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """B_M = B with the rows outside idx zeroed: [(b)][K][packed_b_ld(N)]."""
    bb, K, N, ldb, sB = _mat(B, "B")
    k = idx.shape[-1]
    if out is None:
        shp = (K, packed_b_ld(N))
        out = torch.empty((bb, *shp) if B.dim() == 3 else shp, dtype=B.dtype, device=B.device)
    _check(lib().rmm_mask_rows(_ptr(B), ldb, sB, bb, K, N, _ptr(idx), k, _dtype(B), _ptr(out), _stream(B)))
    return out


def gemm_full(A: torch.Tensor, B_M: torch.Tensor, N: int, out_dtype=torch.float32, out: torch.Tensor | None = None,
              status: torch.Tensor | None = None, causal_off: int = -1) -> torch.Tensor:
    """C = A · B_M over all K slices (bf16 tensor cores), B_M as mask_rows writes it.
    causal_off >= 0 declares A[i][k] = 0 for k > i + causal_off (blocks above are skipped)."""
    ba, M, K, lda, sA = _mat(A, "A")
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_gemm_full(_ptr(A), lda, sA, _ptr(B_M), ba, M, K, N, int(causal_off), _dtype(A), _ptr(out), ldc,
                               sC, _out_code(out.dtype), _ptr(status), _stream(A)))
    return out


# ---------------------------------------------------------------- fused calls
def matmul_reduced(A: torch.Tensor, B: torch.Tensor, rho: float, mode: str = "product",
                   out_dtype=torch.float32, out: torch.Tensor | None = None, workspace: Workspace | None = None,
                   idx_out: torch.Tensor | None = None, b_kmajor: bool = False):
    """C ≈ A·B keeping the top ceil(rho·K) contraction slices (batched when A is 3-D).

    Returns (C, workspace); the workspace can be passed back in to avoid
    re-allocation and to read the device status with check(workspace)."""
    ba, M, K, lda, sA = _mat(A, "A")
    bb, r, c, ldb, sB = _mat(B, "B")
    N = r if b_kmajor else c
    k = keep_count(rho, K)
    ws = _ensure_ws(workspace, _fused_ws_bytes(A, N, k, b_kmajor), A.device)
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_matmul_reduced_batched(_ptr(A), lda, sA, _ptr(B), ldb, sB, int(b_kmajor), ba, M, K, N,
                                            float(rho), _dtype(A), SCORE_MODES[mode], _ptr(out), ldc, sC,
                                            _out_code(out.dtype), _ptr(idx_out), ws.ptr,
                                            ws.nbytes, _stream(A)))
    return out, ws


def matmul_reduced_b_norms(A: torch.Tensor, B: torch.Tensor, b_norm: torch.Tensor, rho: float,
                           out_dtype=torch.float32, out: torch.Tensor | None = None,
                           workspace: Workspace | None = None, idx_out: torch.Tensor | None = None,
                           b_kmajor: bool = False):
    """matmul_reduced in product mode with B's norms cached (see b_norms): the score reads only A."""
    ba, M, K, lda, sA = _mat(A, "A")
    bb, r, c, ldb, sB = _mat(B, "B")
    N = r if b_kmajor else c
    stride = _bn_stride(b_norm, ba, K)
    k = keep_count(rho, K)
    ws = _ensure_ws(workspace, _fused_ws_bytes(A, N, k, b_kmajor), A.device)
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_matmul_reduced_b_norms(_ptr(A), lda, sA, _ptr(B), ldb, sB, int(b_kmajor), _ptr(b_norm),
                                            stride, ba, M, K, N, float(rho), _dtype(A), _ptr(out), ldc, sC,
                                            _out_code(out.dtype), _ptr(idx_out), ws.ptr,
                                            ws.nbytes, _stream(A)))
    return out, ws


def _w8(Wq: torch.Tensor, scale: torch.Tensor):
    """(batch, K, N, ldw, strideW, scale_stride) of an INT8 weight and its column scales."""
    if Wq.dtype != torch.int8:
        raise ValueError("Wq must be int8")
    bw, K, N, ldw, sW = _mat(Wq, "Wq")
    if scale.dtype != torch.float32 or not scale.is_cuda or not scale.is_contiguous():
        raise ValueError("scale must be a contiguous float32 CUDA tensor")
    if scale.dim() == 1:
        if scale.shape[0] != N:
            raise ValueError("scale must hold N values")
        return bw, K, N, ldw, sW, 0
    if tuple(scale.shape) != (bw, N):
        raise ValueError("scale must be [N] or [batch][N]")
    return bw, K, N, ldw, sW, N


def b_norms_w8(Wq: torch.Tensor, scale: torch.Tensor, out: torch.Tensor | None = None,
               status: torch.Tensor | None = None) -> torch.Tensor:
    """||W[k,:]||_2 of the dequantized INT8 weight W = Wq · diag(scale) (f32 [batch][K] or [K])."""
    bw, K, N, ldw, sW, ss = _w8(Wq, scale)
    if out is None:
        out = torch.empty((bw, K) if Wq.dim() == 3 else (K,), dtype=torch.float32, device=Wq.device)
    _check(lib().rmm_b_norms_w8(_ptr(Wq), ldw, sW, _ptr(scale), ss, bw, K, N, _ptr(out), _ptr(status), _stream(Wq)))
    return out


def pack_w8(A: torch.Tensor, Wq: torch.Tensor, scale: torch.Tensor, idx: torch.Tensor, out=None,
            status: torch.Tensor | None = None):
    """(A_S, B_S): A's kept columns and bf16(Wq[idx] · scale) — the operands rmm.gemm takes."""
    ba, M, K, lda, sA = _mat(A, "A")
    bw, K2, N, ldw, sW, ss = _w8(Wq, scale)
    if K2 != K:
        raise ValueError("A and Wq disagree on the contraction dimension")
    k = idx.shape[-1]
    kp = padded_keep(k)
    if out is None:
        A_S = torch.empty((ba, M, kp) if A.dim() == 3 else (M, kp), dtype=A.dtype, device=A.device)
        B_S = torch.empty(packed_b_shape(A.dim() == 3, ba, N, kp, False), dtype=A.dtype, device=A.device)
    else:
        A_S, B_S = out
    _check(lib().rmm_pack_w8(_ptr(A), lda, sA, _ptr(Wq), ldw, sW, _ptr(scale), ss, ba, M, K, N, _ptr(idx), k,
                             _ptr(A_S), _ptr(B_S), _ptr(status), _stream(A)))
    return A_S, B_S


def gemv_gather_w8(A: torch.Tensor, Wq: torch.Tensor, scale: torch.Tensor, idx: torch.Tensor,
                   out_dtype=torch.float32, out: torch.Tensor | None = None) -> torch.Tensor:
    """C = A[:, idx] · (Wq · diag(scale))[idx, :] straight from A (M <= 16 rows) and the INT8 weight."""
    ba, M, K, lda, sA = _mat(A, "A")
    bw, K2, N, ldw, sW, ss = _w8(Wq, scale)
    if K2 != K:
        raise ValueError("A and Wq disagree on the contraction dimension")
    k = idx.shape[-1]
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_gemv_gather_w8(_ptr(A), lda, sA, _ptr(Wq), ldw, sW, _ptr(scale), ss, ba, M, K, N, _ptr(idx), k,
                                    _ptr(out), ldc, sC, _out_code(out.dtype), _stream(A)))
    return out


def matmul_reduced_w8(A: torch.Tensor, Wq: torch.Tensor, scale: torch.Tensor, rho: float,
                      b_norm: torch.Tensor | None = None, mode: str = "product", out_dtype=torch.float32,
                      out: torch.Tensor | None = None, workspace: Workspace | None = None,
                      idx_out: torch.Tensor | None = None):
    """matmul_reduced on an INT8 weight W = Wq · diag(scale); product mode needs b_norm (b_norms_w8)."""
    ba, M, K, lda, sA = _mat(A, "A")
    bw, K2, N, ldw, sW, ss = _w8(Wq, scale)
    if K2 != K:
        raise ValueError("A and Wq disagree on the contraction dimension")
    bn_stride = 0
    if b_norm is not None:
        bn_stride = _bn_stride(b_norm, ba, K)
    elif SCORE_MODES[mode] == 0:
        raise ValueError("product mode needs b_norm (b_norms_w8)")
    k = keep_count(rho, K)
    ws = _ensure_ws(workspace, workspace_size_for(ba, M, K, N, k, A.dtype), A.device)
    if out is None:
        out = torch.empty((ba, M, N) if A.dim() == 3 else (M, N), dtype=out_dtype, device=A.device)
    _, _, _, ldc, sC = _mat(out, "C")
    _check(lib().rmm_matmul_reduced_w8(_ptr(A), lda, sA, _ptr(Wq), ldw, sW, _ptr(scale), ss, _ptr(b_norm), bn_stride,
                                       ba, M, K, N, float(rho), _dtype(A), SCORE_MODES[mode], _ptr(out), ldc, sC,
                                       _out_code(out.dtype), _ptr(idx_out), ws.ptr, ws.nbytes,
                                       _stream(A)))
    return out, ws


def qk_reduced(Q: torch.Tensor, Kmat: torch.Tensor, rho: float, mode: str = "product", out_dtype=torch.float32,
               out: torch.Tensor | None = None, workspace: Workspace | None = None,
               idx_out: torch.Tensor | None = None):
    """S = Q·Kᵀ per head, reduced over head_dim. Q [bh][S_q][d], Kmat [bh][S_k][d]."""
    bh, S_q, d = Q.shape
    S_k = Kmat.shape[1]
    k = keep_count(rho, d)
    ws = _ensure_ws(workspace, _fused_ws_bytes(Q, S_k, k, True), Q.device)
    if out is None:
        out = torch.empty(bh, S_q, S_k, dtype=out_dtype, device=Q.device)
    _check(lib().rmm_qk_reduced(_ptr(Q), _ptr(Kmat), bh, S_q, S_k, d, float(rho), _dtype(Q), SCORE_MODES[mode],
                                _ptr(out), _out_code(out.dtype), _ptr(idx_out), ws.ptr, ws.nbytes,
                                _stream(Q)))
    return out, ws


def pv_reduced(P: torch.Tensor, V: torch.Tensor, rho: float, mode: str = "product", out_dtype=torch.float32,
               out: torch.Tensor | None = None, workspace: Workspace | None = None,
               idx_out: torch.Tensor | None = None):
    """O = P·V per head, reduced over the keys. P [bh][S_q][S_k], V [bh][S_k][d]."""
    bh, S_q, S_k = P.shape
    d = V.shape[2]
    k = keep_count(rho, S_k)
    ws = _ensure_ws(workspace, _fused_ws_bytes(P, d, k, False), P.device)
    if out is None:
        out = torch.empty(bh, S_q, d, dtype=out_dtype, device=P.device)
    _check(lib().rmm_pv_reduced(_ptr(P), _ptr(V), bh, S_q, S_k, d, float(rho), _dtype(P), SCORE_MODES[mode],
                                _ptr(out), _out_code(out.dtype), _ptr(idx_out), ws.ptr, ws.nbytes,
                                _stream(P)))
    return out, ws


# ---------------------------------------------------------------- P·V with its softmax producer
def softmax_row_stats(L: torch.Tensor, scale: float = 1.0, causal: bool = True, out: torch.Tensor | None = None,
                      status: torch.Tensor | None = None) -> torch.Tensor:
    """[bh][S_q][2] f32: max of scale·log2(e)·L over each row's visible keys, and 1 / sum exp2(. - max)."""
    bh, S_q, S_k = L.shape
    if not L.is_contiguous():
        raise ValueError("L must be contiguous")
    if out is None:
        out = torch.empty(bh, S_q, 2, dtype=torch.float32, device=L.device)
    _check(lib().rmm_softmax_row_stats(_ptr(L), _dtype(L), float(scale), int(causal), bh, S_q, S_k, _ptr(out),
                                       _ptr(status), _stream(L)))
    return out


def softmax_score(L: torch.Tensor, stats: torch.Tensor, V: torch.Tensor | None = None, scale: float = 1.0,
                  causal: bool = True, score: bool = True, P: torch.Tensor | None = None,
                  s: torch.Tensor | None = None, status: torch.Tensor | None = None):
    """(P, s): P = softmax(scale·L) stored bf16, and (score=True) s[b][k] =
    ||P[b][:, k]|| · ||V[b][k, :]|| (or ||P[b][:, k]|| without V)."""
    bh, S_q, S_k = L.shape
    if not L.is_contiguous():
        raise ValueError("L must be contiguous")
    if V is not None and (V.dtype != torch.bfloat16 or not V.is_contiguous() or V.shape[:2] != (bh, S_k)):
        raise ValueError("V must be a contiguous bf16 [bh][S_k][d] tensor")
    d = V.shape[2] if V is not None else 0
    if P is None:
        P = torch.empty(bh, S_q, S_k, dtype=torch.bfloat16, device=L.device)
    if score and s is None:
        s = torch.empty(bh, S_k, dtype=torch.float32, device=L.device)
    _check(lib().rmm_softmax_score(_ptr(L), _dtype(L), float(scale), int(causal), _ptr(stats), _ptr(V), d, bh, S_q,
                                   S_k, _ptr(P), _ptr(s if score else None), _ptr(status), _stream(L)))
    return P, (s if score else None)


def pv_softmax_workspace_size(bh: int, S_q: int, S_k: int, d: int, k_keep: int) -> int:
    return int(lib().rmm_pv_softmax_workspace_size(bh, S_q, S_k, d, k_keep))


def pv_softmax_reduced(L: torch.Tensor, V: torch.Tensor, rho: float, scale: float = 1.0, causal: bool = True,
                       mode: str = "product", out_dtype=torch.float32, P: torch.Tensor | None = None,
                       out: torch.Tensor | None = None, workspace: Workspace | None = None,
                       idx_out: torch.Tensor | None = None):
    """O ≈ P·V with P = softmax(scale·L) written by the call (bf16) and scored
    as it is written. Returns (O, P, workspace)."""
    bh, S_q, S_k = L.shape
    d = V.shape[2]
    if not L.is_contiguous() or not V.is_contiguous() or V.dtype != torch.bfloat16:
        raise ValueError("L must be contiguous and V a contiguous bf16 tensor")
    k = keep_count(rho, S_k)
    ws = _ensure_ws(workspace, pv_softmax_workspace_size(bh, S_q, S_k, d, k), L.device)
    if P is None:
        P = torch.empty(bh, S_q, S_k, dtype=torch.bfloat16, device=L.device)
    if out is None:
        out = torch.empty(bh, S_q, d, dtype=out_dtype, device=L.device)
    _check(lib().rmm_pv_softmax_reduced(_ptr(L), _dtype(L), float(scale), int(causal), _ptr(V), bh, S_q, S_k, d,
                                        float(rho), SCORE_MODES[mode], _ptr(P), _ptr(out), _out_code(out.dtype),
                                        _ptr(idx_out), ws.ptr, ws.nbytes, _stream(L)))
    return out, P, ws


# ---------------------------------------------------------------- attention
def _tokens(t: torch.Tensor, name: str):
    """(tokens, heads, d, token_stride, head_stride) of a [tokens][heads][d] CUDA tensor."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens][heads][d]")
    n, h, d = t.shape
    ts, hs, es = t.stride()
    if d > 1 and es != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    return n, h, d, ts if n > 1 else h * d, hs if h > 1 else d


def _i32_vec(t: torch.Tensor, name: str, n: int, device):
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements on {device}")
    return t


def _f32_shape(t: torch.Tensor | None, name: str, shape, device):
    if t is not None and (t.dtype != torch.float32 or t.device != device or not t.is_contiguous()
                          or t.shape != shape):
        raise ValueError(f"{name} must be a contiguous float32 {list(shape)} tensor on {device}")
    return t


def _packed(Q: torch.Tensor, K: torch.Tensor, cu_q, cu_k):
    """Sizes and strides of packed queries and keys, and the number of sequences."""
    T_q, h_q, d, q_ts, q_hs = _tokens(Q, "Q")
    T_k, h_kv, dk, k_ts, k_hs = _tokens(K, "K")
    device = Q.device
    if dk != d or K.device != device or K.dtype != Q.dtype:
        raise ValueError("Q and K disagree on d, dtype or device")
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    n = 1 if cu_q is None else cu_q.numel() - 1
    if n < 0:
        raise ValueError("cu_q must hold n_seq + 1 boundaries")
    if cu_q is not None:
        _i32_vec(cu_q, "cu_q", n + 1, device)
        _i32_vec(cu_k, "cu_k", n + 1, device)
    return T_q, T_k, h_q, h_kv, d, q_ts, q_hs, k_ts, k_hs, n


def attn_prompt(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_q: torch.Tensor | None = None,
                cu_k: torch.Tensor | None = None, scale: float | None = None, causal: bool = True,
                out_dtype=torch.float32, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                status: torch.Tensor | None = None):
    """(O, lse): O = softmax(scale·Q·Kᵀ)·V of packed prompts, lse its rows' log-sum-exp.

    Q [T_q][h_q][d], K, V [T_k][h_kv][d] bf16; sequence i's tokens are
    [cu[i], cu[i+1]) (int32, on the device; None: one sequence). With causal,
    query q sees key k when k <= q + S_k - S_q. scale defaults to 1/sqrt(d).
    O [T_q][h_q][d]; lse f32 [h_q][T_q]. The probabilities are rounded to bf16
    before they multiply V, whatever O's dtype (f32 sums, unrounded row sums)."""
    T_q, T_k, h_q, h_kv, d, q_ts, q_hs, k_ts, k_hs, n = _packed(Q, K, cu_q, cu_k)
    tv, hv, dv, v_ts, v_hs = _tokens(V, "V")
    device = Q.device
    if tv != T_k or hv != h_kv or dv != d or V.device != device or V.dtype != Q.dtype:
        raise ValueError("K and V disagree on shape, dtype or device")
    if out is None:
        out = torch.empty(T_q, h_q, d, dtype=out_dtype, device=device)
        o_ts, o_hs = h_q * d, d
    elif out.shape != (T_q, h_q, d) or out.device != device:
        raise ValueError("out must be [T_q][h_q][d] on Q's device")
    else:
        _, _, _, o_ts, o_hs = _tokens(out, "out")
    if lse is None:
        lse = torch.empty(h_q, T_q, dtype=torch.float32, device=device)
    else:
        _f32_shape(lse, "lse", (h_q, T_q), device)
    status_code = lib().rmm_attn_prompt(
        Q.data_ptr(), q_ts, q_hs, K.data_ptr(), k_ts, k_hs, V.data_ptr(), v_ts, v_hs, _ptr(cu_q), _ptr(cu_k), n, T_q, T_k,
        h_q, h_kv, d, d ** -0.5 if scale is None else float(scale), int(causal), _dtype(Q), out.data_ptr(), o_ts, o_hs,
        _out_code(out.dtype), lse.data_ptr(), _status_ptr(status, device), _stream(Q))
    if status_code:
        _check(status_code)
    return out, lse


def attn_key_weights(Q: torch.Tensor, K: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor | None = None,
                     cu_k: torch.Tensor | None = None, scale: float | None = None, causal: bool = True,
                     w_in: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     status: torch.Tensor | None = None) -> torch.Tensor:
    """[h_kv][T_k] f32: w_in (or 0) plus the attention each key received, summed
    over its sequence's queries and over the query heads that read its head.
    Arguments as attn_prompt's, whose lse it takes; out may be w_in."""
    T_q, T_k, h_q, h_kv, d, q_ts, q_hs, k_ts, k_hs, n = _packed(Q, K, cu_q, cu_k)
    _f32_shape(lse, "lse", (h_q, T_q), Q.device)
    _f32_shape(w_in, "w_in", (h_kv, T_k), Q.device)
    if out is None:
        out = torch.empty(h_kv, T_k, dtype=torch.float32, device=Q.device)
    _f32_shape(out, "out", (h_kv, T_k), Q.device)
    _check(lib().rmm_attn_key_weights(_ptr(Q), q_ts, q_hs, _ptr(K), k_ts, k_hs, _ptr(cu_q), _ptr(cu_k), n, T_q, T_k,
                                      h_q, h_kv, d, float(d ** -0.5 if scale is None else scale), int(causal),
                                      _dtype(Q), _ptr(lse), _ptr(w_in), _ptr(out), _status_ptr(status, Q.device),
                                      _stream(Q)))
    return out


KV4_GROUP = 32


class KV4Cache:
    """The planes of a cache of keys and values in 4 bits (include/rmm.h has the
    layout): kc, vc [batch][heads][cap][d/2] uint8 codes, ks, vs
    [batch][heads][cap][d/32][2] bf16 steps and minima, optionally w
    [batch][heads][cap] f32, the tokens' running attention weights, and
    optionally a status word that stores into the cache report to (empty() makes
    both)."""

    def __init__(self, kc: torch.Tensor, ks: torch.Tensor, vc: torch.Tensor, vs: torch.Tensor,
                 w: torch.Tensor | None = None, status: torch.Tensor | None = None):
        codes, device = kc.shape, kc.device
        if len(codes) != 4 or kc.dtype != torch.uint8 or not kc.is_cuda:
            raise ValueError("kc must be a [batch][heads][cap][d/2] uint8 CUDA tensor")
        self.batch, self.heads, self.cap, half = codes
        self.d = 2 * half
        scales = (self.batch, self.heads, self.cap, self.d // KV4_GROUP, 2)
        if not (vc.dtype == torch.uint8 and ks.dtype == torch.bfloat16 and vs.dtype == torch.bfloat16
                and vc.shape == codes and ks.shape == scales and vs.shape == scales and kc.is_contiguous()
                and vc.is_contiguous() and ks.is_contiguous() and vs.is_contiguous() and vc.device == device
                and ks.device == device and vs.device == device):
            raise ValueError(f"kc, vc must be contiguous uint8 {list(codes)} and ks, vs contiguous bfloat16 "
                             f"{list(scales)} tensors on {device}")
        self.kc, self.ks, self.vc, self.vs = kc, ks, vc, vs
        self.w = None if w is None else _f32_shape(w, "w", (self.batch, self.heads, self.cap), device)
        _status_ptr(status, device)
        self.status = status

    @classmethod
    def empty(cls, batch: int, heads: int, cap: int, d: int, device="cuda", weights: bool = True) -> "KV4Cache":
        """A cache with room for `cap` tokens per sequence (zeroed)."""
        if d % KV4_GROUP:
            raise ValueError(f"d must be a multiple of {KV4_GROUP}")
        codes = lambda: torch.zeros(batch, heads, cap, d // 2, dtype=torch.uint8, device=device)  # noqa: E731
        scales = lambda: torch.zeros(batch, heads, cap, d // KV4_GROUP, 2, dtype=torch.bfloat16,  # noqa: E731
                                     device=device)
        w = torch.zeros(batch, heads, cap, dtype=torch.float32, device=device) if weights else None
        return cls(codes(), scales(), codes(), scales(), w, status_word(device))

    def planes(self):
        """The tensors whose rows belong to a token, for cache_evict."""
        return [self.kc, self.ks, self.vc, self.vs] + ([self.w] if self.w is not None else [])


def kv4_store(cache: KV4Cache, K: torch.Tensor, V: torch.Tensor, start: torch.Tensor,
              cu: torch.Tensor | None = None, w_new: torch.Tensor | None = None,
              status: torch.Tensor | None = None) -> KV4Cache:
    """Quantise tokens into the cache: K, V [T][heads][d] (bf16 or f32), sequence
    b's tokens [cu[b], cu[b+1]) going to its slots start[b], start[b] + 1, ...
    (cu None: one token per sequence). The slots' running weights are set to
    w_new [heads][T], or to 0.

    A token whose slot lies outside the cache's capacity is left out, and a
    NaN, Inf or overflowing group is stored as it may be; both are reported in
    `status` (None: the cache's own word) and raise at the next
    check(cache.status), which waits for the stream."""
    T, h, d, k_ts, k_hs = _tokens(K, "K")
    tv, hv, dv, v_ts, v_hs = _tokens(V, "V")
    if tv != T or hv != h or dv != d or h != cache.heads or d != cache.d or V.dtype != K.dtype:
        raise ValueError("K, V and the cache disagree on shape or dtype")
    kc, batch, device = cache.kc, cache.batch, K.device
    if kc.device != device or V.device != device:
        raise ValueError("K, V and the cache must be on one device")
    _i32_vec(start, "start", batch, device)
    if cu is not None:
        _i32_vec(cu, "cu", batch + 1, device)
    if w_new is not None:
        _f32_shape(w_new, "w_new", (h, T), device)
    status_code = lib().rmm_kv4_store(
        K.data_ptr(), k_ts, k_hs, V.data_ptr(), v_ts, v_hs, _dtype(K), _ptr(cu), start.data_ptr(), batch, T, h, d,
        cache.cap, kc.data_ptr(), cache.ks.data_ptr(), cache.vc.data_ptr(), cache.vs.data_ptr(), _ptr(w_new),
        _ptr(cache.w), _status_ptr(cache.status if status is None else status, device), _stream(K))
    if status_code:
        _check(status_code)
    return cache


@functools.lru_cache(maxsize=1024)
def kv4_attn_workspace_size(batch: int, h_q: int, h_kv: int, d: int, cap: int, weights: bool = False) -> int:
    return int(lib().rmm_kv4_attn_workspace_size(batch, h_q, h_kv, d, cap, int(weights)))


def kv4_attn(Q: torch.Tensor, cache: KV4Cache, lens: torch.Tensor, scale: float | None = None,
             out_dtype=torch.float32, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
             w_in: torch.Tensor | None = None, w_out: torch.Tensor | None = None,
             workspace: Workspace | None = None):
    """(O, lse, workspace): one decode step, Q [batch][h_q][d] bf16 over the first
    lens[b] cached tokens of each sequence. With w_out ([batch][heads][cap] f32)
    the tokens' probabilities, summed over the query heads of their head, are
    added to w_in (None: 0) and written to w_out, which may be w_in."""
    n, h_q, d, q_ss, q_hs = _tokens(Q, "Q")
    kc, heads, cap, device = cache.kc, cache.heads, cache.cap, Q.device
    if n != cache.batch or d != cache.d or kc.device != device:
        raise ValueError("Q and the cache disagree on batch, d or device")
    _i32_vec(lens, "lens", n, device)
    if w_in is not None:
        _f32_shape(w_in, "w_in", (n, heads, cap), device)
    if w_out is not None:
        _f32_shape(w_out, "w_out", (n, heads, cap), device)
    ws = _ensure_ws(workspace, kv4_attn_workspace_size(n, h_q, heads, d, cap, w_out is not None), device)
    if out is None:
        out = torch.empty(n, h_q, d, dtype=out_dtype, device=device)
        o_ss, o_hs = h_q * d, d
    elif out.shape != (n, h_q, d) or out.device != device:
        raise ValueError("out must be [batch][h_q][d] on Q's device")
    else:
        _, _, _, o_ss, o_hs = _tokens(out, "out")
    if lse is None:
        lse = torch.empty(n, h_q, dtype=torch.float32, device=device)
    else:
        _f32_shape(lse, "lse", (n, h_q), device)
    status_code = lib().rmm_kv4_attn(
        Q.data_ptr(), q_ss, q_hs, kc.data_ptr(), cache.ks.data_ptr(), cache.vc.data_ptr(), cache.vs.data_ptr(),
        lens.data_ptr(), n, h_q, heads, d, cap, d ** -0.5 if scale is None else float(scale), _dtype(Q), out.data_ptr(),
        o_ss, o_hs, _out_code(out.dtype), lse.data_ptr(), _ptr(w_in), _ptr(w_out), ws.ptr, ws.nbytes, _stream(Q))
    if status_code:
        _check(status_code)
    return out, lse, ws


@functools.lru_cache(maxsize=1024)
def cache_evict_workspace_size(batch: int, heads: int, budget: int) -> int:
    return int(lib().rmm_cache_evict_workspace_size(batch, heads, budget))


def cache_evict(w: torch.Tensor, lens: torch.Tensor, planes, budget: int, sink: int = 0, recent: int = 0,
                lens_out: torch.Tensor | None = None, idx_out: torch.Tensor | None = None,
                workspace: Workspace | None = None):
    """(lens_out, idx, workspace): keep at most `budget` cached tokens per
    (sequence, head): the first `sink`, the last `recent`, and of the others
    those of greatest weight w [batch][heads][cap] (ties to the lower index).

    planes: the tensors [batch][heads][cap][...] whose rows move with the
    tokens, each alone (moved in place; KV4Cache.planes()) or as a pair (src,
    dst [batch][heads][cap_out][...]). idx [batch][heads][budget] holds the kept
    tokens' former indices, -1 past them. lens_out may be lens."""
    if w.dim() != 3 or w.dtype != torch.float32 or not w.is_cuda or not w.is_contiguous():
        raise ValueError("w must be a contiguous float32 [batch][heads][cap] CUDA tensor")
    head, device, budget = w.shape, w.device, int(budget)
    batch, heads, cap = head
    _i32_vec(lens, "lens", batch, device)
    cap_out, vals = None, []
    for i, pair in enumerate(planes):
        src, dst = pair if isinstance(pair, tuple) else (pair, pair)
        shape, out_shape = src.shape, dst.shape
        if cap_out is None and len(out_shape) >= 3:
            cap_out = out_shape[2]
        if (len(shape) < 3 or (shape if len(shape) == 3 else shape[:3]) != head or src.dtype != dst.dtype or not src.is_contiguous() or src.device != device
                or (cap_out != cap if dst is src else out_shape[:2] != head[:2] or out_shape[2:3] != (cap_out,)
                    or out_shape[3:] != shape[3:] or not dst.is_contiguous() or dst.device != device)):
            raise ValueError(f"plane {i}: src and dst must be contiguous [batch][heads][cap][...] tensors like w, "
                             "the destinations of one capacity")
        row = src.element_size()
        for n in shape[3:]:
            row *= n
        vals += (src.data_ptr(), dst.data_ptr(), row)
    n_planes = len(vals) // 3
    if cap_out is None:
        cap_out = max(cap, budget)
    arr = (ctypes.c_int64 * max(3, len(vals)))(*vals)  # rmm_cache_plane: two pointers and the row's bytes
    if lens_out is None:
        lens_out = torch.empty(batch, dtype=torch.int32, device=device)
    else:
        _i32_vec(lens_out, "lens_out", batch, device)
    if idx_out is None:
        idx_out = torch.empty(batch, heads, budget, dtype=torch.int32, device=device)
    else:
        _i32_vec(idx_out, "idx_out", batch * heads * budget, device)
    ws = _ensure_ws(workspace, cache_evict_workspace_size(batch, heads, budget), device)
    status_code = lib().rmm_cache_evict(
        w.data_ptr(), lens.data_ptr(), batch, heads, cap, budget, int(sink), int(recent), arr, n_planes, cap_out,
        lens_out.data_ptr(), idx_out.data_ptr(), ws.ptr, ws.nbytes, _stream(w))
    if status_code:
        _check(status_code)
    return lens_out, idx_out, ws


def set_wait_limit_ns(ns: int):
    lib().rmm_set_wait_limit_ns(int(ns))


def set_stall_producer_for_test(on: bool):
    lib().rmm_set_stall_producer_for_test(int(bool(on)))


def set_gemm_cta_group(cta_group: int) -> int:
    """2 = 2-SM MMAs on CTA pairs (default), 1 = one SM per tile; returns the previous value."""
    return int(lib().rmm_set_gemm_cta_group(int(cta_group)))


def launch_count() -> int:
    return int(lib().rmm_launch_count())


def set_debug(on: bool) -> bool:
    """Debug checks (kept indices validated on the device before a stage call
    reads through them; fused calls report their device status directly).
    Returns the previous setting."""
    return bool(lib().rmm_set_debug(int(bool(on))))


def set_gemm_events(start: torch.cuda.Event | None, stop: torch.cuda.Event | None):
    """Record `start`/`stop` immediately around every GEMM kernel launch (None, None clears)."""
    def handle(e):
        if e is None:
            return ctypes.c_void_p(0)
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record()
        return ctypes.c_void_p(e.cuda_event)

    lib().rmm_set_gemm_events(handle(start), handle(stop))


def matmul_reduced_noalloc(A: torch.Tensor, B: torch.Tensor, rho: float, mode: str = "product",
                           out_dtype=torch.float32, out: torch.Tensor | None = None,
                           idx_out: torch.Tensor | None = None, status: torch.Tensor | None = None):
    """C ≈ A·B like matmul_reduced, but with the library's static 32 MiB device
    scratch instead of a workspace, for callers that must not allocate device
    memory (only C is allocated here, and only when `out` is None)."""
    _, M, K, lda, _ = _mat(A, "A")
    _, r, N, ldb, _ = _mat(B, "B")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=A.device)
    _, _, _, ldc, _ = _mat(out, "C")
    _check(lib().rmm_matmul_reduced_noalloc(_ptr(A), lda, _ptr(B), ldb, M, K, N, float(rho), _dtype(A),
                                            SCORE_MODES[mode], _ptr(out), ldc, _out_code(out.dtype), _ptr(idx_out),
                                            _ptr(status), _stream(A)))
    return out
