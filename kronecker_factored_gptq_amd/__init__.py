"""MI355X-native BaKron solver.

A thin Python binding over the C ABI of ``libbakron.so`` (include/bakron.h):
argument marshalling only. PyTorch supplies device memory and streams; every
step of the computation runs in the library's HIP kernels. The binding fails
loudly when the library is missing; there is no fallback path.

BaKron ("BaKron: Efficient Quantization with Kronecker-Factored Hessians",
arXiv 2608.06291) quantises W (m x n) with GPTQ on vec(W) under the Hessian
A (x) B, A n x n (input side) and B m x m (output side).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple, Union

import torch

__all__ = ["F32", "F64", "BF16", "F16", "SCALE_NONE", "SCALE_ROW", "SCALE_COL", "BakronError", "lib", "factor",
           "factor_batched",
           "solve", "solve_antidiag", "solve_noalloc", "factor_blockdiag", "solve_blockdiag",
           "loss_blockdiag", "solve_batched", "loss", "loss_batched", "row_scales", "row_scales_mse", "gram",
           "sample_sqnorms", "kfac_factors", "shampoo_factors", "quantize_tokens", "matmul_int8",
           "matmul_int8_grad", "cross_entropy", "cross_entropy_grad", "quantize_fp8", "matmul_fp8", "matmul_fp8_grad",
           "sort_tokens", "gather_tokens", "combine_tokens", "combine_tokens_grad", "solve_schedule", "tile_size",
           "workspace_bytes"]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libbakron.so")

F32, F64, BF16, F16 = 0, 1, 2, 3
SCALE_NONE, SCALE_ROW, SCALE_COL = 0, 1, 2
OK, EINVAL, ENOTSPD, EHIP, EWAIT = 0, -1, -2, -3, -4


class BakronError(RuntimeError):
    def __init__(self, status: int, what: str, bad_pivot: Optional[Tuple[int, int]] = None):
        self.status = status
        self.bad_pivot = bad_pivot
        msg = f"{what}: {_status_string(status)} (status {status})"
        if bad_pivot is not None and bad_pivot[0] >= 0:
            side = "A" if bad_pivot[0] == 0 else "B"
            msg += f"; failing pivot {bad_pivot[1]} of the reversed Cholesky of {side}"
        super().__init__(msg)


_lib = None
_vp, _i64, _i32, _sz, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int


def lib() -> ctypes.CDLL:
    """Load libbakron.so (built by __graft_entry__.build() or
    ``python -m kronecker_factored_gptq_amd.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(f"{LIB_PATH} is not built; run `python -m kronecker_factored_gptq_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    L.bakron_status_string.argtypes = [_int]
    L.bakron_status_string.restype = ctypes.c_char_p
    L.bakron_abi_version.argtypes = []
    L.bakron_abi_version.restype = _int
    L.bakron_tile_size.argtypes = [_int]
    L.bakron_tile_size.restype = _int
    for name in ("bakron_factor_workspace_bytes", "bakron_solve_workspace_bytes",
                 "bakron_loss_workspace_bytes"):
        f = getattr(L, name)
        f.argtypes = [_int, _i64, _i64]
        f.restype = _sz
    L.bakron_factor.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                _vp, _vp, _vp, _sz, ctypes.POINTER(_i64), _vp]
    L.bakron_factor.restype = _int
    L.bakron_solve.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i32, _i32,
                               _int, _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp]
    L.bakron_solve.restype = _int
    for name in ("bakron_factor_blockdiag_workspace_bytes", "bakron_solve_blockdiag_workspace_bytes",
                 "bakron_loss_blockdiag_workspace_bytes"):
        f = getattr(L, name)
        f.argtypes = [_int, _i64, _i64, _i64]
        f.restype = _sz
    L.bakron_factor_blockdiag.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp,
                                          _i64, _vp, _i64, _i64, _vp, _vp, _vp, _sz,
                                          ctypes.POINTER(_i64), _vp]
    L.bakron_factor_blockdiag.restype = _int
    L.bakron_solve_blockdiag.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                         _i64, _i32, _i32, _i32, _int, _vp, _vp, _i64, _vp, _i64,
                                         _vp, _sz, _vp]
    L.bakron_solve_blockdiag.restype = _int
    L.bakron_loss_blockdiag.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp,
                                        _vp, _i64, _vp, _i64, _i64, _vp, _vp, _sz, _vp]
    L.bakron_loss_blockdiag.restype = _int
    L.bakron_solve_antidiag_workspace_bytes.argtypes = [_int, _i64, _i64]
    L.bakron_solve_antidiag_workspace_bytes.restype = _sz
    L.bakron_solve_antidiag.argtypes = L.bakron_solve.argtypes
    L.bakron_solve_antidiag.restype = _int
    L.bakron_solve_noalloc.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32,
                                       _i32, _i32, _int, _vp, _vp, _i64, _vp, _i64, _vp]
    L.bakron_solve_noalloc.restype = _int
    L.bakron_solve_timed.argtypes = L.bakron_solve.argtypes + [_vp, _i64]
    L.bakron_solve_timed.restype = _int
    L.bakron_solve_status.argtypes = [_int, _i64, _i64, _i64, _vp, _sz, _vp]
    L.bakron_solve_status.restype = _int
    L.bakron_debug_set_wait_polls.argtypes = [_i32]
    L.bakron_debug_set_wait_polls.restype = _i32
    L.bakron_solve_schedule.argtypes = [_int, _i64, _i64, _vp, _i64]
    L.bakron_solve_schedule.restype = _i64
    L.bakron_factor_batched_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.bakron_factor_batched_workspace_bytes.restype = _sz
    L.bakron_factor_batched.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                        _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64,
                                        _vp, _sz, ctypes.POINTER(_i64), _vp]
    L.bakron_factor_batched.restype = _int
    L.bakron_solve_batched_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.bakron_solve_batched_workspace_bytes.restype = _sz
    L.bakron_solve_batched.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                       _vp, _i64, _i64, _i32, _i32, _i32, _int, _vp, _i64,
                                       _vp, _i64, _i64, _vp, _i64, _i64, _vp, _sz, _vp]
    L.bakron_solve_batched.restype = _int
    L.bakron_loss.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _vp, _i64, _vp,
                              _i64, _vp, _vp, _sz, _vp]
    L.bakron_loss.restype = _int
    L.bakron_loss_batched_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.bakron_loss_batched_workspace_bytes.restype = _sz
    L.bakron_loss_batched.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                      _int, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp,
                                      _sz, _vp]
    L.bakron_loss_batched.restype = _int
    L.bakron_row_scales.argtypes = [_int, _i64, _i64, _vp, _i64, _i32, _vp, _vp]
    L.bakron_row_scales.restype = _int
    L.bakron_row_scales_mse.argtypes = [_int, _i64, _i64, _vp, _i64, _i32, _i32, _i32,
                                        ctypes.c_double, _vp, _vp]
    L.bakron_row_scales_mse.restype = _int
    L.bakron_gram.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, ctypes.c_double, _vp, _i64, _vp]
    L.bakron_gram.restype = _int
    L.bakron_sample_sqnorms.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _vp]
    L.bakron_sample_sqnorms.restype = _int
    L.bakron_quantize_tokens.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp]
    L.bakron_quantize_tokens.restype = _int
    L.bakron_matmul_int8.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp,
                                     _i64, _vp, _sz, _vp]
    L.bakron_matmul_int8.restype = _int
    L.bakron_matmul_int8_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.bakron_matmul_int8_workspace_bytes.restype = _sz
    L.bakron_matmul_int8_grad_workspace_bytes.argtypes = [_int, _i64, _i64, _i64]
    L.bakron_matmul_int8_grad_workspace_bytes.restype = _sz
    L.bakron_matmul_int8_grad.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp,
                                          _vp, _i64, _vp, _sz, _vp]
    L.bakron_matmul_int8_grad.restype = _int
    for name in ("bakron_cross_entropy_workspace_bytes", "bakron_cross_entropy_grad_workspace_bytes"):
        f = getattr(L, name)
        f.argtypes = [_int, _i64, _i64, _i64]
        f.restype = _sz
    L.bakron_cross_entropy.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                       _vp, _sz, _vp]
    L.bakron_cross_entropy.restype = _int
    L.bakron_cross_entropy_grad.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp,
                                            _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp]
    L.bakron_cross_entropy_grad.restype = _int
    L.bakron_quantize_fp8.argtypes = [_int, _i64, _i64, _i64, _vp, _i64, _i64, _int, _vp, _i64, _i64, _vp, _i64,
                                      _i64, _i64, _vp]
    L.bakron_quantize_fp8.restype = _int
    for f in (L.bakron_matmul_fp8_workspace_bytes, L.bakron_matmul_fp8_aligned_workspace_bytes):
        f.argtypes = [_int, _i64, _i64, _i64, _i64, _i64]
        f.restype = _sz
    L.bakron_matmul_fp8.argtypes = [_int, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                    _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _sz, _vp]
    L.bakron_matmul_fp8.restype = _int
    for f in (L.bakron_matmul_fp8_grad_workspace_bytes, L.bakron_matmul_fp8_grad_aligned_workspace_bytes):
        f.argtypes = [_int, _i64, _i64, _i64, _i64]
        f.restype = _sz
    L.bakron_matmul_fp8_grad.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i64, _i64,
                                         _vp, _vp, _i64, _vp, _sz, _vp]
    L.bakron_matmul_fp8_grad.restype = _int
    L.bakron_sort_tokens_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.bakron_sort_tokens_workspace_bytes.restype = _sz
    L.bakron_sort_tokens.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
    L.bakron_sort_tokens.restype = _int
    L.bakron_gather_tokens.argtypes = [_int, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp]
    L.bakron_gather_tokens.restype = _int
    L.bakron_combine_tokens.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
    L.bakron_combine_tokens.restype = _int
    L.bakron_combine_tokens_grad.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64,
                                             _vp, _vp]
    L.bakron_combine_tokens_grad.restype = _int
    L.bakron_debug_plan.argtypes = [_i64, _i64, _i64, _int, _int, _int, _vp, _vp]
    L.bakron_debug_plan.restype = ctypes.c_double
    _lib = L
    return L


def _status_string(status: int) -> str:
    try:
        return lib().bakron_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - library missing
        return "unknown"


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.float64:
        return F64
    raise TypeError(f"expected float32 or float64, got {t.dtype}")


def _tdt(code: int) -> torch.dtype:
    return torch.float32 if code == F32 else torch.float64


def _ld(t: torch.Tensor, name: str) -> int:
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    return max(int(t.stride(0)), int(t.size(1)), 1)


def _check_out(t: torch.Tensor, shape, dtype: torch.dtype, name: str) -> None:
    """A caller-supplied output must have exactly the shape and element type
    the kernels write, with unit column stride (the C ABI only sees its
    pointer and leading dimension)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() == 2 and t.size(1) > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if t.dim() == 2 and t.size(0) > 1 and t.stride(0) < t.size(1):
        raise ValueError(f"{name} rows overlap (leading dimension below the row length)")


def _check_operand(t: torch.Tensor, shape, dtype: torch.dtype, name: str) -> None:
    """An input read by the kernels: exact shape and element type."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_device(*ts):
    dev = index = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i < 0 or not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")
        if dev is None:
            dev, index = t.device, i
        elif i != index:
            raise ValueError("all tensors must be on one device")
    return dev


def _stream(dev) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _workspace(nbytes: int, dev, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return ws
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=dev)


def tile_size(dtype: int = F32) -> int:
    return int(lib().bakron_tile_size(int(dtype)))


def workspace_bytes(kind: str, dtype: int, m: int, n: int) -> int:
    f = {"factor": lib().bakron_factor_workspace_bytes, "solve": lib().bakron_solve_workspace_bytes,
         "loss": lib().bakron_loss_workspace_bytes}[kind]
    return int(f(int(dtype), int(m), int(n)))


def factor(A: torch.Tensor, B: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
           workspace: Optional[torch.Tensor] = None):
    """L^A = Cholesky(A^-1), L^B = Cholesky(B^-1), columns normalised by their
    diagonals (§3.2 Algorithm 2), plus the diagonals dA, dB. Synchronous.
    Raises BakronError(ENOTSPD) for a non-positive-definite input."""
    dev = _check_device(A, B)
    code = _dt(A)
    if B.dtype != A.dtype:
        raise TypeError("A and B must have the same dtype")
    if out_dtype is not None and out_dtype != A.dtype:
        raise TypeError("out_dtype must equal the input dtype")
    n, m = A.size(0), B.size(0)
    if A.shape != (n, n) or B.shape != (m, m):
        raise ValueError("A and B must be square")
    LA = torch.empty((n, n), dtype=A.dtype, device=dev)
    LB = torch.empty((m, m), dtype=A.dtype, device=dev)
    dA = torch.empty(n, dtype=A.dtype, device=dev)
    dB = torch.empty(m, dtype=A.dtype, device=dev)
    L = lib()
    nbytes = L.bakron_factor_workspace_bytes(code, m, n)
    ws = _workspace(nbytes, dev, workspace)
    bad = (_i64 * 2)(-1, -1)
    with torch.cuda.device(dev):
        rc = L.bakron_factor(code, m, n, _p(A), _ld(A, "A"), _p(B), _ld(B, "B"), _p(LA), n,
                             _p(LB), m, _p(dA), _p(dB), _p(ws), ws.numel(), bad, _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_factor", (int(bad[0]), int(bad[1])))
    return LA, LB, dA, dB


def factor_batched(A: torch.Tensor, B: torch.Tensor, workspace: Optional[torch.Tensor] = None):
    """bakron_factor on a batch of pairs of the same orders in the same
    launches. A is (batch, n, n), B (batch, m, m). Returns LA (batch, n, n),
    LB (batch, m, m), dA (batch, n), dB (batch, m); each pair's result is
    bit-identical to ``factor``. Synchronous. Raises BakronError(ENOTSPD)
    with ``bad_pivot`` = (pair, side, index)."""
    dev = _check_device(A, B, workspace)
    code = _dt(A)
    if B.dtype != A.dtype:
        raise TypeError("A and B must have the same dtype")
    if A.dim() != 3 or B.dim() != 3 or A.size(0) != B.size(0):
        raise ValueError("A must be (batch, n, n) and B (batch, m, m)")
    batch, n, m = A.size(0), A.size(1), B.size(1)
    pa, lda, sa = _batch_operand(A, n, n, batch, "A")
    pb, ldb, sb = _batch_operand(B, m, m, batch, "B")
    LA = torch.empty((batch, n, n), dtype=A.dtype, device=dev)
    LB = torch.empty((batch, m, m), dtype=A.dtype, device=dev)
    dA = torch.empty((batch, n), dtype=A.dtype, device=dev)
    dB = torch.empty((batch, m), dtype=A.dtype, device=dev)
    L = lib()
    ws = _workspace(L.bakron_factor_batched_workspace_bytes(code, batch, m, n), dev, workspace)
    bad = (_i64 * 3)(-1, -1, -1)
    with torch.cuda.device(dev):
        rc = L.bakron_factor_batched(code, batch, m, n, pa, lda, sa, pb, ldb, sb, _p(LA), max(n, 1),
                                     n * n, _p(LB), max(m, 1), m * m, _p(dA), n, _p(dB), m, _p(ws),
                                     ws.numel() * ws.element_size(), bad, _stream(dev))
    if rc != OK:
        err = BakronError(rc, "bakron_factor_batched", (int(bad[1]), int(bad[2])))
        err.bad_pivot = (int(bad[0]), int(bad[1]), int(bad[2]))
        raise err
    return LA, LB, dA, dB


AlphabetLike = Union[Sequence[int], Tuple[int, int, int]]


def _scale_mode(scales: Optional[torch.Tensor], m: int, n: int, scale_mode: Optional[int]) -> int:
    if scales is None:
        if scale_mode not in (None, SCALE_NONE):
            raise ValueError("scales required for this scale_mode")
        return SCALE_NONE
    if scale_mode is None:
        if scales.numel() == m:
            return SCALE_ROW
        if scales.numel() == n:
            return SCALE_COL
        raise ValueError("scales must have length m (rows) or n (columns)")
    want = m if scale_mode == SCALE_ROW else n
    if scale_mode not in (SCALE_ROW, SCALE_COL) or scales.numel() != want:
        raise ValueError("scales do not match scale_mode")
    return scale_mode


def solve(W: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor, alphabet: AlphabetLike = (0, 0, 1),
          scales: Optional[torch.Tensor] = None, scale_mode: Optional[int] = None,
          return_wt: bool = False, workspace: Optional[torch.Tensor] = None,
          out: Optional[torch.Tensor] = None, op_ms: Optional[ctypes.Array] = None,
          check: bool = False):
    """BaKron solve (§3.5 Algorithm 6 on a tiling of W). Returns int32 codes V
    (m x n), and with ``return_wt`` also the value each entry had when it was
    rounded. Asynchronous on the current stream, except with ``op_ms`` (a
    ctypes double array, one slot per schedule record: every leaf-block and
    band-product launch is timed with HIP events and the call waits for
    them) or ``check`` (waits, then raises BakronError(EWAIT) if a leaf
    block's bounded wait gave up)."""
    dev = _check_device(W, LA, LB, scales, workspace, out)
    code = _dt(W)
    m, n = W.shape
    if LA.shape != (n, n) or LB.shape != (m, m) or LA.dtype != W.dtype or LB.dtype != W.dtype:
        raise ValueError("LA must be n x n and LB m x m, same dtype as W")
    lo, hi, unb = (int(alphabet[0]), int(alphabet[1]), int(bool(alphabet[2])))
    mode = _scale_mode(scales, m, n, scale_mode)
    if scales is not None:
        if scales.dtype != W.dtype or not scales.is_contiguous():
            raise ValueError("scales must be contiguous with W's dtype")
    if out is not None:
        _check_out(out, (m, n), torch.int32, "out")
    V = out if out is not None else torch.empty((m, n), dtype=torch.int32, device=dev)
    Wt = torch.empty((m, n), dtype=W.dtype, device=dev) if return_wt else None
    L = lib()
    ws = _workspace(L.bakron_solve_workspace_bytes(code, m, n), dev, workspace)
    args = (code, m, n, _p(W), _ld(W, "W"), _p(LA), _ld(LA, "LA"), _p(LB), _ld(LB, "LB"), lo, hi,
            unb, mode, _p(scales), _p(V), _ld(V, "V"), _p(Wt),
            _ld(Wt, "Wt") if Wt is not None else 0, _p(ws), ws.numel() * ws.element_size(),
            _stream(dev))
    with torch.cuda.device(dev):
        if op_ms is None:
            rc = L.bakron_solve(*args)
        else:
            rc = L.bakron_solve_timed(*args, ctypes.cast(op_ms, ctypes.c_void_p), len(op_ms))
    if rc == OK and check:
        rc = L.bakron_solve_status(code, 1, m, n, _p(ws), ws.numel() * ws.element_size(),
                                   _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_solve")
    return (V, Wt) if return_wt else V


def solve_antidiag(W: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor,
                   alphabet: AlphabetLike = (0, 0, 1), scales: Optional[torch.Tensor] = None,
                   scale_mode: Optional[int] = None, return_wt: bool = False,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None):
    """BaKron-antidiagonal (§3.3 Algorithm 3 on the whole matrix, one launch
    per anti-diagonal): the same codes as ``solve`` (Theorem 3.2) with
    O(m^2 n^2) work, the paper's point of comparison. Arguments and results
    as for ``solve``. Asynchronous on the current stream."""
    dev = _check_device(W, LA, LB, scales, workspace, out)
    code = _dt(W)
    m, n = W.shape
    if LA.shape != (n, n) or LB.shape != (m, m) or LA.dtype != W.dtype or LB.dtype != W.dtype:
        raise ValueError("LA must be n x n and LB m x m, same dtype as W")
    lo, hi, unb = (int(alphabet[0]), int(alphabet[1]), int(bool(alphabet[2])))
    mode = _scale_mode(scales, m, n, scale_mode)
    if scales is not None and (scales.dtype != W.dtype or not scales.is_contiguous()):
        raise ValueError("scales must be contiguous with W's dtype")
    if out is not None:
        _check_out(out, (m, n), torch.int32, "out")
    V = out if out is not None else torch.empty((m, n), dtype=torch.int32, device=dev)
    Wt = torch.empty((m, n), dtype=W.dtype, device=dev) if return_wt else None
    L = lib()
    ws = _workspace(L.bakron_solve_antidiag_workspace_bytes(code, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_solve_antidiag(code, m, n, _p(W), _ld(W, "W"), _p(LA), _ld(LA, "LA"), _p(LB),
                                     _ld(LB, "LB"), lo, hi, unb, mode, _p(scales), _p(V),
                                     _ld(V, "V"), _p(Wt), _ld(Wt, "Wt") if Wt is not None else 0,
                                     _p(ws), ws.numel() * ws.element_size(), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_solve_antidiag")
    return (V, Wt) if return_wt else V


def _blocks(t: torch.Tensor, heads: int, b: int, name: str):
    """(pointer, ld, stride) of h square blocks given as a (heads, b, b) tensor."""
    if t.dim() != 3 or t.shape != (heads, b, b):
        raise ValueError(f"{name} must be ({heads}, {b}, {b})")
    if b > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    ld = max(int(t.stride(1)), b, 1)
    return _p(t), ld, int(t.stride(0)) if heads > 1 else 0


def factor_blockdiag(A: torch.Tensor, Bblocks: torch.Tensor, workspace: Optional[torch.Tensor] = None):
    """L^A of A (n x n) and the normalised Cholesky(B_h^-1) of every block of
    a block-diagonal output factor B = blockdiag(Bblocks[h]) (Bblocks is
    (heads, b, b)). Returns LA (n x n), LB blocks (heads, b, b), dA (n),
    dB (heads * b). Synchronous. BakronError.bad_pivot = (side, block, index)."""
    dev = _check_device(A, Bblocks, workspace)
    code = _dt(A)
    if Bblocks.dtype != A.dtype:
        raise TypeError("A and the B blocks must have the same dtype")
    n = A.size(0)
    if A.shape != (n, n) or Bblocks.dim() != 3:
        raise ValueError("A must be n x n and Bblocks (heads, b, b)")
    heads, b = Bblocks.size(0), Bblocks.size(1)
    pb, ldb, sb = _blocks(Bblocks, heads, b, "Bblocks")
    LA = torch.empty((n, n), dtype=A.dtype, device=dev)
    LB = torch.empty((heads, b, b), dtype=A.dtype, device=dev)
    dA = torch.empty(n, dtype=A.dtype, device=dev)
    dB = torch.empty(heads * b, dtype=A.dtype, device=dev)
    L = lib()
    ws = _workspace(L.bakron_factor_blockdiag_workspace_bytes(code, heads, heads * b, n), dev, workspace)
    bad = (_i64 * 3)(-1, -1, -1)
    with torch.cuda.device(dev):
        rc = L.bakron_factor_blockdiag(code, heads, heads * b, n, _p(A), _ld(A, "A"), pb, ldb, sb,
                                       _p(LA), max(n, 1), _p(LB), max(b, 1), b * b, _p(dA), _p(dB),
                                       _p(ws), ws.numel() * ws.element_size(), bad, _stream(dev))
    if rc != OK:
        err = BakronError(rc, "bakron_factor_blockdiag")
        err.bad_pivot = (int(bad[0]), int(bad[1]), int(bad[2]))
        raise err
    return LA, LB, dA, dB


def solve_blockdiag(W: torch.Tensor, LA: torch.Tensor, LBblocks: torch.Tensor,
                    alphabet: AlphabetLike = (0, 0, 1), scales: Optional[torch.Tensor] = None,
                    scale_mode: Optional[int] = None, return_wt: bool = False,
                    workspace: Optional[torch.Tensor] = None, check: bool = False):
    """The BaKron solve with a block-diagonal L^B given by its blocks
    (heads, b, b), m = heads * b: all heads in the same launches. ``check``:
    as in ``solve``."""
    dev = _check_device(W, LA, LBblocks, scales, workspace)
    code = _dt(W)
    m, n = W.shape
    if LBblocks.dim() != 3 or LBblocks.size(0) * LBblocks.size(1) != m:
        raise ValueError("LBblocks must be (heads, b, b) with heads * b = m")
    heads, b = LBblocks.size(0), LBblocks.size(1)
    if LA.shape != (n, n) or LA.dtype != W.dtype or LBblocks.dtype != W.dtype:
        raise ValueError("LA must be n x n, all of W's dtype")
    plb, ldlb, slb = _blocks(LBblocks, heads, b, "LBblocks")
    lo, hi, unb = (int(alphabet[0]), int(alphabet[1]), int(bool(alphabet[2])))
    mode = _scale_mode(scales, m, n, scale_mode)
    if scales is not None and (scales.dtype != W.dtype or not scales.is_contiguous()):
        raise ValueError("scales must be contiguous with W's dtype")
    V = torch.empty((m, n), dtype=torch.int32, device=dev)
    Wt = torch.empty((m, n), dtype=W.dtype, device=dev) if return_wt else None
    L = lib()
    ws = _workspace(L.bakron_solve_blockdiag_workspace_bytes(code, heads, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_solve_blockdiag(code, heads, m, n, _p(W), _ld(W, "W"), _p(LA), _ld(LA, "LA"),
                                      plb, ldlb, slb, lo, hi, unb, mode, _p(scales), _p(V),
                                      _ld(V, "V"), _p(Wt), _ld(Wt, "Wt") if Wt is not None else 0,
                                      _p(ws), ws.numel() * ws.element_size(), _stream(dev))
    if rc == OK and check:
        rc = L.bakron_solve_status(code, heads, b, n, _p(ws), ws.numel() * ws.element_size(),
                                   _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_solve_blockdiag")
    return (V, Wt) if return_wt else V


def loss_blockdiag(W: torch.Tensor, V: torch.Tensor, A: torch.Tensor, Bblocks: torch.Tensor,
                   scales: Optional[torch.Tensor] = None, scale_mode: Optional[int] = None,
                   workspace: Optional[torch.Tensor] = None, sync: bool = True):
    """tr(B (W - s V) A (W - s V)^T) for B = blockdiag(Bblocks[h]), in float64."""
    dev = _check_device(W, V, A, Bblocks, scales, workspace)
    code = _dt(W)
    m, n = W.shape
    if Bblocks.dim() != 3 or Bblocks.size(0) * Bblocks.size(1) != m:
        raise ValueError("Bblocks must be (heads, b, b) with heads * b = m")
    heads, b = Bblocks.size(0), Bblocks.size(1)
    _check_operand(V, (m, n), torch.int32, "V")
    _check_operand(A, (n, n), W.dtype, "A")
    if Bblocks.dtype != W.dtype:
        raise TypeError("Bblocks must have W's dtype")
    pb, ldb, sb = _blocks(Bblocks, heads, b, "Bblocks")
    mode = _scale_mode(scales, m, n, scale_mode)
    if scales is not None and (scales.dtype != W.dtype or not scales.is_contiguous()):
        raise ValueError("scales must be contiguous with W's dtype")
    out = torch.zeros(1, dtype=torch.float64, device=dev)
    L = lib()
    ws = _workspace(L.bakron_loss_blockdiag_workspace_bytes(code, heads, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_loss_blockdiag(code, heads, m, n, _p(W), _ld(W, "W"), _p(V), _ld(V, "V"), mode,
                                     _p(scales), _p(A), _ld(A, "A"), pb, ldb, sb, _p(out), _p(ws),
                                     ws.numel() * ws.element_size(), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_loss_blockdiag")
    return float(out.item()) if sync else out


# Largest workspace bakron_solve_noalloc takes from its in-library scratch
# (BAKRON_NOALLOC_SCRATCH_BYTES in include/bakron.h).
NOALLOC_SCRATCH_BYTES = 96 << 20


def solve_noalloc(W: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor, alphabet: AlphabetLike,
                  scales: Optional[torch.Tensor], V: torch.Tensor, Wt: Optional[torch.Tensor] = None,
                  scale_mode: Optional[int] = None, check: bool = False) -> torch.Tensor:
    """bakron_solve_noalloc: the solve of ``solve`` with the library's own
    per-GPU scratch instead of a workspace. The caller passes the outputs
    (V int32 m x n, optional Wt of W's dtype); nothing is allocated. Calls
    that overlap on one GPU race on the scratch. ``check``: as in ``solve``."""
    dev = _check_device(W, LA, LB, scales, V, Wt)
    code = _dt(W)
    m, n = W.shape
    if LA.shape != (n, n) or LB.shape != (m, m) or LA.dtype != W.dtype or LB.dtype != W.dtype:
        raise ValueError("LA must be n x n and LB m x m, same dtype as W")
    lo, hi, unb = (int(alphabet[0]), int(alphabet[1]), int(bool(alphabet[2])))
    mode = _scale_mode(scales, m, n, scale_mode)
    if scales is not None and (scales.dtype != W.dtype or not scales.is_contiguous()):
        raise ValueError("scales must be contiguous with W's dtype")
    _check_out(V, (m, n), torch.int32, "V")
    if Wt is not None:
        _check_out(Wt, (m, n), W.dtype, "Wt")
    with torch.cuda.device(dev):
        rc = lib().bakron_solve_noalloc(code, m, n, _p(W), _ld(W, "W"), _p(LA), _ld(LA, "LA"),
                                        _p(LB), _ld(LB, "LB"), lo, hi, unb, mode, _p(scales),
                                        _p(V), _ld(V, "V"), _p(Wt),
                                        _ld(Wt, "Wt") if Wt is not None else 0, _stream(dev))
    if rc == OK and check:
        with torch.cuda.device(dev):
            rc = lib().bakron_solve_status(code, 1, m, n, None, 0, _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_solve_noalloc")
    return V


def _batch_operand(t: torch.Tensor, rows: int, cols: int, batch: int, name: str):
    """(pointer, ld, stride) of a batched operand: a (batch, rows, cols)
    tensor, or a single (rows, cols) matrix shared by every problem."""
    if t.dim() == 2:
        if t.shape != (rows, cols):
            raise ValueError(f"{name} must be {rows} x {cols}")
        return _p(t), _ld(t, name), 0
    if t.dim() != 3 or t.shape != (batch, rows, cols):
        raise ValueError(f"{name} must be ({batch}, {rows}, {cols}) or ({rows}, {cols})")
    if cols > 1 and t.stride(2) != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    ld = max(int(t.stride(1)), cols, 1)
    return _p(t), ld, int(t.stride(0)) if batch > 1 else 0


def solve_batched(W: torch.Tensor, LA: torch.Tensor, LB: torch.Tensor,
                  alphabet: AlphabetLike = (0, 0, 1), scales: Optional[torch.Tensor] = None,
                  scale_mode: Optional[int] = None, return_wt: bool = False,
                  workspace: Optional[torch.Tensor] = None, check: bool = False):
    """bakron_solve on a batch of problems of one shape in the same launches.
    W is (batch, m, n); LA is (batch, n, n) or one (n, n) factor shared by
    all problems, LB likewise (batch, m, m) or (m, m); scales (batch, m) /
    (batch, n) or one shared vector. Returns int32 codes (batch, m, n) and,
    with ``return_wt``, the values at rounding. Each problem's result equals
    ``solve`` on the same inputs bit for bit. ``check``: as in ``solve``."""
    dev = _check_device(W, LA, LB, scales, workspace)
    code = _dt(W)
    if W.dim() != 3:
        raise ValueError("W must be (batch, m, n)")
    batch, m, n = W.shape
    if LA.dtype != W.dtype or LB.dtype != W.dtype:
        raise ValueError("LA and LB must have W's dtype")
    pw, ldw, sw = _batch_operand(W, m, n, batch, "W")
    pla, ldla, sla = _batch_operand(LA, n, n, batch, "LA")
    plb, ldlb, slb = _batch_operand(LB, m, m, batch, "LB")
    lo, hi, unb = (int(alphabet[0]), int(alphabet[1]), int(bool(alphabet[2])))
    ss = 0
    if scales is None:
        if scale_mode not in (None, SCALE_NONE):
            raise ValueError("scales required for this scale_mode")
        mode = SCALE_NONE
    else:
        if scales.dtype != W.dtype or not scales.is_contiguous():
            raise ValueError("scales must be contiguous with W's dtype")
        vec = scales if scales.dim() == 1 else scales[0]
        if scales.dim() not in (1, 2) or (scales.dim() == 2 and scales.size(0) != batch):
            raise ValueError("scales must be (batch, length) or (length,)")
        mode = _scale_mode(vec, m, n, scale_mode)
        ss = int(scales.stride(0)) if scales.dim() == 2 and batch > 1 else 0
    V = torch.empty((batch, m, n), dtype=torch.int32, device=dev)
    Wt = torch.empty((batch, m, n), dtype=W.dtype, device=dev) if return_wt else None
    L = lib()
    ws = _workspace(L.bakron_solve_batched_workspace_bytes(code, batch, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_solve_batched(code, batch, m, n, pw, ldw, sw, pla, ldla, sla, plb, ldlb, slb,
                                    lo, hi, unb, mode, _p(scales), ss, _p(V), max(n, 1), m * n,
                                    _p(Wt), max(n, 1) if return_wt else 0,
                                    m * n if return_wt else 0, _p(ws),
                                    ws.numel() * ws.element_size(), _stream(dev))
    if rc == OK and check:
        rc = L.bakron_solve_status(code, batch, m, n, _p(ws), ws.numel() * ws.element_size(),
                                   _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_solve_batched")
    return (V, Wt) if return_wt else V


def loss(W: torch.Tensor, V: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
         scales: Optional[torch.Tensor] = None, scale_mode: Optional[int] = None,
         workspace: Optional[torch.Tensor] = None, sync: bool = True):
    """tr(B (W - s V) A (W - s V)^T) in float64 (Proposition 3.1). Returns a
    Python float (``sync``) or a 1-element float64 device tensor."""
    dev = _check_device(W, V, A, B, scales, workspace)
    code = _dt(W)
    m, n = W.shape
    mode = _scale_mode(scales, m, n, scale_mode)
    _check_operand(V, (m, n), torch.int32, "V")
    _check_operand(A, (n, n), W.dtype, "A")
    _check_operand(B, (m, m), W.dtype, "B")
    if scales is not None and (scales.dtype != W.dtype or not scales.is_contiguous()):
        raise ValueError("scales must be contiguous with W's dtype")
    out = torch.zeros(1, dtype=torch.float64, device=dev)
    L = lib()
    ws = _workspace(L.bakron_loss_workspace_bytes(code, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_loss(code, m, n, _p(W), _ld(W, "W"), _p(V), _ld(V, "V"), mode, _p(scales),
                           _p(A), _ld(A, "A"), _p(B), _ld(B, "B"), _p(out), _p(ws),
                           ws.numel() * ws.element_size(), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_loss")
    return float(out.item()) if sync else out


def loss_batched(W: torch.Tensor, V: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                 scales: Optional[torch.Tensor] = None, scale_mode: Optional[int] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bakron_loss for a batch in the same launches: W, V (batch, m, n); A
    (batch, n, n) or one (n, n); B (batch, m, m) or one (m, m); scales
    (batch, length) or one vector. Returns a float64 device tensor of
    ``batch`` losses (asynchronous)."""
    dev = _check_device(W, V, A, B, scales, workspace)
    code = _dt(W)
    if W.dim() != 3 or V.dim() != 3 or V.shape != W.shape or V.dtype != torch.int32:
        raise ValueError("W and V must be (batch, m, n), V int32")
    batch, m, n = W.shape
    if A.dtype != W.dtype or B.dtype != W.dtype:
        raise TypeError("A and B must have W's dtype")
    pw, ldw, sw = _batch_operand(W, m, n, batch, "W")
    pv, ldv, sv = _batch_operand(V, m, n, batch, "V")
    pa, lda, sa = _batch_operand(A, n, n, batch, "A")
    pb, ldb, sb = _batch_operand(B, m, m, batch, "B")
    ss = 0
    if scales is None:
        if scale_mode not in (None, SCALE_NONE):
            raise ValueError("scales required for this scale_mode")
        mode = SCALE_NONE
    else:
        if scales.dtype != W.dtype or not scales.is_contiguous():
            raise ValueError("scales must be contiguous with W's dtype")
        if scales.dim() not in (1, 2) or (scales.dim() == 2 and scales.size(0) != batch):
            raise ValueError("scales must be (batch, length) or (length,)")
        vec = scales if scales.dim() == 1 else scales[0]
        mode = _scale_mode(vec, m, n, scale_mode)
        ss = int(scales.stride(0)) if scales.dim() == 2 and batch > 1 else 0
    out = torch.zeros(batch, dtype=torch.float64, device=dev)
    L = lib()
    ws = _workspace(L.bakron_loss_batched_workspace_bytes(code, batch, m, n), dev, workspace)
    with torch.cuda.device(dev):
        rc = L.bakron_loss_batched(code, batch, m, n, pw, ldw, sw, pv, ldv, sv, mode, _p(scales), ss,
                                   pa, lda, sa, pb, ldb, sb, _p(out), _p(ws),
                                   ws.numel() * ws.element_size(), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_loss_batched")
    return out


def row_scales(W: torch.Tensor, hi: int) -> torch.Tensor:
    """s_i = max_j |W_ij| / hi (1 for an all-zero row), in W's dtype."""
    dev = _check_device(W)
    code = _dt(W)
    m, n = W.shape
    s = torch.empty(m, dtype=W.dtype, device=dev)
    with torch.cuda.device(dev):
        rc = lib().bakron_row_scales(code, m, n, _p(W), _ld(W, "W"), int(hi), _p(s), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_row_scales")
    return s


def row_scales_mse(W: torch.Tensor, alphabet: AlphabetLike, grid: int = 100,
                   max_shrink: float = 0.5) -> torch.Tensor:
    """Per-row absmax / hi scales shrunk by up to 1 / (1 - max_shrink) by a
    search over grid + 1 candidates for the smallest round-to-nearest squared
    error of the row (bakron_row_scales_mse), in W's dtype."""
    dev = _check_device(W)
    code = _dt(W)
    m, n = W.shape
    lo, hi = int(alphabet[0]), int(alphabet[1])
    s = torch.empty(m, dtype=W.dtype, device=dev)
    with torch.cuda.device(dev):
        rc = lib().bakron_row_scales_mse(code, m, n, _p(W), _ld(W, "W"), lo, hi, int(grid),
                                         float(max_shrink), _p(s), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_row_scales_mse")
    return s


def gram(X: torch.Tensor, weights: Optional[torch.Tensor] = None, damp_rel: float = 0.0,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(1/N) sum_k w_k x_k x_k^T over the rows of X (N x d), plus
    damp_rel * mean(diag) * I (bakron_gram): the K-FAC factor with no
    weights, the one-step Shampoo factor with the other side's squared norms."""
    dev = _check_device(X, weights, out)
    code = _dt(X)
    N, d = X.shape
    if weights is not None and (weights.dtype != X.dtype or weights.numel() != N
                                or not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous length-N vector of X's dtype")
    if out is not None:
        _check_out(out, (d, d), X.dtype, "out")
    G = out if out is not None else torch.empty((d, d), dtype=X.dtype, device=dev)
    with torch.cuda.device(dev):
        rc = lib().bakron_gram(code, N, d, _p(X), _ld(X, "X"), _p(weights), float(damp_rel),
                               _p(G), _ld(G, "G"), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_gram")
    return G


def sample_sqnorms(X: torch.Tensor) -> torch.Tensor:
    """|x_k|^2 of every row of X (bakron_sample_sqnorms)."""
    dev = _check_device(X)
    code = _dt(X)
    N, d = X.shape
    out = torch.empty(N, dtype=X.dtype, device=dev)
    with torch.cuda.device(dev):
        rc = lib().bakron_sample_sqnorms(code, N, d, _p(X), _ld(X, "X"), _p(out), _stream(dev))
    if rc != OK:
        raise BakronError(rc, "bakron_sample_sqnorms")
    return out


def kfac_factors(Xa: torch.Tensor, Xb: torch.Tensor, damp_rel: float = 0.0):
    """K-FAC-style Kronecker factors A = E[a a^T], B = E[b b^T] (§4.2) from
    the sample rows of Xa (N x n) and Xb (N x m)."""
    return gram(Xa, None, damp_rel), gram(Xb, None, damp_rel)


def shampoo_factors(Xa: torch.Tensor, Xb: torch.Tensor, damp_rel: float = 0.0):
    """One-step Shampoo-style factors A = E[|b|^2 a a^T], B = E[|a|^2 b b^T]
    (§4.2, Appendix A.2)."""
    return gram(Xa, sample_sqnorms(Xb), damp_rel), gram(Xb, sample_sqnorms(Xa), damp_rel)


_FLOATS = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


def _ft(dtype: torch.dtype, name: str) -> int:
    """The element type code of the calls beside the solve."""
    code = _FLOATS.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _matrix(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None):
    """(rows, columns, leading dimension) of a 2-D row-major operand whose rows
    may be any distance apart (at least their length)."""
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    if rows <= 1:
        return rows, cols, max(cols, 1)
    if ld < cols:
        raise ValueError(f"{name} rows overlap (leading dimension below the row length)")
    return rows, cols, max(ld, 1)


def _vector(t: Optional[torch.Tensor], n: int, name: str,
            dtype: torch.dtype = torch.float32) -> Optional[int]:
    """The address of a contiguous vector of length n (None for None)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of length {n}")
    return t.data_ptr()


def _output(t: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype, name: str, dev):
    """A caller's output, checked, or a new one, and its leading dimension."""
    if t is None:
        return torch.empty((rows, cols), dtype=dtype, device=dev), max(cols, 1)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    return t, _matrix(t, name)[2]


def _scratch(nbytes: int, dev, ws: Optional[torch.Tensor]):
    """(tensor, address, size) of a workspace of at least nbytes; nothing for 0."""
    if not nbytes:
        return None, None, 0
    t = _workspace(nbytes, dev, ws)
    return t, t.data_ptr(), t.numel() * t.element_size()


def _call(what: str, dev, f, *args) -> None:
    """f(*args, the current stream) on `dev`, which is made the current device if
    it is not."""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if torch.cuda.current_device() == dev.index:
        rc = f(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = f(*args, stream)
    if rc != OK:
        raise BakronError(rc, what)


def quantize_tokens(X: torch.Tensor, channel_scales: Optional[torch.Tensor] = None):
    """Per-token int8 activations (bakron_quantize_tokens): with x = X[t] *
    channel_scales (a float32 vector; the column scales of a layer solved with
    SCALE_COL), sx[t] = max|x| / 127 (1 for an all-zero token) and
    Xq[t] = clamp(rint(x / sx[t]), -127, 127). X is T x n in float32, bfloat16
    or float16. Returns Xq (int8, T x n, rows starting at multiples of 16
    bytes) and sx (float32, T). Asynchronous."""
    dev = _check_device(X, channel_scales)
    code = _ft(X.dtype, "X")
    T, n, ldx = _matrix(X, "X")
    c = _vector(channel_scales, n, "channel_scales")
    ldq = (n + 15) // 16 * 16
    Xq = torch.empty((T, ldq), dtype=torch.int8, device=dev)
    if ldq != n:
        Xq = Xq[:, :n]
    sx = torch.empty(T, dtype=torch.float32, device=dev)
    _call("bakron_quantize_tokens", dev, lib().bakron_quantize_tokens, code, T, n, X.data_ptr(), ldx, c,
          Xq.data_ptr(), ldq, sx.data_ptr())
    return Xq, sx


def matmul_int8(Xq: torch.Tensor, sx: torch.Tensor, Vq: torch.Tensor,
                sv: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y[t][i] = sx[t] sv[i] sum_j Xq[t][j] Vq[i][j] (bakron_matmul_int8): the
    tokens of ``quantize_tokens`` through a layer held as the solve's codes.
    Xq is T x n and Vq m x n, int8 (``V.to(torch.int8)`` of codes inside
    [-128, 127], made once); sx has length T; sv, the row scales, length m, or
    None for 1 (column scales go to ``quantize_tokens``). The sums are exact
    (n <= 131071). Y is T x m in ``out_dtype`` (float32, bfloat16 or float16),
    or ``out`` and its type. Asynchronous."""
    dev = _check_device(Xq, sx, Vq, sv, out, workspace)
    T, n, ldx = _matrix(Xq, "Xq", torch.int8)
    m, nv, ldv = _matrix(Vq, "Vq", torch.int8)
    if nv != n:
        raise ValueError(f"Xq and Vq must have rows of one length, got {n} and {nv}")
    px, pv = _vector(sx, T, "sx"), _vector(sv, m, "sv")
    dtype = out_dtype if out is None else out.dtype
    code = _ft(dtype, "out_dtype")
    out, ldy = _output(out, T, m, dtype, "out", dev)
    L = lib()
    ws, pw, nw = _scratch(L.bakron_matmul_int8_workspace_bytes(T, m, n), dev, workspace)
    _call("bakron_matmul_int8", dev, L.bakron_matmul_int8, code, T, m, n, Xq.data_ptr(), ldx, px,
          Vq.data_ptr(), ldv, pv, out.data_ptr(), ldy, pw, nw)
    return out


def matmul_int8_grad(G: torch.Tensor, Vq: torch.Tensor, sv: Optional[torch.Tensor] = None,
                     channel_scales: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The input gradient of a layer held as codes (bakron_matmul_int8_grad):
    dX[t][j] = channel_scales[j] sum_i G[t][i] sv[i] Vq[i][j], with the rounding
    of the tokens passed straight through. G is T x m in float32, bfloat16 or
    float16 and dX, T x n, of its type; sv (length m) and channel_scales
    (length n) are float32, None for 1. Asynchronous."""
    dev = _check_device(G, Vq, sv, channel_scales, workspace, out)
    code = _ft(G.dtype, "G")
    T, m, ldg = _matrix(G, "G")
    mv, n, ldv = _matrix(Vq, "Vq", torch.int8)
    if mv != m:
        raise ValueError(f"G must have a column for each row of Vq, got {m} and {mv}")
    pv, pc = _vector(sv, m, "sv"), _vector(channel_scales, n, "channel_scales")
    out, ldx = _output(out, T, n, G.dtype, "out", dev)
    L = lib()
    ws, pw, nw = _scratch(L.bakron_matmul_int8_grad_workspace_bytes(code, T, m, n), dev, workspace)
    _call("bakron_matmul_int8_grad", dev, L.bakron_matmul_int8_grad, code, T, m, n, G.data_ptr(), ldg,
          Vq.data_ptr(), ldv, pv, pc, out.data_ptr(), ldx, pw, nw)
    return out


def _entropy_args(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor):
    """(type, T, d, V, X, ldx, W, ldw, targets) of the cross entropy's operands."""
    code = _ft(X.dtype, "X")
    T, d, ldx = _matrix(X, "X")
    V, dw, ldw = _matrix(W, "W", X.dtype)
    if dw != d:
        raise ValueError(f"X and W must have rows of one length, got {d} and {dw}")
    if V < 1:
        raise ValueError("W must have a row")
    y = _vector(targets, T, "targets", torch.int64)
    return code, T, d, V, X.data_ptr(), ldx, W.data_ptr(), ldw, y


def cross_entropy(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None):
    """Softmax cross entropy of hidden states X (T x d) under the output layer W
    (V x d), one loss per token, the logits X W^T never stored
    (bakron_cross_entropy). X and W are float32, bfloat16 or float16 (one type);
    targets is int64, and one outside [0, V) (-100 by custom) marks a token
    without a target, whose loss is 0. Returns loss and lse = log sum exp of the
    logits, float32 vectors of length T. Asynchronous."""
    dev = _check_device(X, W, targets, workspace)
    args = _entropy_args(X, W, targets)
    code, T, d, V = args[:4]
    loss, lse = torch.empty((2, T), dtype=torch.float32, device=dev).unbind(0)
    L = lib()
    ws, pw, nw = _scratch(L.bakron_cross_entropy_workspace_bytes(code, T, d, V), dev, workspace)
    _call("bakron_cross_entropy", dev, L.bakron_cross_entropy, *args, loss.data_ptr(), lse.data_ptr(), pw, nw)
    return loss, lse


def cross_entropy_grad(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                       g: torch.Tensor, need_dX: bool = True, need_dW: bool = True,
                       workspace: Optional[torch.Tensor] = None):
    """The gradient of sum_t g[t] loss[t] of ``cross_entropy`` with respect to X
    and W (bakron_cross_entropy_grad), of their type: (dX, dW), None where not
    needed. lse is the forward call's, g a float32 vector of length T (1 / (number of
    targets) for their mean). The rows of dX are the output-side samples of the
    layer below (``gram`` takes them in float32). Asynchronous."""
    dev = _check_device(X, W, targets, lse, g, workspace)
    args = _entropy_args(X, W, targets)
    code, T, d, V = args[:4]
    pl, pg = _vector(lse, T, "lse"), _vector(g, T, "g")
    dX = torch.empty((T, d), dtype=X.dtype, device=dev) if need_dX else None
    dW = torch.empty((V, d), dtype=X.dtype, device=dev) if need_dW else None
    L = lib()
    ws, pw, nw = _scratch(L.bakron_cross_entropy_grad_workspace_bytes(code, T, d, V), dev, workspace)
    _call("bakron_cross_entropy_grad", dev, L.bakron_cross_entropy_grad, *args, pl, pg,
          None if dX is None else dX.data_ptr(), max(d, 1), None if dW is None else dW.data_ptr(),
          max(d, 1), pw, nw)
    return dX, dW


E4M3 = torch.float8_e4m3fn
_BLOCK = 128


def quantize_fp8(X: torch.Tensor, block_rows: int = 1):
    """X as 8-bit floating point with a float32 scale for each block of block_rows x
    128 (bakron_quantize_fp8): 1 for tokens, 128 for weights. X is rows x n, or a
    batch of them (experts x rows x n), in float32, bfloat16 or float16. With a the
    largest |x| of a block its scale is s = a / 448 (at least 2^-126; 1 for zeros) and its
    codes x / s to the nearest. Returns the codes (torch.float8_e4m3fn, of X's shape,
    rows starting at multiples of 16 bytes) and the scales (... x ceil(rows /
    block_rows) x ceil(n / 128); for block_rows = 1 a block's scales of all rows lie side by
    side). Asynchronous."""
    dev = _check_device(X)
    code = _ft(X.dtype, "X")
    if block_rows not in (1, _BLOCK):
        raise ValueError(f"block_rows must be 1 or {_BLOCK}, got {block_rows}")
    batch, rows, n, ldx, sX = _matrices(X, "X")
    ldq, nb, na = (n + 15) // 16 * 16, (n + 127) // 128, (rows + block_rows - 1) // block_rows
    lead, steps = ((), ()) if len(X.shape) == 2 else ((batch,), (na * nb,))
    Xq = torch.empty((*lead, rows, ldq), dtype=E4M3, device=dev)
    if ldq != n:
        Xq = Xq[..., :n]
    srow, sblock = (1, na) if block_rows == 1 else (nb, 1)
    s = torch.empty_strided((*lead, na, nb), (*steps, srow, sblock), dtype=torch.float32, device=dev)
    _call("bakron_quantize_fp8", dev, lib().bakron_quantize_fp8, code, batch, rows, n, X.data_ptr(), ldx, sX,
          block_rows, Xq.data_ptr(), ldq, rows * ldq, s.data_ptr(), srow, sblock, na * nb)
    return Xq, s


def _matrices(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None):
    """(batch, rows, columns, leading dimension, stride) of a row-major matrix, or of a
    batch of them (3-D) any distance apart."""
    shape = t.shape
    if len(shape) != 3:
        return 1, *_matrix(t, name, dtype), 0
    batch = shape[0]
    if batch == 0:
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        return 0, shape[1], shape[2], max(shape[2], 1), 0
    return batch, *_matrix(t[0], name, dtype), t.stride(0) if batch > 1 else 0


def _fp8_weights(Wq: torch.Tensor, sw: torch.Tensor, offsets: Optional[torch.Tensor]):
    """(m, n, blocks of n, (Wq, ldw, stride, sw, ldsw, stride), experts, offsets): a layer's
    codes and scales, or those of each expert with the offsets of their rows."""
    if (len(Wq.shape) == 3) != (offsets is not None):
        raise ValueError("Wq is experts x m x n with offsets, and m x n without")
    if offsets is None:
        m, n, ldw = _matrix(Wq, "Wq", E4M3)
        mb, nbs, ldsw = _matrix(sw, "sw", torch.float32)
        nb = (n + 127) // 128
        if mb != (m + 127) // 128 or nbs != nb:
            raise ValueError(f"sw must have shape {((m + 127) // 128, nb)}, got {tuple(sw.shape)}")
        return m, n, nb, (Wq.data_ptr(), ldw, 0, sw.data_ptr(), ldsw, 0), 1, None
    experts, m, n, ldw, stride = _matrices(Wq, "Wq", E4M3)
    if experts < 1:
        raise ValueError("Wq must have an expert")
    nb = (n + 127) // 128
    es, mb, nbs, ldsw, stride_s = _matrices(sw, "sw", torch.float32)
    if es != experts or nbs != nb or mb != (m + 127) // 128 or len(sw.shape) != len(Wq.shape):
        raise ValueError(f"sw must have shape {(*Wq.shape[:-2], (m + 127) // 128, nb)}, got {tuple(sw.shape)}")
    return (m, n, nb, (Wq.data_ptr(), ldw, stride, sw.data_ptr(), ldsw, stride_s), experts,
            _vector(offsets, experts + 1, "offsets", torch.int32))


def _fp8_rows(m: int, p: int, ldw: int, stride: int, *scales) -> int:
    """A multiple of 16 where every row of a layer's codes starts at one."""
    return p | (m > 1 and ldw) | stride


def matmul_fp8(Xq: torch.Tensor, sx: torch.Tensor, Wq: torch.Tensor, sw: torch.Tensor,
               offsets: Optional[torch.Tensor] = None, order: Optional[torch.Tensor] = None, per_token: int = 1,
               out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Tokens times weights, both as ``quantize_fp8`` gives them (bakron_matmul_fp8):
    Y[r][i] = sum_b sx[t][b] sw[i // 128][b] sum_{j in block b} Xq[t][j] Wq[i][j].

    Xq is T x n and sx T x ceil(n / 128), with any strides; Wq m x n with sw
    ceil(m / 128) x ceil(n / 128). For a layer of experts Wq is experts x m x n, sw likewise,
    and ``offsets`` (int32, experts + 1) says which rows of Y are whose: rows
    [offsets[e], offsets[e + 1]) are multiplied by expert e, rows past the last are not
    written. Row r is token r, or with ``order`` (int32; ``sort_tokens`` makes it and the
    offsets) token order[r] // per_token, so that the tokens need not be copied into
    order; Y then has a row for each of ``order``. Y is rows x m in ``out_dtype`` (float32,
    bfloat16 or float16), or ``out`` and its type. Asynchronous."""
    dev = _check_device(Xq, sx, Wq, sw, offsets, order, out, workspace)
    T, n, ldx = _matrix(Xq, "Xq", E4M3)
    m, nw, nb, weights, experts, po = _fp8_weights(Wq, sw, offsets)
    if nw != n:
        raise ValueError(f"Xq and Wq must have rows of one length, got {n} and {nw}")
    if sx.dtype != torch.float32:
        raise TypeError(f"sx must be torch.float32, got {sx.dtype}")
    if sx.shape != (T, nb):
        raise ValueError(f"sx must have shape {(T, nb)}, got {tuple(sx.shape)}")
    if per_token < 1:
        raise ValueError("per_token must be positive")
    R, pr = T, None
    if order is not None:
        if order.dim() != 1:
            raise ValueError("order must be a vector")
        R = order.size(0)
        pr = _vector(order, R, "order", torch.int32)
    dtype = out_dtype if out is None else out.dtype
    code = _ft(dtype, "out_dtype")
    out, ldy = _output(out, R, m, dtype, "out", dev)
    L, px = lib(), Xq.data_ptr()
    query = L.bakron_matmul_fp8_workspace_bytes
    if n % 16 and (px | (T > 1 and ldx) | _fp8_rows(m, *weights)) % 16 == 0:  # else they agree, or copies are made
        query = L.bakron_matmul_fp8_aligned_workspace_bytes
    ws, pws, nws = _scratch(query(code, T, R, experts, m, n), dev, workspace)
    _call("bakron_matmul_fp8", dev, L.bakron_matmul_fp8, code, T, R, experts, m, n, px, ldx,
          sx.data_ptr(), *sx.stride(), *weights, po, pr, per_token, out.data_ptr(), ldy, pws, nws)
    return out


def matmul_fp8_grad(G: torch.Tensor, Wq: torch.Tensor, sw: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The input gradient of ``matmul_fp8`` (bakron_matmul_fp8_grad): dX[r][j] =
    sum_i G[r][i] sw[i // 128][j // 128] Wq[i][j], with the rounding of the tokens
    passed straight through. G is rows x m in float32, bfloat16 or float16 and dX, rows x n, of
    its type. With experts the rows are in their order, as Y's were (``combine_tokens`` adds
    up those of one token), and rows past the last expert's are not written.
    Asynchronous."""
    dev = _check_device(G, Wq, sw, offsets, workspace, out)
    code = _ft(G.dtype, "G")
    R, m, ldg = _matrix(G, "G")
    mw, n, _, weights, experts, po = _fp8_weights(Wq, sw, offsets)
    if mw != m:
        raise ValueError(f"G must have a column for each row of Wq, got {m} and {mw}")
    out, ldx = _output(out, R, n, G.dtype, "out", dev)
    L = lib()
    query = L.bakron_matmul_fp8_grad_workspace_bytes
    if n % 16 and _fp8_rows(m, *weights) % 16 == 0:
        query = L.bakron_matmul_fp8_grad_aligned_workspace_bytes
    ws, pws, nws = _scratch(query(code, R, experts, m, n), dev, workspace)
    _call("bakron_matmul_fp8_grad", dev, L.bakron_matmul_fp8_grad, code, R, experts, m, n, G.data_ptr(), ldg, *weights,
          po, out.data_ptr(), ldx, pws, nws)
    return out


def sort_tokens(experts: torch.Tensor, num_experts: int, workspace: Optional[torch.Tensor] = None):
    """Routes in the order of their experts (bakron_sort_tokens). ``experts`` (int64,
    T x k) holds the k experts of each token; one outside [0, num_experts) (-1 by custom)
    drops that route. Returns int32 ``order`` (T k: the routes t k + j by expert, those of
    one expert in their own order, -1 past the last), ``slots`` (T x k: each route's place
    in it, -1 if dropped) and ``offsets`` (num_experts + 1: where each expert's begin).
    Asynchronous."""
    dev = _check_device(experts, workspace)
    T, k, ld = _matrix(experts, "experts", torch.int64)
    E = int(num_experts)
    if k < 1 or E < 1:
        raise ValueError("a token must have an expert")
    order = torch.empty(T * k, dtype=torch.int32, device=dev)
    slots = torch.empty((T, k), dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    L = lib()
    ws, pws, nws = _scratch(L.bakron_sort_tokens_workspace_bytes(T, k, E), dev, workspace)
    _call("bakron_sort_tokens", dev, L.bakron_sort_tokens, T, k, E, experts.data_ptr(), ld, order.data_ptr(),
          slots.data_ptr(), offsets.data_ptr(), pws, nws)
    return order, slots, offsets


def gather_tokens(X: torch.Tensor, order: torch.Tensor, per_token: int = 1,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Xs[s] = X[order[s] // per_token] (bakron_gather_tokens), zeros where order[s]
    names no token (-1): the tokens of ``sort_tokens``'s experts side by side, for instance
    the samples of each for ``gram``. X is float32, bfloat16 or float16. Its gradient is
    ``combine_tokens(dXs, slots)``. Asynchronous."""
    dev = _check_device(X, order, out)
    code = _ft(X.dtype, "X")
    T, n, ldx = _matrix(X, "X")
    if order.dim() != 1:
        raise ValueError("order must be a vector")
    R = order.size(0)
    if per_token < 1:
        raise ValueError("per_token must be positive")
    po = _vector(order, R, "order", torch.int32)
    out, ldo = _output(out, R, n, X.dtype, "out", dev)
    _call("bakron_gather_tokens", dev, lib().bakron_gather_tokens, code, T, n, X.data_ptr(), ldx, per_token, R, po,
          out.data_ptr(), ldo)
    return out


def _routes(slots: torch.Tensor, weights: Optional[torch.Tensor]):
    """(T, k, slots, weights) of contiguous T x k tensors."""
    if slots.dtype != torch.int32:
        raise TypeError(f"slots must be torch.int32, got {slots.dtype}")
    if slots.dim() != 2 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous T x k tensor")
    if weights is not None:
        if weights.dtype != torch.float32:
            raise TypeError(f"weights must be torch.float32, got {weights.dtype}")
        if weights.shape != slots.shape or not weights.is_contiguous():
            raise ValueError("weights must be contiguous, of slots' shape")
    return slots.size(0), slots.size(1), slots.data_ptr(), None if weights is None else weights.data_ptr()


def combine_tokens(Ys: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y[t] = sum_j weights[t][j] Ys[slots[t][j]] (bakron_combine_tokens): the experts'
    results back at their tokens. Ys has a row for each of ``sort_tokens``'s order, in
    float32, bfloat16 or float16, and Y (T x n) its type; slots is its second result (slots
    outside Ys' rows, -1 by custom, take no part), weights float32 T x k, None for 1. Sums
    are float32. Asynchronous."""
    dev = _check_device(Ys, slots, weights, out)
    code = _ft(Ys.dtype, "Ys")
    R, n, ldys = _matrix(Ys, "Ys")
    T, k, ps, pw = _routes(slots, weights)
    out, ldy = _output(out, T, n, Ys.dtype, "out", dev)
    _call("bakron_combine_tokens", dev, lib().bakron_combine_tokens, code, T, k, n, R, Ys.data_ptr(), ldys, ps, pw,
          out.data_ptr(), ldy)
    return out


def combine_tokens_grad(G: torch.Tensor, Ys: torch.Tensor, slots: torch.Tensor,
                        weights: Optional[torch.Tensor] = None, need_dYs: bool = True, need_dweights: bool = True):
    """The gradient of ``combine_tokens`` (bakron_combine_tokens_grad): (dYs, dweights)
    with dYs[slots[t][j]] = weights[t][j] G[t], of Ys' shape and type, and
    dweights[t][j] = G[t] . Ys[slots[t][j]], float32 T x k (0 for a dropped route); None
    where not needed. G is T x n of Ys' type. Rows of dYs that no slot names are not
    written; no slot may be named twice. Asynchronous."""
    dev = _check_device(G, Ys, slots, weights)
    code = _ft(Ys.dtype, "Ys")
    T, n, ldg = _matrix(G, "G", Ys.dtype)
    R, ny, ldys = _matrix(Ys, "Ys")
    if ny != n:
        raise ValueError(f"G and Ys must have rows of one length, got {n} and {ny}")
    Ts, k, ps, pw = _routes(slots, weights)
    if Ts != T:
        raise ValueError(f"G must have a row for each of slots, got {T} and {Ts}")
    dYs = torch.empty((R, n), dtype=Ys.dtype, device=dev) if need_dYs else None
    dw = torch.empty((T, k), dtype=torch.float32, device=dev) if need_dweights else None
    _call("bakron_combine_tokens_grad", dev, lib().bakron_combine_tokens_grad, code, T, k, n, R, G.data_ptr(), ldg,
          Ys.data_ptr(), ldys, ps, pw, None if dYs is None else dYs.data_ptr(), max(n, 1),
          None if dw is None else dw.data_ptr())
    return dYs, dw


def debug_set_wait_polls(polls: int) -> int:
    """Test hook: the poll bound of the leaf blocks' waits for solves enqueued
    from now on (negative: the default); returns the previous bound."""
    return int(lib().bakron_debug_set_wait_polls(int(polls)))


def debug_plan(M: int, N: int, steps: int, pairs: int = 1, kmajor: bool = False, may_split: bool = True,
               tile: int = 0, splits: int = 0) -> Tuple[int, int, float]:
    """Test hook: (tile, ranges of k, estimated us) of a tiled product, as a call
    divides it, or of the division given. Host only."""
    t, n = _i32(tile), _i32(splits)
    us = lib().bakron_debug_plan(M, N, steps, pairs, int(kmajor), int(may_split), ctypes.byref(t), ctypes.byref(n))
    return t.value, n.value, us


def solve_schedule(dtype: int, m: int, n: int):
    """The solve's launch schedule: list of (kind, a, b, c); kind 0 = leaf
    block of tile anti-diagonals [a, b), kinds 2/3 = the two band products of
    the internal node [a, b) -> [b, c). Host only."""
    L = lib()
    cnt = int(L.bakron_solve_schedule(int(dtype), int(m), int(n), None, 0))
    if cnt < 0:
        raise BakronError(cnt, "bakron_solve_schedule")
    buf = (ctypes.c_int32 * (4 * max(cnt, 1)))()
    L.bakron_solve_schedule(int(dtype), int(m), int(n), ctypes.cast(buf, ctypes.c_void_p), cnt)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(cnt)]
