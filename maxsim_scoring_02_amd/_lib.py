"""ctypes binding of liblik.so: argument marshalling only.

Every function here has the name of the C entry point it calls.  Tensors are
torch tensors on the GPU (PyTorch supplies device memory and the current
stream); outputs and the workspace are allocated with torch and handed to the
library as plain pointers.  All computation happens in the library's HIP
kernels.  There is no fallback: if liblik.so is missing or the call fails, an
exception is raised.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import re
from typing import Optional, Tuple

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "liblik.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG), "include", "lik.h")
ROWS_HEADER_PATH = os.path.join(os.path.dirname(PKG), "include", "lik_rows.h")
CACHE_HEADER_PATH = os.path.join(os.path.dirname(PKG), "include", "lik_cache.h")

LIK_OK, LIK_ERR_INVALID_ARG, LIK_ERR_UNSUPPORTED, LIK_ERR_HIP = 0, 1, 2, 3
LIK_F16, LIK_BF16, LIK_F32, LIK_F32_BF16X3 = 0, 1, 2, 3
(LIK_OP_FWD, LIK_OP_BWD, LIK_OP_PAIRWISE_FWD, LIK_OP_PAIRWISE_BWD,
 LIK_OP_KD_FWD, LIK_OP_KD_BWD) = range(6)

(LIK_ROWS_LOGPROB_FWD, LIK_ROWS_LOGPROB_BWD, LIK_ROWS_DISTILL, LIK_ROWS_POLICY,
 LIK_ROWS_PREFERENCE, LIK_ROWS_VERIFY) = range(6)
LIK_PREF_SIGMOID, LIK_PREF_HINGE, LIK_PREF_SQUARE = range(3)

DTYPE_CODE = {torch.float16: LIK_F16, torch.bfloat16: LIK_BF16, torch.float32: LIK_F32}

_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_I = ctypes.c_int
_F = ctypes.c_float

_FWD_ALLPAIRS = [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]
_BWD_ALLPAIRS = [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]
_FWD_PAIRWISE = [_P, _P, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]
_BWD_PAIRWISE = [_P, _P, _I, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]

SIGNATURES = {
    "lik_abi_version": ([], _I),
    "lik_status_string": ([_I], ctypes.c_char_p),
    "lik_last_error": ([], ctypes.c_char_p),
    "lik_supported_dim": ([_I64], _I),
    "lik_set_profile_events": ([_P, _P], _I),
    "lik_workspace_bytes": ([_I, _I64, _I64, _I64, _I64, _I64, _I, _I], _SZ),
    "lik_plan_value": ([_I, _I64, _I64, _I64, _I64, _I64, _I, _I, ctypes.c_char_p], _I64),
    "lik_maxsim_fwd": (_FWD_ALLPAIRS, _I),
    "lik_maxsim_fwd_noalloc": ([_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P, _P, _P], _I),
    "lik_maxsim_bwd": (_BWD_ALLPAIRS, _I),
    "lik_maxsim_pairwise_fwd": (_FWD_PAIRWISE, _I),
    "lik_maxsim_pairwise_bwd": (_BWD_PAIRWISE, _I),
    "lik_maxsim_kd_fwd": (_FWD_ALLPAIRS, _I),
    "lik_maxsim_kd_bwd": (_BWD_ALLPAIRS, _I),
    "lik_ce_rows": ([_P, _I64, _I64, _P, ctypes.c_float, _P, _P, _P, _P], _I),
}

# include/lik_rows.h
_ROWS = [_P, _I, _I64, _I64, _I64]                 # logits, dtype, R, C, ld
ROWS_SIGNATURES = {
    "lik_rows_workspace_bytes": ([_I, _I64, _I64, _I64, _I, _I], _SZ),
    "lik_logprob_rows_fwd": (_ROWS + [_P, _F, _P, _P, _P, _SZ, _P], _I),
    "lik_logprob_rows_bwd": (_ROWS + [_P, _F, _P, _P, _P, _I64, _P], _I),
    "lik_distill_rows": (_ROWS + [_P, _P, _I64, _P, _F, _P, _P, _P, _P, _I64, _P, _SZ, _P], _I),
    "lik_policy_rows": (_ROWS + [_P, _P, _P, _P, _F, _F, _F, _F, _P, _P, _P, _P, _P, _I64, _P,
                                 _SZ, _P], _I),
    "lik_preference_rows": (_ROWS + [_P, _P, _I64, _P, _P, _I64, _P, _I, _F, _F, _F, _I, _F, _P,
                                     _P, _P, _P, _P, _I64, _P, _SZ, _P], _I),
    "lik_verify_rows": (_ROWS + [_P, _I64, _P, _P, _I64, _F, _F, _P, _P, _P, _P, _P, _P, _SZ, _P],
                        _I),
}

# include/lik_cache.h
_CACHE = [_P] * 4 + [_I64] * 6           # codes, scales; blocks, heads, block size, dim, strides
CACHE_SIGNATURES = {
    "lik_cache_tables": ([_P, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P],
                         _I),
    "lik_cache_append": ([_P, _P, _I, _I64, _I64, _I64, _P] + _CACHE + [_P], _I),
    "lik_cache_workspace_bytes": ([_I64] * 5 + [_I], _SZ),
    "lik_cache_attention": ([_P, _I, _I64, _I64, _I64, _P, _P, _I64, _P, _I64, _I64] + _CACHE +
                            [_F, _P, _I64, _P, _P, _SZ, _P], _I),
}


class LikError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"liblik status {status}: {detail}")
        self.status = status


def header_functions(path: str = HEADER_PATH) -> list:
    """Names of the functions declared in include/lik.h (or another header)."""
    with open(path) as f:
        text = f.read()
    return sorted(set(re.findall(r"^[a-z0-9_ ]+?\**\s*\b(lik_[a-z_]+)\s*\(", text, re.M)))


def lib() -> ctypes.CDLL:
    """Load liblik.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m maxsim_scoring_02_amd.build`")
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in {**SIGNATURES, **ROWS_SIGNATURES, **CACHE_SIGNATURES}.items():
            fn = getattr(l, name)
            fn.argtypes = args
            fn.restype = res
        _lib = l
    return _lib


def _check(status: int):
    if status != LIK_OK:
        raise LikError(status, lib().lik_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _embeddings(Q: torch.Tensor, D: torch.Tensor, fp32_split: bool = False) -> int:
    """dtype code of the inputs; fp32_split asks for LIK_F32_BF16X3 (float32
    inputs scored through bfloat16 high/low parts, see include/lik.h)."""
    if not (Q.is_cuda and D.is_cuda):
        raise ValueError("Q and D must be GPU tensors")
    if Q.device != D.device:
        raise ValueError("Q and D must be on the same device")
    if Q.dtype != D.dtype or Q.dtype not in DTYPE_CODE:
        raise ValueError("Q and D must share a dtype among float16, bfloat16, float32")
    if Q.shape[-1] != D.shape[-1]:
        raise ValueError("Q and D must share the embedding dim")
    if not (Q.is_contiguous() and D.is_contiguous()):
        raise ValueError("Q and D must be contiguous")
    if fp32_split:
        if Q.dtype != torch.float32:
            raise ValueError("fp32_split applies to float32 inputs only")
        return LIK_F32_BF16X3
    return DTYPE_CODE[Q.dtype]


def _same_batch(Q: torch.Tensor, D: torch.Tensor, layout: str) -> None:
    """Pairwise and kd pair query b with document (row) b of D.  The C ABI
    receives B only, so a D with fewer rows would be read past its end on the
    device: the shapes are checked here, before anything is launched."""
    want = 3 if layout == "pairwise" else 4
    if Q.dim() != 3 or D.dim() != want:
        raise ValueError(f"{layout}: Q must be [B, Lq, dim] and D "
                         f"{'[B, Ld, dim]' if want == 3 else '[B, N, Ld, dim]'}")
    if D.shape[0] != Q.shape[0]:
        raise ValueError(f"{layout} Q and D must share the batch size "
                         f"(Q has {Q.shape[0]}, D has {D.shape[0]})")


def _flags(argmax_given: bool, dm, qm) -> int:
    """lik_workspace_bytes flags: bit 0 argmax, bit 1 document mask, bit 2 query mask."""
    return (1 if argmax_given else 0) | (2 if dm is not None else 0) | (4 if qm is not None else 0)


def _mask(m: Optional[torch.Tensor], shape, device) -> Optional[torch.Tensor]:
    if m is None:
        return None
    if tuple(m.shape) != tuple(shape):
        raise ValueError(f"mask shape {tuple(m.shape)} != {tuple(shape)}")
    if m.device != device or m.dtype != torch.bool or not m.is_contiguous():
        raise ValueError("masks must be contiguous bool tensors on the embeddings' device")
    return m.view(torch.uint8)


def _workspace(nbytes: int, device) -> Optional[torch.Tensor]:
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# forward
# ---------------------------------------------------------------------------

def lik_plan_value(op: int, dims, dtype: int, flags: int, key: str) -> int:
    """One value of the launch plan for a call (see include/lik.h); dims =
    (nq_or_b, lq, nd_or_n, ld, dim) as for lik_workspace_bytes."""
    return int(lib().lik_plan_value(op, *dims, dtype, flags, key.encode()))


def lik_maxsim_fwd(Q, D, q_mask=None, d_mask=None, keep_argmax=True, fp32_split=False):
    """All-pairs: Q [Nq, Lq, dim] x D [Nd, Ld, dim] -> scores [Nq, Nd] float32,
    argmax [Nq, Nd, Lq] int32 (or None)."""
    dt = _embeddings(Q, D, fp32_split)
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D.shape
    qm = _mask(q_mask, (Nq, Lq), Q.device)
    dm = _mask(d_mask, (Nd, Ld), Q.device)
    scores = torch.empty((Nq, Nd), dtype=torch.float32, device=Q.device)
    am = (torch.empty((Nq, Nd, Lq), dtype=torch.int32, device=Q.device)
          if keep_argmax else None)
    flags = _flags(keep_argmax, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_FWD, Nq, Lq, Nd, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_fwd(_ptr(Q), _ptr(D), dt, Nq, Lq, Nd, Ld, dim, _ptr(qm), _ptr(dm),
                                _ptr(scores), _ptr(am), _ptr(ws), wsb, _stream()))
    return scores, am


def lik_maxsim_fwd_noalloc(Q, D, q_mask=None, d_mask=None, keep_argmax=True, fp32_split=False):
    """All-pairs forward through the allocation-free entry point: the library
    takes its scratch from a fixed per-device array (the outputs are still
    the caller's, allocated here)."""
    dt = _embeddings(Q, D, fp32_split)
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D.shape
    qm = _mask(q_mask, (Nq, Lq), Q.device)
    dm = _mask(d_mask, (Nd, Ld), Q.device)
    scores = torch.empty((Nq, Nd), dtype=torch.float32, device=Q.device)
    am = (torch.empty((Nq, Nd, Lq), dtype=torch.int32, device=Q.device)
          if keep_argmax else None)
    _check(lib().lik_maxsim_fwd_noalloc(_ptr(Q), _ptr(D), dt, Nq, Lq, Nd, Ld, dim, _ptr(qm),
                                        _ptr(dm), _ptr(scores), _ptr(am), _stream()))
    return scores, am


def lik_maxsim_pairwise_fwd(Q, D, q_mask=None, d_mask=None, keep_argmax=True, fp32_split=False):
    """Pairwise: Q [B, Lq, dim] x D [B, Ld, dim] -> scores [B], argmax [B, Lq]."""
    _same_batch(Q, D, "pairwise")
    dt = _embeddings(Q, D, fp32_split)
    B, Lq, dim = Q.shape
    _, Ld, _ = D.shape
    qm = _mask(q_mask, (B, Lq), Q.device)
    dm = _mask(d_mask, (B, Ld), Q.device)
    scores = torch.empty((B,), dtype=torch.float32, device=Q.device)
    am = torch.empty((B, Lq), dtype=torch.int32, device=Q.device) if keep_argmax else None
    flags = _flags(keep_argmax, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_PAIRWISE_FWD, B, Lq, 1, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_pairwise_fwd(_ptr(Q), _ptr(D), dt, B, Lq, Ld, dim, _ptr(qm),
                                         _ptr(dm), _ptr(scores), _ptr(am), _ptr(ws), wsb,
                                         _stream()))
    return scores, am


def lik_maxsim_kd_fwd(Q, D, q_mask=None, d_mask=None, keep_argmax=True, fp32_split=False):
    """kd: Q [B, Lq, dim] x D [B, N, Ld, dim] -> scores [B, N], argmax [B, N, Lq]."""
    _same_batch(Q, D, "kd")
    dt = _embeddings(Q, D, fp32_split)
    B, Lq, dim = Q.shape
    _, N, Ld, _ = D.shape
    qm = _mask(q_mask, (B, Lq), Q.device)
    dm = _mask(d_mask, (B, N, Ld), Q.device)
    scores = torch.empty((B, N), dtype=torch.float32, device=Q.device)
    am = torch.empty((B, N, Lq), dtype=torch.int32, device=Q.device) if keep_argmax else None
    flags = _flags(keep_argmax, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_KD_FWD, B, Lq, N, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_kd_fwd(_ptr(Q), _ptr(D), dt, B, Lq, N, Ld, dim, _ptr(qm), _ptr(dm),
                                   _ptr(scores), _ptr(am), _ptr(ws), wsb, _stream()))
    return scores, am


# ---------------------------------------------------------------------------
# backward
# ---------------------------------------------------------------------------

def _grad_scores(g: torch.Tensor, shape, device) -> torch.Tensor:
    if tuple(g.shape) != tuple(shape) or g.dtype != torch.float32 or g.device != device:
        raise ValueError(f"grad_scores must be float32 {tuple(shape)} on the embeddings' device")
    return g.contiguous()


def _argmax_in(am: Optional[torch.Tensor], shape, device) -> Optional[torch.Tensor]:
    if am is None:
        return None
    if tuple(am.shape) != tuple(shape) or am.dtype != torch.int32 or am.device != device:
        raise ValueError(f"argmax must be int32 {tuple(shape)} from the forward")
    return am.contiguous()


def lik_maxsim_bwd(Q, D, grad_scores, argmax=None, q_mask=None, d_mask=None,
                   need_grad_q=True, need_grad_d=True, fp32_split=False) -> Tuple:
    dt = _embeddings(Q, D, fp32_split)
    Nq, Lq, dim = Q.shape
    Nd, Ld, _ = D.shape
    qm = _mask(q_mask, (Nq, Lq), Q.device)
    dm = _mask(d_mask, (Nd, Ld), Q.device)
    g = _grad_scores(grad_scores, (Nq, Nd), Q.device)
    am = _argmax_in(argmax, (Nq, Nd, Lq), Q.device)
    gQ = torch.empty((Nq, Lq, dim), dtype=torch.float32, device=Q.device) if need_grad_q else None
    gD = torch.empty((Nd, Ld, dim), dtype=torch.float32, device=Q.device) if need_grad_d else None
    flags = _flags(am is not None, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_BWD, Nq, Lq, Nd, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_bwd(_ptr(Q), _ptr(D), dt, Nq, Lq, Nd, Ld, dim, _ptr(qm), _ptr(dm),
                                _ptr(g), _ptr(am), _ptr(gQ), _ptr(gD), _ptr(ws), wsb, _stream()))
    return gQ, gD


def lik_maxsim_pairwise_bwd(Q, D, grad_scores, argmax=None, q_mask=None, d_mask=None,
                            need_grad_q=True, need_grad_d=True, fp32_split=False) -> Tuple:
    _same_batch(Q, D, "pairwise")
    dt = _embeddings(Q, D, fp32_split)
    B, Lq, dim = Q.shape
    _, Ld, _ = D.shape
    qm = _mask(q_mask, (B, Lq), Q.device)
    dm = _mask(d_mask, (B, Ld), Q.device)
    g = _grad_scores(grad_scores, (B,), Q.device)
    am = _argmax_in(argmax, (B, Lq), Q.device)
    gQ = torch.empty((B, Lq, dim), dtype=torch.float32, device=Q.device) if need_grad_q else None
    gD = torch.empty((B, Ld, dim), dtype=torch.float32, device=Q.device) if need_grad_d else None
    flags = _flags(am is not None, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_PAIRWISE_BWD, B, Lq, 1, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_pairwise_bwd(_ptr(Q), _ptr(D), dt, B, Lq, Ld, dim, _ptr(qm),
                                         _ptr(dm), _ptr(g), _ptr(am), _ptr(gQ), _ptr(gD),
                                         _ptr(ws), wsb, _stream()))
    return gQ, gD


def lik_maxsim_kd_bwd(Q, D, grad_scores, argmax=None, q_mask=None, d_mask=None,
                      need_grad_q=True, need_grad_d=True, fp32_split=False) -> Tuple:
    _same_batch(Q, D, "kd")
    dt = _embeddings(Q, D, fp32_split)
    B, Lq, dim = Q.shape
    _, N, Ld, _ = D.shape
    qm = _mask(q_mask, (B, Lq), Q.device)
    dm = _mask(d_mask, (B, N, Ld), Q.device)
    g = _grad_scores(grad_scores, (B, N), Q.device)
    am = _argmax_in(argmax, (B, N, Lq), Q.device)
    gQ = torch.empty((B, Lq, dim), dtype=torch.float32, device=Q.device) if need_grad_q else None
    gD = torch.empty((B, N, Ld, dim), dtype=torch.float32, device=Q.device) if need_grad_d else None
    flags = _flags(am is not None, dm, qm)
    wsb = lib().lik_workspace_bytes(LIK_OP_KD_BWD, B, Lq, N, Ld, dim, dt, flags)
    ws = _workspace(wsb, Q.device)
    _check(lib().lik_maxsim_kd_bwd(_ptr(Q), _ptr(D), dt, B, Lq, N, Ld, dim, _ptr(qm), _ptr(dm),
                                   _ptr(g), _ptr(am), _ptr(gQ), _ptr(gD), _ptr(ws), wsb,
                                   _stream()))
    return gQ, gD


def lik_ce_rows(scores, labels=None, scale=1.0, want_grad=True) -> Tuple:
    """Loss head: row cross-entropy of float32 scores [R, C] with targets
    `labels` [R] (int32) or the diagonal (None).  Returns (loss [1],
    row_loss [R], grad [R, C] or None), all float32 on the scores' device."""
    if scores.dtype != torch.float32 or scores.dim() != 2 or not scores.is_cuda:
        raise ValueError("scores must be a 2-D float32 CUDA tensor")
    S = scores.contiguous()
    R, C = S.shape
    lab = None
    if labels is not None:
        lab = labels.to(device=S.device, dtype=torch.int32).contiguous()
        if tuple(lab.shape) != (R,):
            raise ValueError(f"labels must have shape ({R},)")
    row_loss = torch.empty((R,), dtype=torch.float32, device=S.device)
    loss = torch.empty((1,), dtype=torch.float32, device=S.device)
    grad = torch.empty((R, C), dtype=torch.float32, device=S.device) if want_grad else None
    _check(lib().lik_ce_rows(_ptr(S), R, C, _ptr(lab), float(scale), _ptr(row_loss), _ptr(loss),
                             _ptr(grad), _stream()))
    return loss, row_loss, grad


# ---------------------------------------------------------------------------
# losses over rows of logits (include/lik_rows.h)
# ---------------------------------------------------------------------------

def _row_stride(x: torch.Tensor, name: str) -> int:
    """Row stride in elements of a 2-D tensor with dense columns."""
    R, C = x.shape
    if C > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have dense columns (stride 1)")
    if R > 1 and x.stride(0) < C:
        raise ValueError(f"{name} rows must not overlap")
    return x.stride(0) if R > 1 else C


def _rows(logits: torch.Tensor) -> Tuple:
    """(dtype code, R, C, row stride) of logits [R, C]."""
    if logits.dim() != 2 or logits.dtype not in DTYPE_CODE:
        raise ValueError("logits must be a 2-D float16, bfloat16 or float32 tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    R, C = logits.shape
    return DTYPE_CODE[logits.dtype], R, C, _row_stride(logits, "logits")


def _row_arg(x, shape, name: str, device, dtype=torch.float32):
    """A dense argument of this shape on the logits' device, or None.  Integer
    arguments may be int32 or int64 (values past int32 count as out of range)."""
    if x is None:
        return None
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(x.shape)}")
    if x.device != device:
        raise ValueError(f"{name} must be on the logits' device")
    if x.dtype != dtype:
        if dtype != torch.int32 or x.dtype != torch.int64:
            raise ValueError(f"{name} must be {dtype}, not {x.dtype}")
        x = x.clamp(-1, 2 ** 31 - 1).to(torch.int32)
    return x.contiguous()


def _row_grad(logits: torch.Tensor, want: bool, out: Optional[torch.Tensor]) -> Tuple:
    """(gradient tensor or None, its row stride)."""
    if not want:
        if out is not None:
            raise ValueError("grad_out given without want_grad")
        return None, 0
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    elif (out.shape != logits.shape or out.dtype != logits.dtype or
          out.device != logits.device):
        raise ValueError("grad_out must have the logits' shape, type and device")
    return out, _row_stride(out, "grad_out")


def _row_outs(R: int, device, *lengths) -> list:
    """float32 outputs; a call without rows writes none of them, so they are 0 then."""
    make = torch.empty if R else torch.zeros
    return [make(n, dtype=torch.float32, device=device) for n in lengths]


@functools.lru_cache(maxsize=1024)
def _rows_workspace_bytes(op: int, R: int, C: int, S: int, dt: int, flags: int) -> int:
    return lib().lik_rows_workspace_bytes(op, R, C, S, dt, flags)


_NO_SIZE = ctypes.c_size_t(-1).value


def _rows_workspace(op: int, R: int, C: int, S: int, dt: int, grad, device) -> Tuple:
    n = _rows_workspace_bytes(op, R, C, S, dt, 0 if grad is None else 1)
    if n == _NO_SIZE:                    # sizes that the call itself refuses
        n = 0
    return _workspace(n, device), n


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


_NOTHING = contextlib.nullcontext()


def _current(device):
    """Makes the tensors' device the current one for the call."""
    return _NOTHING if torch.cuda.current_device() == device.index else torch.cuda.device(device)


# the current stream's handle without a Stream object around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(device):
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def lik_logprob_rows_fwd(logits, targets, scale=1.0) -> Tuple:
    """Log-probabilities of the columns `targets` [R] of softmax(scale * logits
    [R, C]): (logp [R], lse [R]) float32.  Rows with a negative target are not
    read; both are 0 there."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    t = _row_arg(targets, (R,), "targets", dev, torch.int32)
    with _current(dev):
        logp, lse = _row_outs(R, dev, R, R)
        ws, wsb = _rows_workspace(LIK_ROWS_LOGPROB_FWD, R, C, 0, dt, None, dev)
        _check(lib().lik_logprob_rows_fwd(_addr(logits), dt, R, C, ld, _addr(t), float(scale),
                                          _addr(logp), _addr(lse), _addr(ws), wsb, _stream_of(dev)))
    return logp, lse


def lik_logprob_rows_bwd(logits, targets, lse, grad_logp, scale=1.0, grad_out=None):
    """Gradient [R, C] of sum(grad_logp * logp) in the logits' type; lse [R]
    from the forward with the same scale."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    t = _row_arg(targets, (R,), "targets", dev, torch.int32)
    lse = _row_arg(lse, (R,), "lse", dev)
    g = _row_arg(grad_logp, (R,), "grad_logp", dev)
    grad, gld = _row_grad(logits, True, grad_out)
    with _current(dev):
        _check(lib().lik_logprob_rows_bwd(_addr(logits), dt, R, C, ld, _addr(t), float(scale),
                                          _addr(lse), _addr(g), _addr(grad), gld, _stream_of(dev)))
    return grad


def lik_distill_rows(logits, teacher_idx, teacher_logits, teacher_lse=None, scale=1.0,
                     row_weight=None, want_grad=True, grad_out=None) -> Tuple:
    """KL divergence from a teacher known by its top logits: teacher_idx [R, K]
    columns (negative = absent), teacher_logits [R, K] float32.  Without
    teacher_lse the teacher is renormalised over its list; with it [R] (the
    log-sum-exp of scale * its logits over all columns) the mass it leaves to
    the other columns is matched too.  row_weight [R], None = 1 / R.  Returns
    (loss [1], row_loss [R], grad [R, C] in the logits' type or None)."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    if teacher_idx.dim() != 2:
        raise ValueError("teacher_idx must be [R, K]")
    K = teacher_idx.shape[1]
    idx = _row_arg(teacher_idx, (R, K), "teacher_idx", dev, torch.int32)
    val = _row_arg(teacher_logits, (R, K), "teacher_logits", dev)
    tl = _row_arg(teacher_lse, (R,), "teacher_lse", dev)
    w = _row_arg(row_weight, (R,), "row_weight", dev)
    grad, gld = _row_grad(logits, want_grad, grad_out)
    with _current(dev):
        row_loss, loss = _row_outs(R, dev, R, 1)
        ws, wsb = _rows_workspace(LIK_ROWS_DISTILL, R, C, 0, dt, grad, dev)
        _check(lib().lik_distill_rows(_addr(logits), dt, R, C, ld, _addr(idx), _addr(val), K,
                                      _addr(tl), float(scale), _addr(w), _addr(row_loss),
                                      _addr(loss), _addr(grad), gld, _addr(ws), wsb, _stream_of(dev)))
    return loss, row_loss, grad


def lik_policy_rows(logits, targets, old_logp, advantage, ref_logp=None, scale=1.0, clip_low=0.2,
                    clip_high=0.2, kl_coef=0.0, row_weight=None, want_grad=True,
                    grad_out=None) -> Tuple:
    """Clipped policy loss on the columns `targets` [R], with a KL term against
    ref_logp [R] if given.  row_weight [R], None = 1 / R.  Returns (loss [1],
    row_loss [R], logp [R], grad [R, C] in the logits' type or None)."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    t = _row_arg(targets, (R,), "targets", dev, torch.int32)
    old = _row_arg(old_logp, (R,), "old_logp", dev)
    adv = _row_arg(advantage, (R,), "advantage", dev)
    ref = _row_arg(ref_logp, (R,), "ref_logp", dev)
    w = _row_arg(row_weight, (R,), "row_weight", dev)
    grad, gld = _row_grad(logits, want_grad, grad_out)
    with _current(dev):
        row_loss, logp, loss = _row_outs(R, dev, R, R, 1)
        ws, wsb = _rows_workspace(LIK_ROWS_POLICY, R, C, 0, dt, grad, dev)
        _check(lib().lik_policy_rows(_addr(logits), dt, R, C, ld, _addr(t), _addr(old), _addr(adv),
                                     _addr(ref), float(scale), float(clip_low), float(clip_high),
                                     float(kl_coef), _addr(w), _addr(row_loss), _addr(logp),
                                     _addr(loss), _addr(grad), gld, _addr(ws), wsb, _stream_of(dev)))
    return loss, row_loss, logp, grad


def lik_preference_rows(logits, targets, seq_offsets, chosen, rejected, ref_logp=None,
                        kind=LIK_PREF_SIGMOID, beta=0.1, margin=0.0, smoothing=0.0,
                        mean_logp=False, scale=1.0, pair_weight=None, want_grad=True,
                        grad_out=None) -> Tuple:
    """Preference loss on paired log ratios: sequence s is the rows
    seq_offsets[s] .. seq_offsets[s + 1] - 1, pair p sets sequence chosen[p]
    against rejected[p]; ref_logp [S] or None.  pair_weight [P], None = 1 / P.
    Returns (loss [1], pair_loss [P], seq_logp [S], grad [R, C] in the logits'
    type or None).  Without any row (R == 0) nothing is computed: every output is
    0, the losses of pairs of empty sequences too."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1 or chosen.dim() != 1:
        raise ValueError("seq_offsets must be [S + 1], chosen and rejected [P]")
    S, P = seq_offsets.shape[0] - 1, chosen.shape[0]
    t = _row_arg(targets, (R,), "targets", dev, torch.int32)
    off = _row_arg(seq_offsets, (S + 1,), "seq_offsets", dev, torch.int32)
    c = _row_arg(chosen, (P,), "chosen", dev, torch.int32)
    r = _row_arg(rejected, (P,), "rejected", dev, torch.int32)
    ref = _row_arg(ref_logp, (S,), "ref_logp", dev)
    w = _row_arg(pair_weight, (P,), "pair_weight", dev)
    grad, gld = _row_grad(logits, want_grad, grad_out)
    with _current(dev):
        pair_loss, seq, loss = _row_outs(R, dev, P, S, 1)
        ws, wsb = _rows_workspace(LIK_ROWS_PREFERENCE, R, C, S, dt, grad, dev)
        _check(lib().lik_preference_rows(
            _addr(logits), dt, R, C, ld, _addr(t), _addr(off), S, _addr(c), _addr(r), P, _addr(ref),
            int(kind), float(beta), float(margin), float(smoothing), int(bool(mean_logp)),
            float(scale), _addr(w), _addr(pair_loss), _addr(seq), _addr(loss), _addr(grad), gld,
            _addr(ws), wsb, _stream_of(dev)))
    return loss, pair_loss, seq, grad


def lik_verify_rows(logits, draft_tokens, seq_offsets, accept_u, sample_u, draft_logits=None,
                    scale=1.0, draft_scale=1.0) -> Tuple:
    """Drafted tokens verified against softmax(scale * logits [R, C]): sequence s
    is the rows seq_offsets[s] .. seq_offsets[s + 1] - 1, row r has the draft
    draft_tokens[r] (negative: no draft from here on), the last row none.  Drafts
    were drawn from softmax(draft_scale * draft_logits [R, C]), or copied (None).
    accept_u [R] and sample_u [S] are uniform numbers within [0, 1).  Returns
    (tokens [R] int32: accepted drafts and then the drawn token, -1 elsewhere;
    accepted [S] int32; logp [R] float32 of the tokens, 0 elsewhere)."""
    dt, R, C, ld = _rows(logits)
    dev = logits.device
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
        raise ValueError("seq_offsets must be [S + 1]")
    S = seq_offsets.shape[0] - 1
    x = _row_arg(draft_tokens, (R,), "draft_tokens", dev, torch.int32)
    off = _row_arg(seq_offsets, (S + 1,), "seq_offsets", dev, torch.int32)
    u = _row_arg(accept_u, (R,), "accept_u", dev)
    su = _row_arg(sample_u, (S,), "sample_u", dev)
    dld = 0
    if draft_logits is not None:
        if (draft_logits.shape != logits.shape or draft_logits.dtype != logits.dtype or
                draft_logits.device != dev):
            raise ValueError("draft_logits must have the logits' shape, type and device")
        dld = _row_stride(draft_logits, "draft_logits")
    with _current(dev):
        tokens = torch.empty(R, dtype=torch.int32, device=dev)
        accepted = (torch.empty if R else torch.zeros)(S, dtype=torch.int32, device=dev)
        logp = torch.empty(R, dtype=torch.float32, device=dev)
        ws, wsb = _rows_workspace(LIK_ROWS_VERIFY, R, C, S, dt, draft_logits, dev)
        _check(lib().lik_verify_rows(
            logits.data_ptr(), dt, R, C, ld, _addr(draft_logits), dld, x.data_ptr(), off.data_ptr(),
            S, scale, draft_scale, u.data_ptr(), su.data_ptr(), tokens.data_ptr(),
            accepted.data_ptr(), logp.data_ptr(), _addr(ws), wsb, _stream_of(dev)))
    return tokens, accepted, logp


# ---------------------------------------------------------------------------
# a paged cache in 8 bits (include/lik_cache.h)
# ---------------------------------------------------------------------------

_F8 = torch.float8_e4m3fn


def _ints(x, shape, name: str, device):
    """A dense int32 argument of this shape on the device of the others."""
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(x.shape)}")
    if x.dtype != torch.int32:
        raise ValueError(f"{name} must be torch.int32, not {x.dtype}")
    if x.device != device:
        raise ValueError(f"{name} must be on {device}, not {x.device}")
    return x.contiguous()


def _in_place(x, shape, name: str, device):
    """One that the call changes: as it is."""
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _ints(x, shape, name, device)


def _table(block_table, S: int, device) -> Tuple:
    """(entries a row, row stride) of a block table."""
    if block_table.dim() != 2 or block_table.shape[0] != S:
        raise ValueError(f"block_table must be [{S}, max_blocks], not {tuple(block_table.shape)}")
    if block_table.dtype != torch.int32 or block_table.device != device:
        raise ValueError(f"block_table must be torch.int32 on {device}")
    return block_table.shape[1], _row_stride(block_table, "block_table")


def lik_cache_tables(old_len, new_len, block_table, ring, ring_state, block_size, tokens) -> Tuple:
    """Block tables of requests that go from old_len [S] to new_len [S] tokens:
    blocks of block_size tokens are taken from the pool of free ones (ring [N]
    with ring_state [4] = head, count, 0, 0) or given back to it, and
    block_table [S, max_blocks] is changed to match, all in place, all int32.
    Returns (granted [S]: the new length, or the old one where the pool or the
    table is too short; token_offsets [S + 1] of the new tokens; slots [tokens]
    of the new tokens, -1 where there is none)."""
    if not old_len.is_cuda:
        raise ValueError("old_len must be a GPU tensor")
    if old_len.dim() != 1 or ring.dim() != 1:
        raise ValueError("old_len must be [S] and ring [N]")
    dev, S, N = old_len.device, old_len.shape[0], ring.shape[0]
    old = _ints(old_len, (S,), "old_len", dev)
    new = _ints(new_len, (S,), "new_len", dev)
    width, ld = _table(block_table, S, dev)
    _in_place(ring, (N,), "ring", dev)
    _in_place(ring_state, (4,), "ring_state", dev)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    with _current(dev):
        granted = torch.empty(S, dtype=torch.int32, device=dev)
        offsets = torch.empty(S + 1, dtype=torch.int32, device=dev)
        slots = torch.empty(tokens, dtype=torch.int32, device=dev)
        _check(lib().lik_cache_tables(
            old.data_ptr(), new.data_ptr(), S, block_size, block_table.data_ptr(), width, ld,
            ring.data_ptr(), N, ring_state.data_ptr(), granted.data_ptr(), offsets.data_ptr(),
            slots.data_ptr(), tokens, _stream_of(dev)))
    return granted, offsets, slots


def _block_stride(x, name: str) -> int:
    """Bytes from block to block of one that is dense within a block."""
    N, heads, rows, last = x.shape
    a, b, c, d = x.stride()
    inner = rows * last
    if d != 1 or c != last or (heads > 1 and b != inner) or (N > 1 and a < heads * inner):
        raise ValueError(f"{name} must be dense within a block")
    return a if N > 1 else heads * inner


def _blocks(k_cache, v_cache, k_scale, v_scale, device) -> Tuple:
    """What the C ABI takes of a cache: addresses, sizes and block strides."""
    if k_cache.dim() != 4 or k_cache.dtype != _F8 or v_cache.dtype != _F8:
        raise ValueError("k_cache must be [N, heads, block_size, dim] and v_cache "
                         "[N, heads, dim, block_size], float8_e4m3fn")
    N, heads, bs, dim = k_cache.shape
    if v_cache.shape != (N, heads, dim, bs):
        raise ValueError(f"v_cache must have shape {(N, heads, dim, bs)}, not {tuple(v_cache.shape)}")
    inner = bs * dim
    size = heads * inner
    k_stride = v_stride = size
    if k_cache.stride() != (size, inner, dim, 1) or v_cache.stride() != (size, inner, bs, 1):
        k_stride, v_stride = _block_stride(k_cache, "k_cache"), _block_stride(v_cache, "v_cache")
    for x, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        if x.shape != (N, heads) or x.dtype != torch.float32 or not x.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 of shape {(N, heads)}")
    if not (device == k_cache.device == v_cache.device == k_scale.device == v_scale.device):
        raise ValueError(f"the cache must be on {device}")
    return (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), N,
            heads, bs, dim, k_stride, v_stride)


def _token_stride(x, heads: int, dim: int, name: str) -> int:
    """Token stride of [T, heads, dim] with dense heads."""
    if x.dim() != 3 or x.shape[1] != heads or x.shape[2] != dim:
        raise ValueError(f"{name} must have shape [T, {heads}, {dim}], not {tuple(x.shape)}")
    a, b, c = x.stride()
    if c != 1 or (heads > 1 and b != dim) or (x.shape[0] > 1 and a < heads * dim):
        raise ValueError(f"{name} must have dense heads and tokens that do not overlap")
    return a if x.shape[0] > 1 else heads * dim


def _tokens(x, name: str) -> int:
    """dtype code of a tensor of tokens."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if x.dtype not in DTYPE_CODE:
        raise ValueError(f"{name} must be float16, bfloat16 or float32")
    return DTYPE_CODE[x.dtype]


def lik_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale) -> None:
    """Writes the keys and values of T tokens, k and v [T, heads, dim], to their
    slots [T] (int32, negative: none) of the cache in place: k_cache
    [N, heads, block_size, dim] and v_cache [N, heads, dim, block_size] in
    float8_e4m3fn, with scales [N, heads] in float32.  The tokens of a block
    follow each other; a call with a block's first slot starts the block anew."""
    dt = _tokens(k, "k")
    dev = k.device
    if v.shape != k.shape or v.dtype != k.dtype or v.device != dev:
        raise ValueError("v must have k's shape, type and device")
    cache = _blocks(k_cache, v_cache, k_scale, v_scale, dev)
    heads, dim = cache[5], cache[7]
    kld, vld = _token_stride(k, heads, dim, "k"), _token_stride(v, heads, dim, "v")
    T = k.shape[0]
    at = _ints(slots, (T,), "slots", dev)
    with _current(dev):
        _check(lib().lik_cache_append(k.data_ptr(), v.data_ptr(), dt, T, kld, vld, at.data_ptr(),
                                      *cache, _stream_of(dev)))


@functools.lru_cache(maxsize=1024)
def _attention_workspace_bytes(T: int, S: int, hq: int, hkv: int, dim: int, dt: int) -> int:
    n = lib().lik_cache_workspace_bytes(T, S, hq, hkv, dim, dt)
    return 0 if n == _NO_SIZE else n     # sizes that the call itself refuses


def lik_cache_attention(q, q_offsets, kv_len, block_table, k_cache, v_cache, k_scale, v_scale,
                        scale=None, out=None, want_lse=False) -> Tuple:
    """Causal attention of q [T, q_heads, dim] over a cache in 8 bits: the rows
    q_offsets[s] .. q_offsets[s + 1] - 1 are the last tokens of request s, which has
    kv_len[s] tokens in the blocks of row s of block_table [S, max_blocks] (all
    int32).  scale None = dim ** -0.5.  Returns (out [T, q_heads, dim] in q's
    type, lse [T, q_heads] float32 or None); rows that attend to nothing or
    belong to no request are 0, with lse -inf."""
    dt = _tokens(q, "q")
    dev = q.device
    cache = _blocks(k_cache, v_cache, k_scale, v_scale, dev)
    hkv, dim = cache[5], cache[7]
    T, hq = q.shape[0], q.shape[1] if q.dim() > 1 else 0
    qld = _token_stride(q, hq, dim, "q")
    if kv_len.dim() != 1:
        raise ValueError("kv_len must be [S]")
    S = kv_len.shape[0]
    off = _ints(q_offsets, (S + 1,), "q_offsets", dev)
    lens = _ints(kv_len, (S,), "kv_len", dev)
    width, ld = _table(block_table, S, dev)
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype or out.device != dev):
        raise ValueError("out must have q's shape, type and device")
    with _current(dev):
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        lse = torch.empty((T, hq), dtype=torch.float32, device=dev) if want_lse else None
        wsb = _attention_workspace_bytes(T, S, hq, hkv, dim, dt)
        ws = _workspace(wsb, dev)
        _check(lib().lik_cache_attention(
            q.data_ptr(), dt, T, hq, qld, off.data_ptr(), lens.data_ptr(), S,
            block_table.data_ptr(), width, ld, *cache, dim ** -0.5 if scale is None else scale,
            out.data_ptr(), _token_stride(out, hq, dim, "out"), _addr(lse), _addr(ws), wsb,
            _stream_of(dev)))
    return out, lse


FORWARD = {"allpairs": lik_maxsim_fwd, "pairwise": lik_maxsim_pairwise_fwd,
           "kd": lik_maxsim_kd_fwd}
BACKWARD = {"allpairs": lik_maxsim_bwd, "pairwise": lik_maxsim_pairwise_bwd,
            "kd": lik_maxsim_kd_bwd}
