"""Thin ctypes binding of librlq.so (include/rlq.h).

The functions named ``rlq_*`` mirror the C entry points one to one: plain
integers for device pointers, sizes and the stream, and an ``RlqError`` raised
for a non-OK status.  The lower-case helpers below them take torch tensors,
allocate outputs with torch (device memory is PyTorch's plumbing here) and call
the same entry points; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or cannot be
loaded, the first call raises.

``stream`` names the stream that a helper launches on (a torch stream or a handle); without
it that is the current one.  Scratch comes from the launching stream's pool, outputs from
the current stream's.  So where the two differ, the named stream has to have waited for the
current one, as for any tensor that is made on one stream and used on another.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from . import build as _build

GRP = 128

_P = ctypes.c_void_p
_I = ctypes.c_int64
_F = ctypes.c_float

_SIGS = {
    "rlq_quant_act_1x128": [_P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P],
    "rlq_quant_weight_128x128": [_P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P],
    "rlq_rmsnorm_quant_act_1x128": [_P, _I, _I, _I, _P, ctypes.c_float, _P, _P, _I, _P, _I, _P, _I, _P, _I, _P],
    "rlq_gemm_fprop": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_gemm_dgrad": [_P, _I, _P, _I, _P, _I, ctypes.c_int, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_gemm_wgrad": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_gemm_splitk_workspace_bytes": [ctypes.c_int, _I, _I, _I, ctypes.POINTER(_I)],
    "rlq_gemm_fprop_splitk": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_gemm_dgrad_splitk": [_P, _I, _P, _I, _P, _I, ctypes.c_int, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_gemm_wgrad_splitk": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_gemm_fprop_splitk_static": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_quant_per_row": [_P, _I, _I, _I, _P, _I, _P, _P, _I, _P],
    "rlq_gemm_fprop_per_channel": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_gemm_fprop_per_channel_splitk": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_uaq_fold": [_P, _I, _I, _I, _P, _P, _I, _I, _P],
    "rlq_gemm_wgrad_accumulate": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_quant_nvfp4": [_P, _I, _I, _I, _P, _I, _P, _I, _P, _P],
    "rlq_gemm_nvfp4_weight_only": [_P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _P],
    "rlq_gemm_nvfp4_weight_only_splitk": [_P, _I, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _P, _I, _P],
    "rlq_aqn_sigma": [ctypes.c_float, ctypes.c_float, _I, _I, ctypes.POINTER(ctypes.c_float)],
    "rlq_aqn_perturb": [_P, _I, _P, ctypes.c_float, _P],
    "rlq_add_rmsnorm_quant_act_1x128": [_P, _I, _P, _I, _I, _I, _P, _F, _P, _I, _P, _P, _I, _P, _I, _P, _I, _P, _I, _P],
    "rlq_rmsnorm_backward_workspace_bytes": [_I, _I, ctypes.POINTER(_I)],
    "rlq_rmsnorm_backward": [_P, _I, _P, _I, _P, _P, _P, _I, _P, _I, _P, _I, _I, _P, _I, _P],
    "rlq_gemm_gated_fprop": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _P],
    "rlq_gated_backward": [_P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _P],
    "rlq_quant_mxfp4": [_P, _I, _I, _I, _P, _I, _P, _P, _I, _P, _P],
    "rlq_dequant_mxfp4": [_P, _I, _P, _I, _I, _P, _I, _P],
    "rlq_gemm_mxfp4": [_P, _I, _P, _P, _I, _P, _P, ctypes.c_int, _I, _I, _I, _I, _P],
    "rlq_token_logprobs": [_P, ctypes.c_int, _I, _I, _I, _P, _F, _P, _P, _P],
    "rlq_token_logprobs_top": [_P, ctypes.c_int, _I, _I, _I, _P, _F, _I, _P, _P, _P, _P, _P, _P],
    "rlq_token_logprobs_backward": [_P, ctypes.c_int, _I, _I, _I, _P, _F, _P, _P, _P, _P, _P, _I, _P],
    "rlq_policy_loss": [_P, ctypes.c_int, _I, _I, _I, _P, _F, _P, _P, _P, _P, _P, _P, _F, _F, _F, _F, _P, _P, _P, _I,
                        _P],
    "rlq_check": [_P],
    "rlq_diag_bounded_wait": [_I, _P],
    "rlq_diag_arm_gemm_stall": [],
    "rlq_diag_gemm_mxfp4_cut": [_I, _I, _I, ctypes.c_int, ctypes.c_int, _P],
}

STATUS = {0: "RLQ_OK", 1: "RLQ_ERR_INVALID_ARG", 2: "RLQ_ERR_UNSUPPORTED", 3: "RLQ_ERR_MISALIGNED",
          4: "RLQ_ERR_CUDA", 5: "RLQ_ERR_TIMEOUT"}


class RlqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load librlq.so (building it first if its sources are newer)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path) or _build._stale():
                _build.build()
            L = ctypes.CDLL(path)
            for name, args in _SIGS.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            L.rlq_status_string.argtypes = [ctypes.c_int]
            L.rlq_status_string.restype = ctypes.c_char_p
            L.rlq_last_error.argtypes = []
            L.rlq_last_error.restype = ctypes.c_char_p
            L.rlq_version.argtypes = []
            L.rlq_version.restype = ctypes.c_char_p
            _lib = L
    return _lib


_fns: dict = {}  # entry points looked up so far


def _call(name: str, *args) -> int:
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    st = fn(*args)
    if st != 0:
        raise RlqError(st, lib().rlq_last_error().decode(errors="replace"))
    return st


# ------------------------------------------------- raw C-ABI mirrors ---

def rlq_quant_act_1x128(x, M, K, ldx, q, ldq, s, lds, qT, ldqT, sc, ldsc, stream):
    return _call("rlq_quant_act_1x128", x, M, K, ldx, q, ldq, s, lds, qT, ldqT, sc, ldsc, stream)


def rlq_rmsnorm_quant_act_1x128(h, M, K, ldh, gamma, eps, rstd, q, ldq, s, lds, qT, ldqT, sc, ldsc, stream):
    return _call("rlq_rmsnorm_quant_act_1x128", h, M, K, ldh, gamma, eps, rstd, q, ldq, s, lds, qT, ldqT, sc, ldsc,
                 stream)


def rlq_quant_weight_128x128(w, N, K, ldw, q, ldq, s, lds, qT, ldqT, stream):
    return _call("rlq_quant_weight_128x128", w, N, K, ldw, q, ldq, s, lds, qT, ldqT, stream)


def rlq_gemm_fprop(xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, stream):
    return _call("rlq_gemm_fprop", xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, stream)


def rlq_gemm_dgrad(dyq, lddyq, dys, lddys, w, ldw, wq_is_transposed, ws, ldws, dx, lddx, M, N, K, stream):
    return _call("rlq_gemm_dgrad", dyq, lddyq, dys, lddys, w, ldw, wq_is_transposed, ws, ldws, dx, lddx,
                 M, N, K, stream)


def rlq_gemm_wgrad(dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw, lddw, M, N, K, stream):
    return _call("rlq_gemm_wgrad", dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw, lddw, M, N, K, stream)


GEMM_FPROP, GEMM_DGRAD, GEMM_WGRAD, GEMM_NVFP4_WEIGHT_ONLY = 0, 1, 2, 3


def rlq_gemm_splitk_workspace_bytes(kind, M, N, K) -> int:
    out = _I(0)
    _call("rlq_gemm_splitk_workspace_bytes", kind, M, N, K, ctypes.byref(out))
    return out.value


def rlq_gemm_fprop_splitk(xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, workspace, workspace_bytes,
                          stream):
    return _call("rlq_gemm_fprop_splitk", xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, workspace,
                 workspace_bytes, stream)


def rlq_gemm_dgrad_splitk(dyq, lddyq, dys, lddys, w, ldw, wq_is_transposed, ws, ldws, dx, lddx, M, N, K, workspace,
                          workspace_bytes, stream):
    return _call("rlq_gemm_dgrad_splitk", dyq, lddyq, dys, lddys, w, ldw, wq_is_transposed, ws, ldws, dx, lddx,
                 M, N, K, workspace, workspace_bytes, stream)


def rlq_gemm_wgrad_splitk(dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw, lddw, M, N, K, workspace,
                          workspace_bytes, stream):
    return _call("rlq_gemm_wgrad_splitk", dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw, lddw, M, N, K,
                 workspace, workspace_bytes, stream)


# Size of the library's static split-K scratch (RLQ_STATIC_SCRATCH_BYTES in rlq.h).
STATIC_SCRATCH_BYTES = 16 << 20


def rlq_gemm_fprop_splitk_static(xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, stream):
    """Split-K FProp on the library's static scratch, for callers that cannot
    allocate device memory (see rlq.h); the plan must fit STATIC_SCRATCH_BYTES."""
    return _call("rlq_gemm_fprop_splitk_static", xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, y, ldy, M, N, K, stream)


def rlq_quant_per_row(x, M, K, ldx, q, ldq, s, s_rep, ld_rep, stream):
    return _call("rlq_quant_per_row", x, M, K, ldx, q, ldq, s, s_rep, ld_rep, stream)


def rlq_gemm_fprop_per_channel(xq, ldxq, xs_rep, ldxs, wq, ldwq, ws_rep, ldws, y, ldy, M, N, K, stream):
    return _call("rlq_gemm_fprop_per_channel", xq, ldxq, xs_rep, ldxs, wq, ldwq, ws_rep, ldws, y, ldy, M, N, K,
                 stream)


def rlq_gemm_fprop_per_channel_splitk(xq, ldxq, xs_rep, ldxs, wq, ldwq, ws_rep, ldws, y, ldy, M, N, K, workspace,
                                      workspace_bytes, stream):
    return _call("rlq_gemm_fprop_per_channel_splitk", xq, ldxq, xs_rep, ldxs, wq, ldwq, ws_rep, ldws, y, ldy, M, N,
                 K, workspace, workspace_bytes, stream)


def rlq_gemm_wgrad_accumulate(dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw_acc, ld_acc, M, N, K,
                              workspace, workspace_bytes, stream):
    return _call("rlq_gemm_wgrad_accumulate", dyqT, lddyqT, dysc, lddysc, xqT, ldxqT, xsc, ldxsc, dw_acc, ld_acc,
                 M, N, K, workspace, workspace_bytes, stream)


def rlq_quant_nvfp4(w, N, K, ldw, q, ldq, sb, ldsb, st, stream):
    return _call("rlq_quant_nvfp4", w, N, K, ldw, q, ldq, sb, ldsb, st, stream)


def rlq_gemm_nvfp4_weight_only(x, ldx, wq, ldwq, wsb, ldwsb, wst, y, ldy, M, N, K, stream):
    return _call("rlq_gemm_nvfp4_weight_only", x, ldx, wq, ldwq, wsb, ldwsb, wst, y, ldy, M, N, K, stream)


def rlq_gemm_nvfp4_weight_only_splitk(x, ldx, wq, ldwq, wsb, ldwsb, wst, y, ldy, M, N, K, workspace,
                                      workspace_bytes, stream):
    return _call("rlq_gemm_nvfp4_weight_only_splitk", x, ldx, wq, ldwq, wsb, ldwsb, wst, y, ldy, M, N, K, workspace,
                 workspace_bytes, stream)


DTYPE_BF16, DTYPE_F32 = 0, 1


def rlq_quant_mxfp4(x, M, K, ldx, q, ldq, s, qT, ldqT, sT, stream):
    return _call("rlq_quant_mxfp4", x, M, K, ldx, q, ldq, s, qT, ldqT, sT, stream)


def rlq_dequant_mxfp4(q, ldq, s, rows, cols, x, ldx, stream):
    return _call("rlq_dequant_mxfp4", q, ldq, s, rows, cols, x, ldx, stream)


def rlq_gemm_mxfp4(xq, ldxq, xs, wq, ldwq, ws, y, dtype, ldy, M, N, K, stream):
    return _call("rlq_gemm_mxfp4", xq, ldxq, xs, wq, ldwq, ws, y, dtype, ldy, M, N, K, stream)


def rlq_aqn_sigma(sigma_start, sigma_end, t, T) -> float:
    out = ctypes.c_float()
    _call("rlq_aqn_sigma", sigma_start, sigma_end, t, T, ctypes.byref(out))
    return out.value


def rlq_aqn_perturb(gamma, K, z, sigma, stream):
    return _call("rlq_aqn_perturb", gamma, K, z, sigma, stream)


def rlq_uaq_fold(w, N, K, ldw, s, prev, R, ldp, stream):
    return _call("rlq_uaq_fold", w, N, K, ldw, s, prev, R, ldp, stream)


def rlq_add_rmsnorm_quant_act_1x128(res, ldr, delta, ldd, M, K, gamma, eps, h, ldh, rstd, q, ldq, s, lds, qT, ldqT, sc,
                                    ldsc, stream):
    return _call("rlq_add_rmsnorm_quant_act_1x128", res, ldr, delta, ldd, M, K, gamma, eps, h, ldh, rstd, q, ldq, s, lds,
                 qT, ldqT, sc, ldsc, stream)


def rlq_rmsnorm_backward_workspace_bytes(M, K) -> int:
    out = _I(0)
    _call("rlq_rmsnorm_backward_workspace_bytes", M, K, ctypes.byref(out))
    return out.value


def rlq_rmsnorm_backward(dx, lddx, h, ldh, rstd, gamma, dres, lddres, dh, lddh, dgamma, M, K, workspace,
                         workspace_bytes, stream):
    return _call("rlq_rmsnorm_backward", dx, lddx, h, ldh, rstd, gamma, dres, lddres, dh, lddh, dgamma, M, K, workspace,
                 workspace_bytes, stream)


def rlq_gemm_gated_fprop(xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, aq, ldaq, as_, ldas, guq, ldguq, gus, ldgus, M, F, K,
                         stream):
    return _call("rlq_gemm_gated_fprop", xq, ldxq, xs, ldxs, wq, ldwq, ws, ldws, aq, ldaq, as_, ldas, guq, ldguq, gus,
                 ldgus, M, F, K, stream)


def rlq_gated_backward(da, ldda, guq, ldguq, gus, ldgus, q, ldq, s, lds, qT, ldqT, sc, ldsc, aT, ldaT, ac, ldac, M, F,
                       stream):
    return _call("rlq_gated_backward", da, ldda, guq, ldguq, gus, ldgus, q, ldq, s, lds, qT, ldqT, sc, ldsc, aT, ldaT,
                 ac, ldac, M, F, stream)


def rlq_token_logprobs(logits, dtype, ld, rows, V, targets, temperature, lp, lse, stream):
    return _call("rlq_token_logprobs", logits, dtype, ld, rows, V, targets, temperature, lp, lse, stream)


def rlq_token_logprobs_top(logits, dtype, ld, rows, V, targets, temperature, top, lp, lse, entropy, top_ids, top_lp,
                           stream):
    return _call("rlq_token_logprobs_top", logits, dtype, ld, rows, V, targets, temperature, top, lp, lse, entropy,
                 top_ids, top_lp, stream)


def rlq_token_logprobs_backward(logits, dtype, ld, rows, V, targets, temperature, lse, entropy, dlp, dentropy, dlogits,
                                ldd, stream):
    return _call("rlq_token_logprobs_backward", logits, dtype, ld, rows, V, targets, temperature, lse, entropy, dlp,
                 dentropy, dlogits, ldd, stream)


def rlq_policy_loss(logits, dtype, ld, rows, V, targets, temperature, lp_old, adv, weight, lp_behav, lp_ref, clip_hi,
                    eps_lo, eps_hi, tis_cap, kl_beta, loss, lp, dlogits, ldd, stream):
    return _call("rlq_policy_loss", logits, dtype, ld, rows, V, targets, temperature, lp_old, adv, weight, lp_behav,
                 lp_ref, clip_hi, eps_lo, eps_hi, tis_cap, kl_beta, loss, lp, dlogits, ldd, stream)


def rlq_check(stream):
    return _call("rlq_check", stream)


def rlq_diag_bounded_wait(timeout_us, stream):
    return _call("rlq_diag_bounded_wait", timeout_us, stream)


def rlq_diag_arm_gemm_stall():
    return _call("rlq_diag_arm_gemm_stall")


def rlq_diag_gemm_mxfp4_cut(M, N, K, dtype, aligned) -> tuple:
    """(pairs, staged outputs, rows of a tile, CTAs that share a contraction, two CTAs to an SM, tiles
    of the busiest CTA or pair)."""
    out = (ctypes.c_int32 * 6)()
    _call("rlq_diag_gemm_mxfp4_cut", M, N, K, dtype, int(aligned), out)
    return tuple(out)


def rlq_status_string(status: int) -> str:
    return lib().rlq_status_string(status).decode()


def rlq_last_error() -> str:
    return lib().rlq_last_error().decode(errors="replace")


def rlq_version() -> str:
    return lib().rlq_version().decode()


# ------------------------------------------------------ torch helpers ---

def _stream(stream) -> int:
    if stream is None:
        # the current stream's handle without building a Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """Workspace of a call on ``stream``, out of that stream's pool.  Nothing that is queued
    on another stream uses such a block, and once the helper has let go of it, only work
    behind the call gets it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        # (a stream object made around handle 0 would be a new stream, not the default one)
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _given(workspace: torch.Tensor):
    """(address, bytes) of a caller's workspace, which the kernels write as plain memory."""
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if not workspace.is_cuda:
        raise ValueError("workspace must be a CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _ld(t) -> int:
    """Row pitch in elements of a 2-D tensor whose rows are contiguous.  The stride of a
    dimension of size 1 is arbitrary (torch counts any as contiguous) and not looked at."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("expected a 2-D tensor with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _round_up(v: int, m: int) -> int:
    return (v + m - 1) // m * m


def empty_codes_T(K: int, M: int, device) -> torch.Tensor:
    """[K, M] uint8 view of a [K, round_up(M, 16)] buffer (TMA-ready pitch)."""
    return torch.empty((K, _round_up(max(M, 1), 16)), dtype=torch.uint8, device=device)[:, :M]


def quant_act_1x128(x: torch.Tensor, colwise: bool = False, stream=None):
    """1x128 quantization of bf16 x [M, K]; with ``colwise`` also the fused
    128x1 codes (transposed) and scales.

    Returns (q [M,K] u8, s [K/128, M] f32, qT [K, M] u8 or None, sc [ceil(M/128), K] f32 or None).
    """
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    M, K = x.shape
    dev = x.device
    q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    s = torch.empty((K // GRP, M), dtype=torch.float32, device=dev)
    qT = sc = None
    if colwise:
        qT = empty_codes_T(K, M, dev)
        sc = torch.empty(((M + GRP - 1) // GRP, K), dtype=torch.float32, device=dev)
    rlq_quant_act_1x128(x.data_ptr(), M, K, _ld(x), q.data_ptr(), K, s.data_ptr(), max(M, 1),
                        _ptr(qT), _ld(qT) if qT is not None else 0, _ptr(sc), K if sc is not None else 0,
                        _stream(stream))
    return q, s, qT, sc


def rmsnorm_quant_act_1x128(h: torch.Tensor, gamma: torch.Tensor, eps: float, colwise: bool = False, stream=None):
    """RMSNorm of the bf16 hidden state h [M, K] with the (UAQ-folded) bf16 norm
    weight gamma [K], quantized 1x128 (and with ``colwise`` 128x1) without
    writing the normalised activation.

    Returns (q, s, qT, sc) as ``quant_act_1x128`` and rstd [M] f32."""
    if h.dtype != torch.bfloat16 or gamma.dtype != torch.bfloat16:
        raise TypeError("h and gamma must be bfloat16")
    M, K = h.shape
    if gamma.shape != (K,) or not gamma.is_contiguous():
        raise ValueError("gamma must be a contiguous [K] tensor")
    dev = h.device
    q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    s = torch.empty((K // GRP, M), dtype=torch.float32, device=dev)
    rstd = torch.empty((max(M, 1),), dtype=torch.float32, device=dev)[:M]
    qT = sc = None
    if colwise:
        qT = empty_codes_T(K, M, dev)
        sc = torch.empty(((M + GRP - 1) // GRP, K), dtype=torch.float32, device=dev)
    rlq_rmsnorm_quant_act_1x128(h.data_ptr(), M, K, _ld(h), gamma.data_ptr(), eps, rstd.data_ptr(), q.data_ptr(), K,
                                s.data_ptr(), max(M, 1), _ptr(qT), _ld(qT) if qT is not None else 0, _ptr(sc),
                                K if sc is not None else 0, _stream(stream))
    return q, s, qT, sc, rstd


def quant_weight_128x128(w: torch.Tensor, transposed: bool = False, stream=None):
    """128x128 block quantization of bf16 w [N, K].

    Returns (q [N,K] u8, s [N/128, K/128] f32, qT [K,N] u8 or None).
    """
    if w.dtype != torch.bfloat16:
        raise TypeError("w must be bfloat16")
    N, K = w.shape
    dev = w.device
    q = torch.empty((N, K), dtype=torch.uint8, device=dev)
    s = torch.empty((N // GRP, K // GRP), dtype=torch.float32, device=dev)
    qT = torch.empty((K, N), dtype=torch.uint8, device=dev) if transposed else None
    rlq_quant_weight_128x128(w.data_ptr(), N, K, _ld(w), q.data_ptr(), K, s.data_ptr(), max(K // GRP, 1),
                             _ptr(qT), N if qT is not None else 0, _stream(stream))
    return q, s, qT


def quant_per_row(x: torch.Tensor, replicate: bool = True, stream=None):
    """Per-row FP8 quantization of bf16 x [M, K] (per-token activations, or
    per-channel weights with x = W).

    Returns (q [M,K] u8, s [M] f32, s_rep [K/128, M] f32 or None): s_rep holds
    each row's scale once per K-block, the layout ``gemm_fprop_per_channel`` reads.
    """
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    M, K = x.shape
    dev = x.device
    q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    s = torch.empty((max(M, 1),), dtype=torch.float32, device=dev)[:M]
    Mp = _round_up(max(M, 1), 4)
    s_rep = torch.empty((K // GRP, Mp), dtype=torch.float32, device=dev)[:, :M] if replicate else None
    rlq_quant_per_row(x.data_ptr(), M, K, _ld(x), q.data_ptr(), K, s.data_ptr(), _ptr(s_rep),
                      Mp if replicate else 0, _stream(stream))
    return q, s, s_rep


def gemm_fprop_per_channel(xq, xs_rep, wq, ws_rep, out=None, stream=None, split_k: bool = False, workspace=None):
    """Y [M, N] bf16 = diag(sx) Qx Qw^T diag(sw) from per-token X codes and
    per-channel W codes, with the scales in the replicated [K/128, rows] layout.
    ``split_k`` as in ``gemm_fprop`` (the FProp plan)."""
    M, K = xq.shape
    N = wq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    args = (xq.data_ptr(), _ld(xq), xs_rep.data_ptr(), _ld(xs_rep), wq.data_ptr(), _ld(wq), ws_rep.data_ptr(),
            _ld(ws_rep), y.data_ptr(), _ld(y), M, N, K)
    if split_k:
        rlq_gemm_fprop_per_channel_splitk(*args, *_workspace(GEMM_FPROP, M, N, K, workspace, xq.device, stream),
                                          _stream(stream))
    else:
        rlq_gemm_fprop_per_channel(*args, _stream(stream))
    return y


def _workspace(kind: int, M: int, N: int, K: int, workspace, device, stream):
    """(pointer, bytes) of the split-K workspace: the caller's uint8 tensor, or
    one allocated with torch for the library's plan (None when it is one pass)."""
    if workspace is not None:
        return _given(workspace)
    nbytes = rlq_gemm_splitk_workspace_bytes(kind, M, N, K)
    if nbytes == 0:
        return None, 0
    return _scratch(nbytes, device, stream).data_ptr(), nbytes


def gemm_fprop(xq, xs, wq, ws, out=None, stream=None, split_k: bool = False, workspace=None):
    """Y [M, N] bf16 = X W^T from 1x128 X codes and 128x128 W codes.

    ``split_k`` runs the split-K form with ``workspace`` (a device tensor) or
    a workspace allocated here for the library's plan."""
    M, K = xq.shape
    N = wq.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    args = (xq.data_ptr(), _ld(xq), xs.data_ptr(), _ld(xs), wq.data_ptr(), _ld(wq), ws.data_ptr(), _ld(ws),
            y.data_ptr(), _ld(y), M, N, K)
    if split_k:
        rlq_gemm_fprop_splitk(*args, *_workspace(GEMM_FPROP, M, N, K, workspace, xq.device, stream), _stream(stream))
    else:
        rlq_gemm_fprop(*args, _stream(stream))
    return y


def gemm_dgrad(dyq, dys, w, ws, transposed: bool = True, out=None, stream=None, split_k: bool = False,
               workspace=None):
    """dX [M, K] bf16 = dY W.  ``w`` is the transposed weight codes [K, N]
    (``transposed=True``) or the FProp codes [N, K]."""
    M, N = dyq.shape
    K = w.shape[0] if transposed else w.shape[1]
    dx = out if out is not None else torch.empty((M, K), dtype=torch.bfloat16, device=dyq.device)
    args = (dyq.data_ptr(), _ld(dyq), dys.data_ptr(), _ld(dys), w.data_ptr(), _ld(w), 1 if transposed else 0,
            ws.data_ptr(), _ld(ws), dx.data_ptr(), _ld(dx), M, N, K)
    if split_k:
        rlq_gemm_dgrad_splitk(*args, *_workspace(GEMM_DGRAD, M, N, K, workspace, dyq.device, stream), _stream(stream))
    else:
        rlq_gemm_dgrad(*args, _stream(stream))
    return dx


def gemm_wgrad(dyqT, dysc, xqT, xsc, out=None, stream=None, split_k: bool = False, workspace=None):
    """dW [N, K] bf16 = dY^T X from the 128x1 (transposed) codes of dY and X."""
    N, M = dyqT.shape
    K = xqT.shape[0]
    dw = out if out is not None else torch.empty((N, K), dtype=torch.bfloat16, device=dyqT.device)
    args = (dyqT.data_ptr(), _ld(dyqT), dysc.data_ptr(), _ld(dysc), xqT.data_ptr(), _ld(xqT),
            xsc.data_ptr(), _ld(xsc), dw.data_ptr(), _ld(dw), M, N, K)
    if split_k:
        rlq_gemm_wgrad_splitk(*args, *_workspace(GEMM_WGRAD, M, N, K, workspace, dyqT.device, stream), _stream(stream))
    else:
        rlq_gemm_wgrad(*args, _stream(stream))
    return dw


def gemm_wgrad_accumulate_(dw_acc: torch.Tensor, dyqT, dysc, xqT, xsc, workspace=None, stream=None):
    """dw_acc [N, K] fp32 += dY^T X (the WGrad product, kept in fp32).  The
    workspace (uint8 device tensor) defaults to the library's split-K plan (none
    when the plan is one pass: the GEMM's epilogue then adds into dw_acc)."""
    if dw_acc.dtype != torch.float32:
        raise TypeError("dw_acc must be float32")
    N, M = dyqT.shape
    K = xqT.shape[0]
    ptr, nbytes = _workspace(GEMM_WGRAD, M, N, K, workspace, dw_acc.device, stream)
    rlq_gemm_wgrad_accumulate(dyqT.data_ptr(), _ld(dyqT), dysc.data_ptr(), _ld(dysc), xqT.data_ptr(), _ld(xqT),
                              xsc.data_ptr(), _ld(xsc), dw_acc.data_ptr(), _ld(dw_acc), M, N, K, ptr, nbytes,
                              _stream(stream))
    return dw_acc


def uaq_fold_(w: torch.Tensor, s: torch.Tensor, prev: torch.Tensor | None = None, stream=None):
    """In-place UAQ fold: w[:, k] /= s[k], prev[:, k] *= s[k] (bf16, fp32 math)."""
    N, K = w.shape
    R = prev.shape[0] if prev is not None else 0
    rlq_uaq_fold(w.data_ptr(), N, K, _ld(w), s.data_ptr(), _ptr(prev), R, _ld(prev) if prev is not None else 0,
                 _stream(stream))
    return w, prev


def quant_nvfp4(w: torch.Tensor, stream=None):
    """NVFP4 quantization of bf16 w [N, K] (K % 16 == 0).

    Returns (q [N, K/2] u8 packed E2M1 codes, low nibble first; sb [N, K/16] u8
    E4M3 block-scale codes; st [1] f32 tensor scale)."""
    if w.dtype != torch.bfloat16:
        raise TypeError("w must be bfloat16")
    N, K = w.shape
    dev = w.device
    # pitches rounded to 16 bytes: the layout gemm_nvfp4_weight_only reads by TMA
    kq = _round_up(max(K // 2, 1), 16)
    ks = _round_up(max(K // 16, 1), 16)
    q = torch.empty((N, kq), dtype=torch.uint8, device=dev)[:, :K // 2]
    sb = torch.empty((N, ks), dtype=torch.uint8, device=dev)[:, :K // 16]
    st = torch.empty((1,), dtype=torch.float32, device=dev)
    rlq_quant_nvfp4(w.data_ptr(), N, K, _ld(w), q.data_ptr(), kq, sb.data_ptr(), ks, st.data_ptr(), _stream(stream))
    return q, sb, st


def gemm_nvfp4_weight_only(x: torch.Tensor, q, sb, st, out=None, stream=None, split_k: bool = False,
                           workspace=None):
    """Y [M, N] bf16 = X W^T with bf16 X [M, K] and NVFP4 weights (the outputs of
    ``quant_nvfp4``: q [N, K/2] packed E2M1, sb [N, K/16] E4M3, st [1] f32).

    ``split_k`` runs the split-K form with ``workspace`` (a uint8 device tensor)
    or a workspace allocated here for the library's plan."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    M, K = x.shape
    N = q.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    args = (x.data_ptr(), _ld(x), q.data_ptr(), q.stride(0), sb.data_ptr(), sb.stride(0), st.data_ptr(),
            y.data_ptr(), _ld(y), M, N, K)
    if split_k:
        ws = _workspace(GEMM_NVFP4_WEIGHT_ONLY, M, N, K, workspace, x.device, stream)
        rlq_gemm_nvfp4_weight_only_splitk(*args, *ws, _stream(stream))
    else:
        rlq_gemm_nvfp4_weight_only(*args, _stream(stream))
    return y


def aqn_perturb_(gamma: torch.Tensor, z: torch.Tensor, sigma: float, stream=None):
    """In-place AQN: gamma[k] = bf16(gamma[k] + sigma * z[k]) for a bf16 norm scale
    gamma [K] and one standard-normal draw per channel z [K] (f32)."""
    if gamma.dtype != torch.bfloat16 or z.dtype != torch.float32 or gamma.dim() != 1 or z.shape != gamma.shape:
        raise TypeError("gamma must be 1-D bfloat16 and z float32 of the same length")
    if not (gamma.is_contiguous() and z.is_contiguous()):
        raise ValueError("gamma and z must be contiguous")
    rlq_aqn_perturb(gamma.data_ptr(), gamma.numel(), z.data_ptr(), sigma, _stream(stream))
    return gamma


def _rows_of(name, t, M, K, dtype=torch.bfloat16):
    """Row pitch of ``t``, a [M, K] CUDA tensor of ``dtype`` with contiguous rows; an error
    that names it otherwise."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != (M, K):
        raise ValueError(f"{name} must be a [{M}, {K}] tensor")
    ld, inner = t.stride()
    if inner != 1 and K > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return ld if M > 1 else max(ld, K)


def _codes_T(K: int, M: int, device):
    """(transposed codes [K, M], their pitch), the pitch a multiple of 16 as the GEMMs' copies take it."""
    ld = (max(M, 1) + 15) & ~15
    return torch.empty_strided((K, M), (ld, 1), dtype=torch.uint8, device=device), ld


def _vector(name, t, n, dtype=torch.float32):
    """Address of ``t``, a contiguous [n] CUDA tensor of ``dtype``."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.data_ptr()


def add_rmsnorm_quant_act_1x128(res: torch.Tensor, delta: torch.Tensor | None, gamma: torch.Tensor, eps: float,
                                colwise: bool = False, inplace: bool = False, stream=None):
    """h = bf16(res + delta), then RMSNorm with the bf16 weight gamma [K], quantized
    1x128 (and with ``colwise`` 128x1) from fp32.  ``inplace`` writes h over res;
    without ``delta``, h is res itself.

    Returns (h [M, K] bf16, q, s, qT, sc) with q .. sc as ``quant_act_1x128``, and rstd [M] f32."""
    if res.dim() != 2:
        raise ValueError("res must be a [M, K] tensor")
    M, K = res.shape
    ldr = _rows_of("res", res, M, K)
    ldd = _rows_of("delta", delta, M, K) if delta is not None else 0
    g = _vector("gamma", gamma, K, torch.bfloat16)
    dev = res.device
    h = res if delta is None or inplace else torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    q = torch.empty((M, K), dtype=torch.uint8, device=dev)
    s = torch.empty((K // GRP, M), dtype=torch.float32, device=dev)
    rstd = torch.empty((M,), dtype=torch.float32, device=dev)
    qT = sc = None
    ldT = 0
    if colwise:
        qT, ldT = _codes_T(K, M, dev)
        sc = torch.empty(((M + GRP - 1) // GRP, K), dtype=torch.float32, device=dev)
    _call("rlq_add_rmsnorm_quant_act_1x128", res.data_ptr(), ldr, _ptr(delta), ldd, M, K, g, eps,
          h.data_ptr() if delta is not None else None, ldr if h is res else K, rstd.data_ptr(), q.data_ptr(), K,
          s.data_ptr(), max(M, 1), _ptr(qT), ldT, _ptr(sc), K if colwise else 0, _stream(stream))
    return h, q, s, qT, sc, rstd


def rmsnorm_backward(dx: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                     dres: torch.Tensor | None = None, inplace: bool = False, workspace=None, stream=None):
    """Gradient of the residual norm: dh = dres + d rmsnorm(h) * gamma / dh . dx (bf16) and
    the norm weight's gradient (fp32 [K]).  ``inplace`` writes dh over dres; without
    ``dres`` dh is a new tensor either way.

    Returns (dh [M, K] bf16, dgamma [K] f32)."""
    if dx.dim() != 2:
        raise ValueError("dx must be a [M, K] tensor")
    M, K = dx.shape
    lddx, ldh = _rows_of("dx", dx, M, K), _rows_of("h", h, M, K)
    ldres = _rows_of("dres", dres, M, K) if dres is not None else 0
    g, r = _vector("gamma", gamma, K, torch.bfloat16), _vector("rstd", rstd, M)
    dh = dres if inplace and dres is not None else torch.empty((M, K), dtype=torch.bfloat16, device=dx.device)
    dgamma = torch.empty((K,), dtype=torch.float32, device=dx.device)
    if workspace is None:
        nbytes = _norm_workspace_bytes(M, K, torch._C._cuda_getDevice())
        if nbytes:
            workspace = _scratch(nbytes, dx.device, stream)
    else:
        nbytes = _given(workspace)[1]
    _call("rlq_rmsnorm_backward", dx.data_ptr(), lddx, h.data_ptr(), ldh, r, g, _ptr(dres), ldres, dh.data_ptr(),
          ldres if dh is dres else K, dgamma.data_ptr(), M, K, _ptr(workspace), nbytes, _stream(stream))
    return dh, dgamma


@functools.lru_cache(maxsize=1024)
def _norm_workspace_bytes(M: int, K: int, device: int) -> int:
    """The library's workspace size for a shape on a device (its plan depends on nothing else)."""
    return rlq_rmsnorm_backward_workspace_bytes(M, K)


def gemm_gated_fprop(xq, xs, wq, ws, checkpoint: bool = False, stream=None):
    """Gated feed-forward block: a = silu(X Wg^T) * (X Wu^T) from 1x128 X codes and the
    stacked 128x128 codes [2F, K] of the gate and the up projection, gate first.

    Returns (aq [M, F] u8, as [F/128, M] f32, guq, gus): a's 1x128 codes and scales and,
    with ``checkpoint``, those of the two projections [M, 2F] (else None)."""
    if xq.dim() != 2:
        raise ValueError("xq must be a [M, K] tensor")
    M, K = xq.shape
    F = wq.shape[0] // 2
    ldx, ldw = _rows_of("xq", xq, M, K, torch.uint8), _rows_of("wq", wq, 2 * F, K, torch.uint8)
    ldxs = _rows_of("xs", xs, K // GRP, M, torch.float32)
    ldws = _rows_of("ws", ws, 2 * F // GRP, K // GRP, torch.float32)
    dev = xq.device
    aq = torch.empty((M, F), dtype=torch.uint8, device=dev)
    a_s = torch.empty((F // GRP, M), dtype=torch.float32, device=dev)
    guq = gus = None
    if checkpoint:
        guq = torch.empty((M, 2 * F), dtype=torch.uint8, device=dev)
        gus = torch.empty((2 * F // GRP, M), dtype=torch.float32, device=dev)
    _call("rlq_gemm_gated_fprop", xq.data_ptr(), ldx, xs.data_ptr(), max(ldxs, 1), wq.data_ptr(), ldw, ws.data_ptr(),
          ldws, aq.data_ptr(), F, a_s.data_ptr(), max(M, 1), _ptr(guq), 2 * F, _ptr(gus), max(M, 1), M, F, K,
          _stream(stream))
    return aq, a_s, guq, gus


def gated_backward(da: torch.Tensor, guq, gus, stream=None):
    """Gradient of the gated block's activation from its 8-bit checkpoint.

    Returns (q [M, 2F], s, qT [2F, M], sc) of [dg | du], as ``quant_act_1x128`` with
    ``colwise``, and (aT [F, M], ac) the 128x1 codes and scales of a."""
    if da.dim() != 2:
        raise ValueError("da must be a [M, F] tensor")
    M, F = da.shape
    ldda, ldgu = _rows_of("da", da, M, F), _rows_of("guq", guq, M, 2 * F, torch.uint8)
    ldgs = _rows_of("gus", gus, 2 * F // GRP, M, torch.float32)
    dev = da.device
    nb = (M + GRP - 1) // GRP
    q = torch.empty((M, 2 * F), dtype=torch.uint8, device=dev)
    s = torch.empty((2 * F // GRP, M), dtype=torch.float32, device=dev)
    (qT, ldT), (aT, _) = _codes_T(2 * F, M, dev), _codes_T(F, M, dev)
    sc = torch.empty((nb, 2 * F), dtype=torch.float32, device=dev)
    ac = torch.empty((nb, F), dtype=torch.float32, device=dev)
    _call("rlq_gated_backward", da.data_ptr(), ldda, guq.data_ptr(), ldgu, gus.data_ptr(), ldgs, q.data_ptr(), 2 * F,
          s.data_ptr(), max(M, 1), qT.data_ptr(), ldT, sc.data_ptr(), 2 * F, aT.data_ptr(), ldT, ac.data_ptr(), F, M, F,
          _stream(stream))
    return q, s, qT, sc, aT, ac


def _current(t):
    """The current CUDA device's number (no tensor's number where there is none)."""
    return torch._C._cuda_getDevice() if t.is_cuda else -2


def _here(name, t):
    """Refuses a tensor of another device than the current one, on whose streams calls run."""
    if t.get_device() != _current(t):
        raise ValueError(f"{name} must be on the current CUDA device")


def _mx_operand(name, q, s):
    """(rows, bytes a row, pitch) of packed MXFP4 codes with their scale tiles; an error that names
    what is wrong with them otherwise."""
    if q.dim() != 2:
        raise ValueError(f"{name}: codes must be a 2-D tensor")
    R, B = q.shape
    ld = _rows_of(name, q, R, B, torch.uint8)
    _here(name, q)
    if s.dtype is not torch.uint8:
        raise TypeError(f"{name}: scales must be uint8")
    if s.shape != mxfp4_scales_shape(R, 2 * B) or not s.is_contiguous():
        raise ValueError(f"{name}: scales must be a contiguous {mxfp4_scales_shape(R, 2 * B)} tensor")
    if s.device != q.device:
        raise ValueError(f"{name}: scales must be on the codes' device")
    return R, B, ld


def mxfp4_scales_shape(rows: int, cols: int):
    """Shape of the uint8 scale tiles of an MXFP4 matrix [rows, cols]: the byte of row r, block b
    (columns 32 b .. 32 b + 31) is ``s[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]``."""
    return (rows + 127) // 128, (cols + 127) // 128, 32, 4, 4


def quant_mxfp4(x: torch.Tensor, colwise: bool = False, stream=None):
    """MXFP4 quantization of bf16 x [M, K] (K % 32 == 0): E2M1 codes, two a byte, and a
    power-of-two scale per 32 elements along K; with ``colwise`` also of x transposed, per
    32 rows of x, from the same read.

    Returns (q [M, K/2] u8, s, qT [K, ceil(M/2)] u8 or None, sT or None), s and sT in tiles
    (``mxfp4_scales_shape``)."""
    if x.dim() != 2:
        raise ValueError("x must be a [M, K] tensor")
    M, K = x.shape
    ldx, inner = x.stride()
    d = x.get_device()
    if x.dtype is not torch.bfloat16 or (inner != 1 and K > 1) or d != _current(x):
        _rows_of("x", x, M, K)  # says which of it
        _here("x", x)
    if M <= 1 and ldx < K:
        ldx = K
    dev = x.device
    # (K / 2 is a multiple of 16, but for a K that the call refuses)
    q = torch.empty((M, K >> 1), dtype=torch.uint8, device=dev)
    s = torch.empty(((M + 127) >> 7, (K + 127) >> 7, 32, 4, 4), dtype=torch.uint8, device=dev)
    if not colwise:
        _call("rlq_quant_mxfp4", x.data_ptr(), M, K, ldx, q.data_ptr(), K >> 1, s.data_ptr(), None, 0, None,
              _stream(stream) if stream is not None else torch._C._cuda_getCurrentRawStream(d))
        return q, s, None, None
    qT, ldT = _codes_T(K, (M + 1) // 2, dev)
    sT = torch.empty(mxfp4_scales_shape(K, M), dtype=torch.uint8, device=dev)
    _call("rlq_quant_mxfp4", x.data_ptr(), M, K, ldx, q.data_ptr(), K >> 1, s.data_ptr(), qT.data_ptr(), ldT,
          sT.data_ptr(), _stream(stream))
    return q, s, qT, sT


def dequant_mxfp4(q: torch.Tensor, s: torch.Tensor, cols: int | None = None, stream=None):
    """The values (bf16 [rows, cols], exact) of MXFP4 codes and scale tiles.  ``cols`` is needed
    where it is odd; rows are on 16-byte boundaries, so the result is a view of longer rows
    where cols is not a multiple of 8."""
    R, B, ld = _mx_operand("q", q, s)
    C = 2 * B if cols is None else int(cols)
    if (C + 1) // 2 != B:
        raise ValueError(f"cols must be {2 * B} or {2 * B - 1}")
    ldx = (C + 7) & ~7
    x = torch.empty_strided((R, C), (ldx, 1), dtype=torch.bfloat16, device=q.device)
    _call("rlq_dequant_mxfp4", q.data_ptr(), ld, s.data_ptr(), R, C, x.data_ptr(), ldx, _stream(stream))
    return x


def gemm_mxfp4(xq, xs, wq, ws, out=None, out_dtype: torch.dtype = torch.bfloat16, stream=None):
    """Y [M, N] = X W^T from two MXFP4 operands (codes [M, K/2] and [N, K/2], scale tiles) on
    the FP4 tensor cores, in bf16 or fp32 (``out_dtype``, or that of ``out``).  DGrad takes
    the weight's transposed codes, WGrad those of dY and X."""
    u8, d = torch.uint8, xq.get_device()
    # (one condition for a pass, the checks one by one for what is wrong)
    if (xq.dtype is u8 and xs.dtype is u8 and wq.dtype is u8 and ws.dtype is u8 and xq.dim() == 2 and wq.dim() == 2 and
            d == _current(xq) and d == xs.get_device() == wq.get_device() == ws.get_device() and xs.is_contiguous() and
            ws.is_contiguous()):
        M, B = xq.shape
        N, Bw = wq.shape
        ldx, ix = xq.stride()
        ldw, iw = wq.stride()
        tiles = (B + 63) >> 6
        fine = (ix == 1 == iw and B == Bw and xs.shape == ((M + 127) >> 7, tiles, 32, 4, 4) and
                ws.shape == ((N + 127) >> 7, tiles, 32, 4, 4))
        # (the stride of a dimension of size 1 is arbitrary)
        ldx, ldw = ldx if M > 1 else max(ldx, B), ldw if N > 1 else max(ldw, B)
    else:
        fine = False
    if not fine:
        M, B, ldx = _mx_operand("xq", xq, xs)
        N, Bw, ldw = _mx_operand("wq", wq, ws)
        if B != Bw:
            raise ValueError(f"xq and wq have rows of {B} and {Bw} bytes: the contraction lengths differ")
        if wq.device != xq.device:
            raise ValueError("wq must be on xq's device")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=xq.device)
        ldy = N or 1
    else:
        out_dtype = out.dtype
        ldy = _rows_of("out", out, M, N, out_dtype)
        _here("out", out)
    dt = DTYPE_BF16 if out_dtype is torch.bfloat16 else DTYPE_F32 if out_dtype is torch.float32 else None
    if dt is None:
        raise TypeError("the output must be bfloat16 or float32")
    _call("rlq_gemm_mxfp4", xq.data_ptr(), ldx, xs.data_ptr(), wq.data_ptr(), ldw, ws.data_ptr(), out.data_ptr(), dt,
          ldy, M, N, 2 * B, _stream(stream) if stream is not None else torch._C._cuda_getCurrentRawStream(d))
    return out


def _logits(logits, targets):
    """(rows, V, dtype code, pitch, targets' address) of the logits."""
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("logits must be bfloat16 or float32")
    if logits.dim() != 2:
        raise ValueError("logits must be a [rows, V] tensor")
    T, V = logits.shape
    ld = _rows_of("logits", logits, T, V, logits.dtype)
    return T, V, (DTYPE_BF16 if logits.dtype is torch.bfloat16 else DTYPE_F32), ld, _vector("targets", targets, T,
                                                                                         torch.int64)


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, temperature: float = 1.0, stream=None):
    """Log probabilities (fp32 [rows]) of the int64 ``targets`` under bf16 or fp32
    ``logits`` [rows, V] divided by ``temperature``, and each row's log-sum-exp."""
    T, V, dt, ld, tg = _logits(logits, targets)
    lp = torch.empty((T,), dtype=torch.float32, device=logits.device)
    lse = torch.empty((T,), dtype=torch.float32, device=logits.device)
    _call("rlq_token_logprobs", logits.data_ptr(), dt, ld, T, V, tg, temperature, lp.data_ptr(), lse.data_ptr(),
          _stream(stream))
    return lp, lse


def token_logprobs_top(logits: torch.Tensor, targets: torch.Tensor, top: int = 0, temperature: float = 1.0, stream=None):
    """Log probabilities of the int64 ``targets`` under bf16 or fp32 ``logits`` [rows, V]
    divided by ``temperature``, each row's log-sum-exp and entropy, and the ``top`` (at most
    64, or V) most likely tokens with their log probabilities, among equal logits the lowest
    token first.  Masks should be -inf: where numbers such as -1e9 leave a row fewer tokens than
    ``top``, it takes many times as long.

    Returns (lp [rows] f32, lse [rows] f32, entropy [rows] f32, ids [rows, top] int64,
    top_lp [rows, top] f32)."""
    T, V, dt, ld, tg = _logits(logits, targets)
    _here("logits", logits)
    top = min(top, V)
    dev = logits.device
    lp = torch.empty((T,), dtype=torch.float32, device=dev)
    lse = torch.empty((T,), dtype=torch.float32, device=dev)
    H = torch.empty((T,), dtype=torch.float32, device=dev)
    ids = torch.empty((T, max(top, 0)), dtype=torch.int64, device=dev)
    top_lp = torch.empty((T, max(top, 0)), dtype=torch.float32, device=dev)
    _call("rlq_token_logprobs_top", logits.data_ptr(), dt, ld, T, V, tg, temperature, top, lp.data_ptr(), lse.data_ptr(),
          H.data_ptr(), ids.data_ptr(), top_lp.data_ptr(), _stream(stream))
    return lp, lse, H, ids, top_lp


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor, entropy=None, dlp=None,
                            dentropy=None, temperature: float = 1.0, inplace: bool = False, stream=None):
    """Gradient with respect to the logits of a loss whose derivatives by the targets' log
    probabilities and by the entropies are ``dlp`` and ``dentropy`` (fp32 [rows], one of them
    may be None), from the forward call's ``lse`` and, with ``dentropy``, ``entropy``.
    ``inplace`` writes it over the logits.  Returns dlogits, of the logits' shape and type."""
    T, V, dt, ld, tg = _logits(logits, targets)
    _here("logits", logits)
    opt = lambda name, t: None if t is None else _vector(name, t, T)  # noqa: E731
    args = _vector("lse", lse, T), opt("entropy", entropy), opt("dlp", dlp), opt("dentropy", dentropy)
    if inplace:
        d, ldd = logits, ld
    else:
        # (the least pitch whose rows share the logits' 16-byte phases: a part of wide rows gets no wide rows)
        ldd = V + (ld - V) % (4 if dt == DTYPE_F32 else 8)
        d = torch.empty_strided((T, V), (ldd, 1), dtype=logits.dtype, device=logits.device)
    _call("rlq_token_logprobs_backward", logits.data_ptr(), dt, ld, T, V, tg, temperature, *args, d.data_ptr(), ldd,
          _stream(stream))
    return d


def policy_loss(logits: torch.Tensor, targets: torch.Tensor, logp_old: torch.Tensor, adv: torch.Tensor,
                weight: torch.Tensor, logp_behav=None, logp_ref=None, clip_hi=None, eps_lo: float = 0.2,
                eps_hi: float = 0.2, tis_cap: float = 2.0, kl_beta: float = 0.0, temperature: float = 1.0,
                grad: bool = True, inplace: bool = False, stream=None):
    """Clipped policy loss with a truncated importance weight and a KL term (see
    rlq_policy_loss in include/rlq.h): per-row losses whose sum is the batch's loss,
    and the gradient of that sum with respect to the logits.  ``inplace`` writes the
    gradient over the logits.

    Returns (loss [rows] f32, logp [rows] f32, dlogits like logits or None)."""
    T, V, dt, ld, tg = _logits(logits, targets)
    opt = lambda name, t: None if t is None else _vector(name, t, T)  # noqa: E731
    loss = torch.empty((T,), dtype=torch.float32, device=logits.device)
    lp = torch.empty((T,), dtype=torch.float32, device=logits.device)
    d = None
    if grad and inplace:
        d = logits
    elif grad:
        # the logits' own pitch, so that their rows share 16-byte phases
        d = torch.empty_strided((T, V), (ld, 1), dtype=logits.dtype, device=logits.device)
    _call("rlq_policy_loss", logits.data_ptr(), dt, ld, T, V, tg, temperature, _vector("logp_old", logp_old, T),
          _vector("adv", adv, T), _vector("weight", weight, T), opt("logp_behav", logp_behav),
          opt("logp_ref", logp_ref), opt("clip_hi", clip_hi), eps_lo, eps_hi, tis_cap, kl_beta, loss.data_ptr(),
          lp.data_ptr(), _ptr(d), ld if grad else 0, _stream(stream))
    return loss, lp, d


def check(stream=None):
    """Synchronise the stream and raise RlqError on a recorded device-side timeout."""
    return rlq_check(_stream(stream))
