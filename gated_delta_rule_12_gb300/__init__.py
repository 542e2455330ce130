"""GB300 (sm_103a) gated delta rule: Python binding of libgdn.so.

This module only marshals arguments: it checks tensor placement, dtype and
contiguity, allocates outputs/workspace with PyTorch when the caller does not
pass them, and calls the C ABI declared in ``include/gdn.h`` through ctypes on
the current PyTorch CUDA stream.  Every step of the computation runs in the
library's CUDA kernels; there is no other code path.  If ``libgdn.so`` cannot
be loaded the calls raise: there is no fallback.

Every call enqueues on the current stream, or on ``stream=`` where that is given (a torch stream or
a raw handle).  The caller then orders the inputs before the call and the use of its results behind it.

Entry points (same names as the C ABI, without the ``gdn_`` prefix):
    chunk_fwd(q, k, v, g, beta, ...)      -> (out, final_state)
    decode_step(state, q, k, v, g, beta)  -> out            (state updated in place)
    decode_multi(state, q, k, v, g, beta) -> out [N,T,H,dv] (T tokens per call, state in place)
    prologue(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, ...) -> (q, k, v, g, beta)
    prologue_chunk_fwd(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, ...) -> (out, final_state)
                                          (prologue fused into the chunked forward)
    chunk_fwd_workspace_size(...)         -> bytes
    chunk_fwd_kernel_count(...)           -> kernels one chunk_fwd call launches
    chunk_bwd(q, k, v, g, beta, dout, ...) -> (dq, dk, dv, dg, dbeta, dinit_state)
    gated_scan_fwd(x, g, ...)             -> (out, final_state)   per-channel gated linear recurrence
    gated_scan_bwd(x, g, out, dout, ...)  -> (dx, dg, dinit_state)
    gated_scan_step(state, x, g)          -> out            (state updated in place)
    layer_norm_fwd(x, weight, bias, eps)  -> (out, mean, rstd)
    layer_norm_bwd(dout, x, mean, rstd, weight) -> (dx, dweight, dbias)
    linear_cross_entropy_fwd(h, weight, targets) -> (loss, lse)   no logits array
    linear_cross_entropy_bwd(h, weight, targets, lse, dloss) -> (dh, dweight)
    check_device_error(workspace)         -> None or raises
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libgdn.so")

GDN_OK = 0
STATUS = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED", 3: "GDN_ERR_WORKSPACE",
          4: "GDN_ERR_CUDA", 5: "GDN_ERR_DEVICE_TIMEOUT", 6: "GDN_ERR_RANGE"}
GDN_F32, GDN_BF16 = 0, 1
CHUNK = 64

EXPORTS = ["gdn_status_string", "gdn_chunk_fwd_workspace_size", "gdn_chunk_fwd_kernel_count", "gdn_chunk_fwd",
           "gdn_chunk_bwd_workspace_size", "gdn_chunk_bwd", "gdn_decode_step", "gdn_decode_multi", "gdn_prologue",
           "gdn_check_device_error", "gdn_chunk_fwd_noalloc", "gdn_prologue_chunk_fwd_workspace_size",
           "gdn_prologue_chunk_fwd", "gdn_gated_scan_fwd", "gdn_gated_scan_bwd", "gdn_gated_scan_step",
           "gdn_layer_norm_fwd", "gdn_layer_norm_bwd_workspace_size", "gdn_layer_norm_bwd",
           "gdn_linear_cross_entropy_workspace_size", "gdn_linear_cross_entropy_fwd",
           "gdn_linear_cross_entropy_bwd"]
NOALLOC_SCRATCH_BYTES = 32 << 20


class GDNError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what} failed: {STATUS.get(code, code)}")


_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_sz = ctypes.c_size_t


def load_library(path: str = LIB_PATH, build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libgdn.so (optionally building it first) and declare the ABI."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            if build_if_missing:
                from . import build as _b
                path = _b.build()
            else:
                raise RuntimeError(f"libgdn.so not found at {path}; run gated_delta_rule_12_gb300.build.build()")
        lib = ctypes.CDLL(path)
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_chunk_fwd_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]
        lib.gdn_chunk_fwd_workspace_size.restype = _sz
        lib.gdn_chunk_fwd_kernel_count.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]
        lib.gdn_chunk_fwd_kernel_count.restype = _i32
        lib.gdn_chunk_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                      _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _f32, _i32, _i32,
                                      _vp, _sz, _vp]
        lib.gdn_chunk_fwd.restype = ctypes.c_int
        lib.gdn_chunk_bwd_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]
        lib.gdn_chunk_bwd_workspace_size.restype = _sz
        lib.gdn_chunk_bwd.argtypes = [_vp] * 6 + [_vp, _i32] + [_vp] * 8 + [_i32] * 5 + [ctypes.c_int, _f32, _i32, _i32,
                                                                                         _vp, _sz, _vp]
        lib.gdn_chunk_bwd.restype = ctypes.c_int
        lib.gdn_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                        _i32, _i32, _i32, _i32, ctypes.c_int, _f32, _i32, _vp]
        lib.gdn_decode_step.restype = ctypes.c_int
        lib.gdn_decode_multi.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _f32, _i32, _vp]
        lib.gdn_decode_multi.restype = ctypes.c_int
        lib.gdn_prologue.argtypes = [_vp] * 12 + [_vp, _i32] + [_vp] * 5 + [_i32] * 6 + [ctypes.c_int, _vp]
        lib.gdn_prologue.restype = ctypes.c_int
        lib.gdn_check_device_error.argtypes = [_vp, _vp]
        lib.gdn_check_device_error.restype = ctypes.c_int
        lib.gdn_selftest_wait_timeout.argtypes = [_vp, ctypes.c_uint32, _vp]
        lib.gdn_selftest_wait_timeout.restype = ctypes.c_int
        lib.gdn_chunk_fwd_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                                              _i32, _i32, _i32, _i32, _i32, ctypes.c_int, _f32, _i32, _i32,
                                              _vp]
        lib.gdn_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.gdn_prologue_chunk_fwd_workspace_size.argtypes = [_i32, _i32, _i32, _i32, _i32, _i32, ctypes.c_int]
        lib.gdn_prologue_chunk_fwd_workspace_size.restype = _sz
        lib.gdn_prologue_chunk_fwd.argtypes = [_vp] * 13 + [_vp, _i32, _vp, _vp] + [_i32] * 6 + \
            [ctypes.c_int, _f32, _i32, _i32, _vp, _sz, _vp]
        lib.gdn_prologue_chunk_fwd.restype = ctypes.c_int
        _ci = ctypes.c_int
        lib.gdn_gated_scan_fwd.argtypes = [_vp] * 4 + [_i32, _vp, _vp] + [_i32] * 3 + [_ci, _i32, _vp]
        lib.gdn_gated_scan_bwd.argtypes = [_vp] * 7 + [_i32] + [_vp] * 3 + [_i32] * 3 + [_ci, _i32, _vp]
        lib.gdn_gated_scan_step.argtypes = [_vp] * 4 + [_i32] * 2 + [_ci, _i32, _vp]
        lib.gdn_layer_norm_fwd.argtypes = [_vp] * 6 + [ctypes.c_int64, _i32, _ci, _f32, _vp]
        lib.gdn_layer_norm_bwd_workspace_size.argtypes = [ctypes.c_int64, _i32, _ci]
        lib.gdn_layer_norm_bwd_workspace_size.restype = _sz
        lib.gdn_layer_norm_bwd.argtypes = [_vp] * 8 + [ctypes.c_int64, _i32, _ci, _vp, _sz, _vp]
        lib.gdn_linear_cross_entropy_workspace_size.argtypes = [_i32] * 3 + [_ci, _i32]
        lib.gdn_linear_cross_entropy_workspace_size.restype = _sz
        lib.gdn_linear_cross_entropy_fwd.argtypes = [_vp] * 5 + [_i32] * 3 + [_ci, _vp, _sz, _vp]
        lib.gdn_linear_cross_entropy_bwd.argtypes = [_vp] * 7 + [_i32] * 3 + [_ci, _vp, _sz, _vp]
        lib.gdn_selftest_linear_cross_entropy_timeout.argtypes = [_i32, ctypes.c_uint32] + [_vp] * 7 + [_i32] * 3 + \
            [_vp, _sz, _vp]
        lib.gdn_selftest_linear_cross_entropy_timeout.restype = _ci
        for name in ("gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "layer_norm_fwd", "layer_norm_bwd",
                     "linear_cross_entropy_fwd", "linear_cross_entropy_bwd"):
            getattr(lib, "gdn_" + name).restype = _ci
        _lib = lib
        return lib


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return GDN_F32
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _elsewhere(stream, call, *args):
    """``call(*args)`` on the stream that the caller names, a torch stream or a raw handle.

    It is the current one meanwhile, so outputs and workspaces come from memory that this stream has done with: memory of
    the caller's current stream may still be in use by work queued there.  What the call made is used on the caller's
    stream next; the allocator keeps it until that use is over too."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        got = call(*args)
    given = {id(t) for a in args for t in (a if isinstance(a, (tuple, list)) else (a,))}
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None and id(t) not in given:
            t.record_stream(here)
    return got


def _check_chunk_args(q, k, v, g, beta, init_state, cu_seqlens, out, final_state):
    """The checks every chunked-forward wrapper makes before it hands raw pointers to the C ABI:
    dtypes (the kernels read cu_seqlens as int32 and g, beta and the states as fp32, so any other
    dtype would be misread on the device), shapes, placement and contiguity."""
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:3] != q.shape[:3]:
        raise ValueError("q, k must be [B,T,H,dk] and v [B,T,H,dv]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must share one dtype")
    _dt(q)
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32:
            raise TypeError("cu_seqlens must be int32")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N+1] with N >= 1")
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    for t, what in ((g, "g"), (beta, "beta")):
        if t.dtype != torch.float32:
            raise TypeError(f"{what} must be float32")
        if tuple(t.shape) != (B, T, H):
            raise ValueError(f"{what} must be [B,T,H]")
    for t, what in ((init_state, "init_state"), (final_state, "final_state")):
        if t is None:
            continue
        if t.dtype != torch.float32:
            raise TypeError(f"{what} must be float32")
        if tuple(t.shape) != (N, H, dv, dk):
            raise ValueError(f"{what} must be [N,H,dv,dk] = {(N, H, dv, dk)}")
    if out is not None:
        if out.dtype != q.dtype:
            raise TypeError("out must have the dtype of q")
        if tuple(out.shape) != (B, T, H, dv):
            raise ValueError(f"out must be [B,T,H,dv] = {(B, T, H, dv)}")
    _need_cuda(q, k, v, g, beta, init_state, cu_seqlens, out, final_state)

def chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs=0, dtype=torch.bfloat16) -> int:
    dt = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load_library().gdn_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, dt))


def chunk_fwd_kernel_count(B, T, H, dk, dv, num_seqs=0, dtype=torch.bfloat16) -> int:
    """Kernels one ``chunk_fwd`` call of this size launches (0 if unsupported)."""
    dt = GDN_BF16 if dtype == torch.bfloat16 else GDN_F32
    return int(load_library().gdn_chunk_fwd_kernel_count(B, T, H, dk, dv, num_seqs, dt))


def chunk_fwd(q, k, v, g, beta, init_state=None, cu_seqlens=None, scale=None, use_qk_l2norm=True,
              out=None, final_state=None, output_final_state=True, workspace=None, chunk_size=CHUNK,
              stream=None):
    """Chunked forward of the gated delta rule (see ``gdn_chunk_fwd`` in include/gdn.h).

    q, k [B,T,H,dk], v [B,T,H,dv] (fp32 or bf16); g, beta [B,T,H] fp32;
    init_state [N,H,dv,dk] fp32 or None; cu_seqlens int32 [N+1] (device) or None.
    Returns ``(out, final_state)``; final_state is None if not requested.
    """
    if stream is not None:
        return _elsewhere(stream, chunk_fwd, q, k, v, g, beta, init_state, cu_seqlens, scale, use_qk_l2norm,
                          out, final_state, output_final_state, workspace, chunk_size)
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device)
    _check_chunk_args(q, k, v, g, beta, init_state, cu_seqlens, out, final_state)
    dt = _dt(q)
    num_seqs = N if cu_seqlens is not None else 0
    need = int(lib.gdn_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, dt))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib.gdn_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state),
                           _ptr(cu_seqlens), num_seqs, _ptr(out), _ptr(final_state),
                           B, T, H, dk, dv, dt, float(scale), int(bool(use_qk_l2norm)), int(chunk_size),
                           _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_chunk_fwd")
    return out, final_state


def chunk_bwd(q, k, v, g, beta, dout, init_state=None, dfinal_state=None, cu_seqlens=None, scale=None,
              use_qk_l2norm=True, want_dinit=True, workspace=None, chunk_size=CHUNK, stream=None):
    """Backward of ``chunk_fwd`` (``gdn_chunk_bwd``): returns ``(dq, dk, dv, dg, dbeta, dinit_state)``
    for the loss gradients ``dout`` [B,T,H,dv] and ``dfinal_state`` [N,H,dv,dk] (or None)."""
    if stream is not None:
        return _elsewhere(stream, chunk_bwd, q, k, v, g, beta, dout, init_state, dfinal_state, cu_seqlens, scale,
                          use_qk_l2norm, want_dinit, workspace, chunk_size)
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    dq, dkk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    db = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    dinit = torch.empty((N, H, dv, dk), dtype=torch.float32, device=q.device) if want_dinit else None
    for t in (g, beta, init_state, dfinal_state):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("g, beta and states must be float32")
    if dout.dtype != q.dtype:
        raise TypeError("dout must have the dtype of q")
    _need_cuda(q, k, v, g, beta, dout, init_state, dfinal_state, cu_seqlens)
    dt = _dt(q)
    num_seqs = N if cu_seqlens is not None else 0
    need = int(lib.gdn_chunk_bwd_workspace_size(B, T, H, dk, dv, num_seqs, dt))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib.gdn_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state), _ptr(cu_seqlens),
                           num_seqs, _ptr(dout), _ptr(dfinal_state), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dg),
                           _ptr(db), _ptr(dinit), B, T, H, dk, dv, dt, float(scale), int(bool(use_qk_l2norm)),
                           int(chunk_size), _ptr(workspace), workspace.numel() * workspace.element_size(),
                           _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_chunk_bwd")
    return dq, dkk, dvv, dg, db, dinit


def decode_step(state, q, k, v, g, beta, scale=None, use_qk_l2norm=True, out=None, stream=None):
    """One decode token per (sequence, head); ``state`` [N,H,dv,dk] fp32 is updated in place.

    q, k [N,H,dk], v [N,H,dv] (fp32 or bf16); g, beta [N,H] fp32.  Returns out [N,H,dv].
    """
    if stream is not None:
        return _elsewhere(stream, decode_step, state, q, k, v, g, beta, scale, use_qk_l2norm, out)
    lib = load_library()
    N, H, dv, dk = state.shape
    if scale is None:
        scale = dk ** -0.5
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    if state.dtype != torch.float32 or g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("state, g and beta must be float32")
    _need_cuda(state, q, k, v, g, beta, out)
    rc = lib.gdn_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out),
                             N, H, dk, dv, _dt(q), float(scale), int(bool(use_qk_l2norm)), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_decode_step")
    return out


def decode_multi(state, q, k, v, g, beta, scale=None, use_qk_l2norm=True, out=None, stream=None):
    """T decode tokens per (sequence, head) in one call; ``state`` [N,H,dv,dk] fp32 is updated in place.

    q, k [N,T,H,dk], v [N,T,H,dv] (fp32 or bf16); g, beta [N,T,H] fp32.  Returns out [N,T,H,dv],
    the same as T successive ``decode_step`` calls.
    """
    if stream is not None:
        return _elsewhere(stream, decode_multi, state, q, k, v, g, beta, scale, use_qk_l2norm, out)
    lib = load_library()
    N, H, dv, dk = state.shape
    T = q.shape[1]
    if scale is None:
        scale = dk ** -0.5
    if out is None:
        out = torch.empty((N, T, H, dv), dtype=q.dtype, device=q.device)
    if state.dtype != torch.float32 or g.dtype != torch.float32 or beta.dtype != torch.float32:
        raise TypeError("state, g and beta must be float32")
    if q.shape != (N, T, H, dk) or k.shape != (N, T, H, dk) or v.shape != (N, T, H, dv) or g.shape != (N, T, H) \
            or beta.shape != (N, T, H) or out.shape != (N, T, H, dv):
        raise ValueError("decode_multi: inconsistent shapes")
    _need_cuda(state, q, k, v, g, beta, out)
    rc = lib.gdn_decode_multi(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(out),
                              N, T, H, dk, dv, _dt(q), float(scale), int(bool(use_qk_l2norm)), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_decode_multi")
    return out


def prologue(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in=None, conv_state_out=None,
             cu_seqlens=None, out=None, stream=None):
    """Block prologue (``gdn_prologue``): q, k, v = SiLU(short causal conv of the projections),
    g = -exp(A_log) softplus(a + dt_bias), beta = sigmoid(b), in one pass.

    xq, xk [B,T,H,dk], xv [B,T,H,dv] (fp32 or bf16); wq, wk [H,dk,K], wv [H,dv,K] fp32;
    a, b [B,T,H] fp32; A_log, dt_bias [H] fp32; conv states [N,K-1,H,2dk+dv] (dtype of x) or None.
    Returns ``(q, k, v, g, beta)``; ``out`` may pass those five tensors preallocated.
    """
    if stream is not None:
        return _elsewhere(stream, prologue, xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in,
                          conv_state_out, cu_seqlens, out)
    lib = load_library()
    B, T, H, dk = xq.shape
    dv = xv.shape[-1]
    K = wq.shape[-1]
    if out is None:
        out = (torch.empty_like(xq), torch.empty_like(xk), torch.empty_like(xv),
               torch.empty((B, T, H), dtype=torch.float32, device=xq.device),
               torch.empty((B, T, H), dtype=torch.float32, device=xq.device))
    q, k, v, g, beta = out
    for t in (wq, wk, wv, a, b, A_log, dt_bias, g, beta):
        if t.dtype != torch.float32:
            raise TypeError("filters, gate projections, gate parameters and g, beta must be float32")
    if wq.shape != (H, dk, K) or wk.shape != (H, dk, K) or wv.shape != (H, dv, K):
        raise ValueError("prologue: filters must be [H, d, K]")
    _need_cuda(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in, conv_state_out, cu_seqlens,
               q, k, v, g, beta)
    num_seqs = (cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    rc = lib.gdn_prologue(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(a), _ptr(b),
                          _ptr(A_log), _ptr(dt_bias), _ptr(conv_state_in), _ptr(conv_state_out),
                          _ptr(cu_seqlens), num_seqs, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                          B, T, H, dk, dv, K, _dt(xq), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_prologue")
    return q, k, v, g, beta


def prologue_chunk_fwd(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in=None, conv_state_out=None,
                       init_state=None, cu_seqlens=None, scale=None, use_qk_l2norm=True, out=None, final_state=None,
                       output_final_state=True, workspace=None, chunk_size=CHUNK, stream=None):
    """Block prologue and chunked forward in one call (``gdn_prologue_chunk_fwd``): the result of
    ``prologue`` followed by ``chunk_fwd``, without q, k, v, g, beta ever being written out.

    xq, xk [B,T,H,dk], xv [B,T,H,dv] bf16 (dk = 128, dv a multiple of 128); wq, wk [H,dk,K], wv [H,dv,K]
    fp32; a, b [B,T,H] fp32; A_log, dt_bias [H] fp32; conv states [N,K-1,H,2dk+dv] bf16 or None;
    init_state [N,H,dv,dk] fp32 or None; cu_seqlens int32 [N+1] or None.  Returns ``(out, final_state)``.
    """
    if stream is not None:
        return _elsewhere(stream, prologue_chunk_fwd, xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in,
                          conv_state_out, init_state, cu_seqlens, scale, use_qk_l2norm, out, final_state,
                          output_final_state, workspace, chunk_size)
    lib = load_library()
    B, T, H, dk = xq.shape
    dv = xv.shape[-1]
    K = wq.shape[-1]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    if xq.dtype != torch.bfloat16 or xk.dtype != torch.bfloat16 or xv.dtype != torch.bfloat16:
        raise TypeError("prologue_chunk_fwd: projections must be bfloat16")
    for t in (wq, wk, wv, a, b, A_log, dt_bias, init_state, final_state):
        if t is not None and t.dtype != torch.float32:
            raise TypeError("filters, gate projections, gate parameters and states must be float32")
    if wq.shape != (H, dk, K) or wk.shape != (H, dk, K) or wv.shape != (H, dv, K):
        raise ValueError("prologue_chunk_fwd: filters must be [H, d, K]")
    if a.shape != (B, T, H) or b.shape != (B, T, H) or A_log.shape != (H,) or dt_bias.shape != (H,):
        raise ValueError("prologue_chunk_fwd: gate shapes")
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    for t in (conv_state_in, conv_state_out):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != (N, K - 1, H, 2 * dk + dv)):
            raise ValueError("conv states must be bfloat16 [N, K-1, H, 2dk+dv]")
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=torch.bfloat16, device=xq.device)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dv, dk), dtype=torch.float32, device=xq.device)
    _need_cuda(xq, xk, xv, wq, wk, wv, a, b, A_log, dt_bias, conv_state_in, conv_state_out, init_state, cu_seqlens,
               out, final_state)
    num_seqs = N if cu_seqlens is not None else 0
    need = int(lib.gdn_prologue_chunk_fwd_workspace_size(B, T, H, dk, dv, num_seqs, GDN_BF16))
    if need == 0:
        raise GDNError(2, "gdn_prologue_chunk_fwd (unsupported size)")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=xq.device)
    rc = lib.gdn_prologue_chunk_fwd(_ptr(xq), _ptr(xk), _ptr(xv), _ptr(wq), _ptr(wk), _ptr(wv), _ptr(a), _ptr(b),
                                    _ptr(A_log), _ptr(dt_bias), _ptr(conv_state_in), _ptr(conv_state_out),
                                    _ptr(init_state), _ptr(cu_seqlens), num_seqs, _ptr(out), _ptr(final_state),
                                    B, T, H, dk, dv, K, GDN_BF16, float(scale), int(bool(use_qk_l2norm)),
                                    int(chunk_size), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_prologue_chunk_fwd")
    return out, final_state


# Calls of a few microseconds are held up by what surrounds them, so the wrappers below look torch's attributes up once
# and take the current stream as the raw handle (0.1 us; the stream object takes 3).
_F32, _BF16 = torch.float32, torch.bfloat16
_empty, _empty_like = torch.empty, torch.empty_like
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream_of(t):
    return _raw_stream(t.get_device())


_MOST = 2 ** 31 - 1   # what a size may be in the C ABI; ctypes would cut a larger one down to its low 32 bits


def _too_large(**sizes):
    raise ValueError("sizes go up to 2^31 - 1, not " + ", ".join(f"{k} = {v}" for k, v in sizes.items()))


def _check_scan_args(x, g, cu_seqlens, dtype, states, same):
    """Shapes, dtypes, placement and contiguity of a gated-scan call; returns (B, T, D, N).  ``states`` are the
    [N,D] fp32 tensors, ``same`` further tensors that must match g."""
    shape = g.shape
    if len(shape) != 3:
        raise ValueError("x and g must be [B,T,D]")
    B, T, D = shape
    if B > _MOST or T > _MOST or D > _MOST:
        _too_large(B=B, T=T, D=D)
    N = B
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int32:
            raise TypeError("cu_seqlens must be int32")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or B != 1:
            raise ValueError("cu_seqlens must be [N+1] with N >= 1, and B = 1")
        N = cu_seqlens.numel() - 1
    for t in (x, g, *same):
        if t is not None:
            if t.dtype is not dtype:
                raise TypeError("x, g and the other token tensors must share one dtype")
            if t.shape != shape:
                raise ValueError("x, g and the other token tensors must share one shape")
    for t in states:
        if t is not None:
            if t.dtype is not _F32:
                raise TypeError("states must be float32")
            if t.shape != (N, D):
                raise ValueError(f"states must be [N,D] = {(N, D)}")
    _need_cuda(x, g, cu_seqlens, *states, *same)
    return B, T, D, N


def gated_scan_fwd(x, g, init_state=None, cu_seqlens=None, input_gate=False, out=None, final_state=None,
                   output_final_state=True, stream=None):
    """Per-channel gated linear recurrence (``gdn_gated_scan_fwd``): h_t = a_t h_{t-1} + c_t x_t with a = exp(g)
    and c = 1, or 1 - a with ``input_gate``.

    x, g [B,T,D] (fp32 or bf16, one dtype); init_state [N,D] fp32 or None; cu_seqlens int32 [N+1] (device) or
    None.  Returns ``(out, final_state)``; final_state is None if not requested.  B may be 0.
    """
    if stream is not None:
        return _elsewhere(stream, gated_scan_fwd, x, g, init_state, cu_seqlens, input_gate, out, final_state,
                          output_final_state)
    lib = _lib or load_library()
    B, T, D, N = _check_scan_args(x, g, cu_seqlens, x.dtype, (init_state, final_state), (out,))
    dt = _dt(x)
    if out is None:
        out = _empty_like(x)
    if final_state is None and output_final_state:
        final_state = _empty((N, D), dtype=_F32, device=x.device)
    if B == 0:
        return out, final_state
    rc = lib.gdn_gated_scan_fwd(x.data_ptr(), g.data_ptr(), _ptr(init_state), _ptr(cu_seqlens),
                                N if cu_seqlens is not None else 0, out.data_ptr(), _ptr(final_state), B, T, D,
                                dt, int(bool(input_gate)), _stream_of(g))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_gated_scan_fwd")
    return out, final_state


def gated_scan_bwd(x, g, out, dout, init_state=None, dfinal_state=None, cu_seqlens=None, input_gate=False,
                   want_dinit=True, stream=None):
    """Backward of ``gated_scan_fwd`` (``gdn_gated_scan_bwd``): returns ``(dx, dg, dinit_state)`` for the loss
    gradients ``dout`` [B,T,D] and ``dfinal_state`` [N,D] (or None).  ``out`` is the forward's output; ``x`` may be
    None without ``input_gate``."""
    if stream is not None:
        return _elsewhere(stream, gated_scan_bwd, x, g, out, dout, init_state, dfinal_state, cu_seqlens, input_gate,
                          want_dinit)
    lib = _lib or load_library()
    if input_gate and x is None:
        raise ValueError("gated_scan_bwd: x is needed with the input gate")
    B, T, D, N = _check_scan_args(x, g, cu_seqlens, g.dtype, (init_state, dfinal_state), (out, dout))
    dt = _dt(g)
    dx, dg = _empty_like(g), _empty_like(g)
    dinit = _empty((N, D), dtype=_F32, device=g.device) if want_dinit else None
    if B == 0:
        return dx, dg, dinit
    rc = lib.gdn_gated_scan_bwd(_ptr(x), g.data_ptr(), out.data_ptr(), dout.data_ptr(), _ptr(init_state),
                                _ptr(dfinal_state), _ptr(cu_seqlens), N if cu_seqlens is not None else 0,
                                dx.data_ptr(), dg.data_ptr(), _ptr(dinit), B, T, D, dt, int(bool(input_gate)),
                                _stream_of(g))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_gated_scan_bwd")
    return dx, dg, dinit


def _sound(t, dtype):
    """What a kernel takes: the dtype, on the GPU, contiguous."""
    return t.dtype is dtype and t.is_cuda and t.is_contiguous()


def gated_scan_step(state, x, g, input_gate=False, out=None, stream=None):
    """One token of the gated scan per sequence (``gdn_gated_scan_step``); ``state`` [N,D] fp32 is updated in
    place.  x, g [N,D] (fp32 or bf16).  Returns out [N,D]."""
    if stream is not None:
        return _elsewhere(stream, gated_scan_step, state, x, g, input_gate, out)
    lib = _lib or load_library()
    shape, dtype = state.shape, x.dtype
    if len(shape) != 2 or x.shape != shape or g.shape != shape or (out is not None and out.shape != shape):
        raise ValueError("gated_scan_step: state, x, g and out must be [N,D]")
    N, D = shape
    if N > _MOST or D > _MOST:
        _too_large(N=N, D=D)
    if state.dtype is not _F32:
        raise TypeError("state must be float32")
    if g.dtype is not dtype or (out is not None and out.dtype is not dtype):
        raise TypeError("x, g and out must share one dtype")
    _need_cuda(state, x, g, out)
    if out is None:
        out = _empty_like(x)
    rc = lib.gdn_gated_scan_step(state.data_ptr(), x.data_ptr(), g.data_ptr(), out.data_ptr(), N, D, _dt(x),
                                 1 if input_gate else 0, _stream_of(x))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_gated_scan_step")
    return out


def _check_norm_args(x, params, stats, same):
    """Shapes, dtypes, placement and contiguity of a layer-norm call; returns (rows, D)."""
    shape = x.shape
    if not shape or shape[-1] < 1:
        raise ValueError("x must be [..., D] with D >= 1")
    D = shape[-1]
    if D > _MOST:
        _too_large(D=D)
    rows = x.numel() // D
    for t in params:
        if t is not None:
            if t.dtype is not _F32:
                raise TypeError("weight and bias must be float32")
            if t.shape != (D,):
                raise ValueError("weight and bias must be [D]")
    for t in stats:
        if t.dtype is not _F32:
            raise TypeError("mean and rstd must be float32")
        if t.numel() != rows:
            raise ValueError("mean and rstd must hold one value a row")
    for t in same:
        if t is not None:
            if t.dtype is not x.dtype:
                raise TypeError("x and the other row tensors must share one dtype")
            if t.shape != shape:
                raise ValueError("x and the other row tensors must share one shape")
    _need_cuda(x, *params, *stats, *same)
    return rows, D


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, out=None, stream=None):
    """Layer norm over the last axis (``gdn_layer_norm_fwd``).  x [..., D] (fp32 or bf16); weight, bias [D] fp32 or
    None.  Returns ``(out, mean, rstd)``, the statistics fp32 of shape ``x.shape[:-1]``."""
    if stream is not None:
        return _elsewhere(stream, layer_norm_fwd, x, weight, bias, eps, out)
    lib = _lib or load_library()
    # everything in order takes the short way; the long one says what is not
    shape = x.shape
    D = shape[-1] if shape else 0
    if 0 < D <= _MOST and out is None and x.is_cuda and x.is_contiguous() and \
            (weight is None or (_sound(weight, _F32) and weight.shape == (D,))) and \
            (bias is None or (_sound(bias, _F32) and bias.shape == (D,))):
        rows = x.numel() // D
    else:
        rows, D = _check_norm_args(x, (weight, bias), (), (out,))
    dt = _dt(x)
    if out is None:
        out = _empty_like(x)
    mean = _empty(shape[:-1], dtype=_F32, device=x.device)
    rstd = _empty_like(mean)
    rc = lib.gdn_layer_norm_fwd(x.data_ptr(), None if weight is None else weight.data_ptr(),
                                None if bias is None else bias.data_ptr(), out.data_ptr(), mean.data_ptr(),
                                rstd.data_ptr(), rows, D, dt, eps, _stream_of(x))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_layer_norm_fwd")
    return out, mean, rstd


def layer_norm_bwd_workspace_size(rows, D, dtype=torch.bfloat16) -> int:
    dt = GDN_BF16 if dtype == _BF16 else GDN_F32
    if D > _MOST:
        return 0
    return int(load_library().gdn_layer_norm_bwd_workspace_size(rows, D, dt))


def _workspace(given, need, device):
    """The caller's workspace and its size, or one of the size needed."""
    if given is None:
        need = max(256, need)
        return _empty(need, dtype=torch.uint8, device=device), need
    _need_cuda(given)
    return given, given.numel() * given.element_size()


def layer_norm_bwd(dout, x, mean, rstd, weight=None, workspace=None, stream=None):
    """Backward of ``layer_norm_fwd`` (``gdn_layer_norm_bwd``): returns ``(dx, dweight, dbias)``, the last two [D]
    fp32.  ``mean`` and ``rstd`` are the forward's."""
    if stream is not None:
        return _elsewhere(stream, layer_norm_bwd, dout, x, mean, rstd, weight, workspace)
    lib = _lib or load_library()
    rows, D = _check_norm_args(x, (weight,), (mean, rstd), (dout,))
    dt = _dt(x)
    device = x.device
    dx = _empty_like(x)
    dw = _empty(D, dtype=_F32, device=device)
    db = _empty_like(dw)
    ws, size = _workspace(workspace, 0 if workspace is not None else
                          lib.gdn_layer_norm_bwd_workspace_size(rows, D, dt), device)
    rc = lib.gdn_layer_norm_bwd(dout.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _ptr(weight),
                                dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows, D, dt, ws.data_ptr(), size,
                                _stream_of(x))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_layer_norm_bwd")
    return dx, dw, db


def _check_ce_args(h, weight, targets, rows):
    """Shapes, dtypes, placement and contiguity of a cross-entropy call; returns (N, D, V)."""
    hs, ws = h.shape, weight.shape
    if len(hs) != 2 or len(ws) != 2 or hs[1] != ws[1]:
        raise ValueError("h must be [N,D] and weight [V,D]")
    if weight.dtype is not h.dtype:
        raise TypeError("h and weight must share one dtype")
    if targets.dtype is not torch.int32:
        raise TypeError("targets must be int32")
    N = hs[0]
    if N > _MOST or hs[1] > _MOST or ws[0] > _MOST:
        _too_large(N=N, D=hs[1], V=ws[0])
    if targets.shape != (N,):
        raise ValueError("targets must be [N]")
    for t in rows:
        if t.dtype is not _F32:
            raise TypeError("lse and dloss must be float32")
        if t.shape != (N,):
            raise ValueError("lse and dloss must be [N]")
    _need_cuda(h, weight, targets, *rows)
    return N, hs[1], ws[0]


def linear_cross_entropy_workspace_size(N, D, V, dtype=torch.bfloat16, backward=False) -> int:
    dt = GDN_BF16 if dtype == _BF16 else GDN_F32
    if max(N, D, V) > _MOST:
        return 0
    return int(load_library().gdn_linear_cross_entropy_workspace_size(N, D, V, dt, int(bool(backward))))


def linear_cross_entropy_fwd(h, weight, targets, workspace=None, stream=None):
    """Softmax cross entropy of the logits ``h @ weight.T`` without forming them
    (``gdn_linear_cross_entropy_fwd``).

    h [N,D], weight [V,D] (fp32 or bf16); targets int32 [N], rows with a target outside [0,V) are ignored.
    Returns ``(loss, lse)``, both [N] fp32 and 0 in ignored rows.
    """
    if stream is not None:
        return _elsewhere(stream, linear_cross_entropy_fwd, h, weight, targets, workspace)
    lib = _lib or load_library()
    N, D, V = _check_ce_args(h, weight, targets, ())
    dt = _dt(h)
    device = h.device
    loss = _empty(N, dtype=_F32, device=device)
    lse = _empty_like(loss)
    ws, size = _workspace(workspace, 0 if workspace is not None else
                          lib.gdn_linear_cross_entropy_workspace_size(N, D, V, dt, 0), device)
    rc = lib.gdn_linear_cross_entropy_fwd(h.data_ptr(), weight.data_ptr(), targets.data_ptr(), loss.data_ptr(),
                                          lse.data_ptr(), N, D, V, dt, ws.data_ptr(), size, _stream_of(h))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_linear_cross_entropy_fwd")
    return loss, lse


def linear_cross_entropy_bwd(h, weight, targets, lse, dloss, workspace=None, stream=None):
    """Gradient of ``linear_cross_entropy_fwd`` (``gdn_linear_cross_entropy_bwd``) for the gradient ``dloss`` [N]
    fp32 of each row's loss: returns ``(dh, dweight)`` in the dtype of h.  ``lse`` is the forward's."""
    if stream is not None:
        return _elsewhere(stream, linear_cross_entropy_bwd, h, weight, targets, lse, dloss, workspace)
    lib = _lib or load_library()
    N, D, V = _check_ce_args(h, weight, targets, (lse, dloss))
    dt = _dt(h)
    dh, dw = _empty_like(h), _empty_like(weight)
    ws, size = _workspace(workspace, 0 if workspace is not None else
                          lib.gdn_linear_cross_entropy_workspace_size(N, D, V, dt, 1), h.device)
    rc = lib.gdn_linear_cross_entropy_bwd(h.data_ptr(), weight.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                                          dloss.data_ptr(), dh.data_ptr(), dw.data_ptr(), N, D, V, dt, ws.data_ptr(),
                                          size, _stream_of(h))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_linear_cross_entropy_bwd")
    return dh, dw


def check_device_error(workspace, stream=None):
    rc = load_library().gdn_check_device_error(_ptr(workspace), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_check_device_error")


def selftest_wait_timeout(workspace, limit_us=20000, stream=None):
    """``gdn_selftest_wait_timeout``: enqueue a kernel whose bounded wait on a phase that nothing
    completes gives up after ``limit_us`` and records the timeout in ``workspace``'s error word
    (read back by ``check_device_error``, which then raises GDN_ERR_DEVICE_TIMEOUT)."""
    _need_cuda(workspace)
    rc = load_library().gdn_selftest_wait_timeout(_ptr(workspace), int(limit_us), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_selftest_wait_timeout")


def selftest_linear_cross_entropy_timeout(step, h, weight, targets, lse, dloss, out0, out1, workspace, limit_us=20000,
                                          stream=None):
    """``gdn_selftest_linear_cross_entropy_timeout``: a cross-entropy call (``step`` 0 forward, 1 and 2 backward) one of
    whose kernels waits in vain, gives up after ``limit_us`` and leaves NaN in the results that it reaches."""
    N, D, V = _check_ce_args(h, weight, targets, [t for t in (lse, dloss) if t is not None])
    _need_cuda(out0, out1, workspace)
    rc = load_library().gdn_selftest_linear_cross_entropy_timeout(
        step, limit_us, _ptr(h), _ptr(weight), _ptr(targets), _ptr(lse), _ptr(dloss), _ptr(out0), _ptr(out1), N, D, V,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_selftest_linear_cross_entropy_timeout")


def chunk_fwd_noalloc(q, k, v, g, beta, out, final_state=None, init_state=None, cu_seqlens=None, scale=None,
                      use_qk_l2norm=True, chunk_size=CHUNK, stream=None):
    """``gdn_chunk_fwd_noalloc``: the chunked forward with the library's fixed
    device scratch array instead of a workspace, for callers that cannot
    allocate.  The caller passes every output buffer; nothing is allocated.
    Problems needing more than ``NOALLOC_SCRATCH_BYTES`` of scratch are
    rejected (GDN_ERR_WORKSPACE).  Calls that overlap on the GPU race."""
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if scale is None:
        scale = dk ** -0.5
    if out is None:
        raise ValueError("chunk_fwd_noalloc allocates nothing: pass out")
    _check_chunk_args(q, k, v, g, beta, init_state, cu_seqlens, out, final_state)
    num_seqs = (cu_seqlens.numel() - 1) if cu_seqlens is not None else 0
    rc = lib.gdn_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(init_state),
                                   _ptr(cu_seqlens), num_seqs, _ptr(out), _ptr(final_state),
                                   B, T, H, dk, dv, _dt(q), float(scale), int(bool(use_qk_l2norm)),
                                   int(chunk_size), _stream(stream))
    if rc != GDN_OK:
        what = "gdn_chunk_fwd_noalloc"
        if rc == 3:
            what += f" (problem needs more than the {NOALLOC_SCRATCH_BYTES >> 20} MiB fixed scratch)"
        raise GDNError(rc, what)
    return out, final_state
