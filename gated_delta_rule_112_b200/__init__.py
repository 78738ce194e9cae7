"""Gated delta rule forward pass and decode step on B200 (sm_100a).

A thin ctypes binding over ``libgdn.so`` (C ABI in ``include/gdn.h``). This
module only marshals arguments: it allocates outputs and workspace with
PyTorch, passes device pointers and the current CUDA stream, and checks the
returned status. Every step of the computation runs in the library's CUDA
kernels; there is no CPU fallback -- if the library or a GPU is missing, the
calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import NamedTuple

import torch

__all__ = ["chunk_fwd", "chunk_bwd", "chunk_fwd_save", "chunk_bwd_saved", "decode_step",
           "workspace_size", "chunk_path", "get_status",
           "recurrent_fwd", "qk_norm_rope_fwd", "qk_norm_rope_bwd", "Packed", "pack", "unpack",
           "chunk_fwd_packed", "chunk_bwd_packed", "Checkpoint", "status_block",
           "lib", "GdnError", "BF16", "F32", "PATH_TCGEN05", "PATH_SIMT"]

_HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_LIBRARY selects another build of the same library (e.g. the bounds-checked
# libgdn_checked.so); the default is the in-tree libgdn.so.
LIB_PATH = os.environ.get("GDN_LIBRARY") or os.path.join(_HERE, "libgdn.so")

(OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT,
 ERR_DEVICE_BOUNDS) = range(7)
BF16, F32 = 0, 1
PATH_TCGEN05, PATH_SIMT = 1, 2

NORM_NONE, NORM_L2, NORM_RMS = range(3)
_NORMS = {"none": NORM_NONE, "l2": NORM_L2, "rms": NORM_RMS}

_lib = None


class _Rows(ctypes.Structure):          # gdn_rows
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _PackedRows(ctypes.Structure):    # gdn_packed
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class _QkParams(ctypes.Structure):      # gdn_qk_params
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "H_q", "H_k", "d", "rot", "interleaved", "norm",
                                               "dtype")] +
                [(n, ctypes.c_float) for n in ("eps", "weight_offset", "q_scale", "rope_scale")] +
                [(n, ctypes.c_void_p) for n in ("positions", "inv_freq", "w_q", "w_k")])


class GdnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {_status_string(code)} ({code})")


def _status_string(code: int) -> str:
    try:
        return lib().gdn_status_string(code).decode()
    except Exception:  # library missing
        return str(code)


def lib() -> ctypes.CDLL:
    """Load libgdn.so (built in-tree by ``gated_delta_rule_112_b200.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgdn.so not built ({LIB_PATH}); run "
                               "python -m gated_delta_rule_112_b200.build")
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
        ci, sz = ctypes.c_int, ctypes.c_size_t
        chunk_args = [vp, vp, vp, fp, fp, fp, ip, ci, ci, ci, ci, ci, ci, ci, ci, vp, fp, vp,
                      sz, vp]
        L.gdn_chunk_fwd.argtypes = chunk_args
        L.gdn_chunk_fwd.restype = ci
        L.gdn_chunk_fwd_simt.argtypes = chunk_args
        L.gdn_chunk_fwd_simt.restype = ci
        L.gdn_chunk_fwd_workspace_size.argtypes = [ci] * 8
        L.gdn_chunk_fwd_workspace_size.restype = sz
        L.gdn_chunk_fwd_scan_segments.argtypes = [ci] * 9
        L.gdn_chunk_fwd_scan_segments.restype = ci
        L.gdn_selftest_wait_timeout.argtypes = [vp, vp]
        L.gdn_selftest_wait_timeout.restype = ci
        L.gdn_chunk_fwd_path.argtypes = [ci] * 4
        L.gdn_chunk_fwd_path.restype = ci
        L.gdn_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, ci, ci, ci, ci, ci, vp]
        L.gdn_decode_step.restype = ci
        L.gdn_kda_chunk_fwd.argtypes = chunk_args
        L.gdn_kda_chunk_fwd.restype = ci
        L.gdn_kda_chunk_fwd_workspace_size.argtypes = [ci] * 8
        L.gdn_kda_chunk_fwd_workspace_size.restype = sz
        L.gdn_kda_decode_step.argtypes = L.gdn_decode_step.argtypes
        L.gdn_kda_decode_step.restype = ci
        L.gdn_chunk_bwd_workspace_size.argtypes = [ci] * 7
        L.gdn_chunk_bwd_workspace_size.restype = sz
        L.gdn_chunk_bwd_exact_workspace_size.argtypes = [ci] * 6
        L.gdn_chunk_bwd_exact_workspace_size.restype = sz
        L.gdn_chunk_bwd.argtypes = [vp, vp, vp, fp, fp, fp, ip, vp, fp, ci, ci, ci, ci, ci, ci,
                                    ci, fp, fp, fp, fp, fp, fp, vp, sz, vp]
        L.gdn_chunk_bwd.restype = ci
        L.gdn_chunk_bwd_saved.argtypes = L.gdn_chunk_bwd.argtypes
        L.gdn_chunk_bwd_saved.restype = ci
        L.gdn_chunk_fwd_save.argtypes = [vp, vp, vp, fp, fp, fp, ip, ci, ci, ci, ci, ci, ci, ci,
                                         vp, fp, vp, sz, vp]
        L.gdn_chunk_fwd_save.restype = ci
        L.gdn_chunk_bwd_exact.argtypes = [vp, vp, vp, fp, fp, fp, ip, vp, fp, ci, ci, ci, ci, ci, ci,
                                    ci, fp, fp, fp, fp, fp, fp, vp, sz, vp]
        L.gdn_chunk_bwd_exact.restype = ci
        i64, rp = ctypes.c_int64, ctypes.POINTER(_Rows)
        pp, kp = ctypes.POINTER(_QkParams), ctypes.POINTER(_PackedRows)
        L.gdn_recurrent_fwd.argtypes = ([vp, vp, vp, fp, fp, vp, ip, ip, ip, vp] + [ci] * 6 +
                                        [i64] * 4 + [ci] * 3 + [vp, vp, vp])
        L.gdn_recurrent_fwd.restype = ci
        L.gdn_qk_norm_rope_fwd.argtypes = [pp, rp, rp, rp, rp, kp, kp, vp]
        L.gdn_qk_norm_rope_fwd.restype = ci
        L.gdn_qk_norm_rope_fwd_packed.argtypes = [pp, kp, kp, rp, rp, vp]
        L.gdn_qk_norm_rope_fwd_packed.restype = ci
        L.gdn_qk_norm_rope_bwd_workspace_size.argtypes = [pp]
        L.gdn_qk_norm_rope_bwd_workspace_size.restype = sz
        L.gdn_qk_norm_rope_bwd.argtypes = [pp, rp, rp, ci, rp, rp, rp, rp, fp, fp, vp, sz, vp]
        L.gdn_qk_norm_rope_bwd.restype = ci
        L.gdn_qk_norm_rope_bwd_packed.argtypes = [pp, rp, rp, ci, kp, kp, rp, rp, fp, fp, vp, sz,
                                                  vp]
        L.gdn_qk_norm_rope_bwd_packed.restype = ci
        L.gdn_get_status.argtypes = [vp, vp]
        L.gdn_get_status.restype = ci
        L.gdn_set_profile_events.argtypes = [vp, vp, vp, vp]
        L.gdn_set_profile_events.restype = ci
        L.gdn_checked_build.argtypes = []
        L.gdn_checked_build.restype = ci
        L.gdn_status_string.argtypes = [ci]
        L.gdn_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return BF16
    if t == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t}; use bfloat16 or float32")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, what: str):
    if code != OK:
        raise GdnError(code, what)


def workspace_size(B, T, H, d_k, d_v, num_seqs=0, chunk=64, dtype=torch.bfloat16) -> int:
    return int(lib().gdn_chunk_fwd_workspace_size(B, T, H, d_k, d_v, num_seqs, chunk,
                                                  _dtype_code(dtype)))


def chunk_path(d_k, d_v, chunk=64, dtype=torch.bfloat16) -> int:
    return int(lib().gdn_chunk_fwd_path(d_k, d_v, chunk, _dtype_code(dtype)))


def _require_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")


def chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk=64,
              output_final_state=True, workspace=None, out=None, force_simt=False,
              stream=None):
    """Chunkwise forward pass. Returns ``(o, final_state or None)``.

    q, k: [B,T,H,d_k]; v: [B,T,H,d_v] (bf16 or fp32, same dtype); g (= log
    alpha), beta: [B,T,H] fp32; initial_state: [N,H,d_k,d_v] fp32 or None;
    cu_seqlens: int32 [N+1] CUDA tensor (packed sequences, B == 1) or None.
    """
    fn = lib().gdn_chunk_fwd_simt if force_simt else lib().gdn_chunk_fwd
    return _chunk_call(fn, "gdn_chunk_fwd", lib().gdn_chunk_fwd_workspace_size, q, k, v, g,
                       beta, initial_state, cu_seqlens, chunk, output_final_state, workspace,
                       out, stream, channel_gate=False)


def kda_workspace_size(B, T, H, d_k, d_v, num_seqs=0, chunk=64, dtype=torch.bfloat16) -> int:
    return int(lib().gdn_kda_chunk_fwd_workspace_size(B, T, H, d_k, d_v, num_seqs, chunk,
                                                      _dtype_code(dtype)))


def kda_chunk_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk=64,
                  output_final_state=True, workspace=None, out=None, stream=None):
    """Chunkwise forward pass with the channel-wise gate: as ``chunk_fwd`` but
    g (= log alpha) is [B,T,H,d_k] fp32. Returns ``(o, final_state or None)``."""
    return _chunk_call(lib().gdn_kda_chunk_fwd, "gdn_kda_chunk_fwd",
                       lib().gdn_kda_chunk_fwd_workspace_size, q, k, v, g, beta, initial_state,
                       cu_seqlens, chunk, output_final_state, workspace, out, stream,
                       channel_gate=True)


def _chunk_call(fn, name, ws_fn, q, k, v, g, beta, initial_state, cu_seqlens, chunk,
                output_final_state, workspace, out, stream, channel_gate):
    _require_cuda(q, k, v, g, beta, initial_state, cu_seqlens)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(g.shape) != ((B, T, H, dk) if channel_gate else (B, T, H)):
        raise ValueError(f"{name}: g has shape {tuple(g.shape)}")
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    N = num_seqs if cu_seqlens is not None else B
    dt = _dtype_code(q.dtype)
    o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device) if out is None else out
    fs = (torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
          if output_final_state else None)
    need = int(ws_fn(B, T, H, dk, dv, num_seqs, chunk, dt))
    if need == 0:
        raise GdnError(ERR_INVALID_ARG, name + "_workspace_size")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
            _ptr(cu_seqlens), B, T, H, dk, dv, num_seqs, chunk, dt, _ptr(o), _ptr(fs),
            _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc, name)
    return o, fs


def bwd_workspace_size(B, T, H, d_k, d_v, num_seqs=0, dtype=torch.bfloat16,
                       exact=False) -> int:
    """Workspace bytes of ``chunk_bwd`` (exact=False: the path gdn_chunk_bwd
    picks for dtype; exact=True: the token-level fp32 path)."""
    if exact:
        return int(lib().gdn_chunk_bwd_exact_workspace_size(B, T, H, d_k, d_v, num_seqs))
    return int(lib().gdn_chunk_bwd_workspace_size(B, T, H, d_k, d_v, num_seqs,
                                                   _dtype_code(dtype)))


def chunk_bwd(q, k, v, g, beta, d_o, initial_state=None, cu_seqlens=None, d_final_state=None,
              workspace=None, stream=None, exact=False, _saved=False):
    """Gradients of ``chunk_fwd`` (scalar gate) for the loss
    sum(d_o * o) + sum(d_final_state * final_state).

    Inputs as for ``chunk_fwd``, plus d_o [B,T,H,d_v] (same dtype as v) and
    d_final_state [N,H,d_k,d_v] fp32 or None. Returns a dict of fp32 CUDA
    tensors: dq, dk [B,T,H,d_k], dv [B,T,H,d_v], dg, dbeta [B,T,H],
    d_initial_state [N,H,d_k,d_v]. bf16 with d_k = d_v = 128 runs the chunkwise
    tensor-core backward; exact=True (or any other size or dtype) the
    token-level fp32 backward.
    """
    _require_cuda(q, k, v, g, beta, d_o, initial_state, cu_seqlens, d_final_state)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    N = num_seqs if cu_seqlens is not None else B
    dev = q.device
    f32 = dict(dtype=torch.float32, device=dev)
    out = dict(dq=torch.empty(B, T, H, dk, **f32), dk=torch.empty(B, T, H, dk, **f32),
               dv=torch.empty(B, T, H, dv, **f32), dg=torch.empty(B, T, H, **f32),
               dbeta=torch.empty(B, T, H, **f32),
               d_initial_state=torch.empty(N, H, dk, dv, **f32))
    need = bwd_workspace_size(B, T, H, dk, dv, num_seqs, q.dtype, exact)
    if need == 0:
        raise GdnError(ERR_INVALID_ARG, "gdn_chunk_bwd_workspace_size")
    if _saved:
        if workspace is None or workspace.numel() < need:
            raise GdnError(ERR_WORKSPACE, "gdn_chunk_bwd_saved")
    elif workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    fn = (lib().gdn_chunk_bwd_saved if _saved else
          lib().gdn_chunk_bwd_exact if exact else lib().gdn_chunk_bwd)
    name = "gdn_chunk_bwd_saved" if _saved else "gdn_chunk_bwd_exact" if exact else "gdn_chunk_bwd"
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
            _ptr(cu_seqlens), _ptr(d_o), _ptr(d_final_state), B, T, H, dk, dv,
            num_seqs, _dtype_code(q.dtype), _ptr(out["dq"]), _ptr(out["dk"]),
            _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
            _ptr(out["d_initial_state"]), _ptr(workspace), workspace.numel(),
            _stream_ptr(stream))
    _check(rc, name)
    return out


def chunk_fwd_save(q, k, v, g, beta, initial_state=None, cu_seqlens=None,
                   output_final_state=True, workspace=None, out=None, stream=None):
    """Forward pass of a training step (bf16, d_k = d_v = 128): ``chunk_fwd``
    that also keeps in its workspace what ``chunk_bwd_saved`` needs (the chunk
    map, the prep tiles and every chunk's entering state). Returns ``(o,
    final_state or None, saved)``; hand ``saved`` unchanged to
    ``chunk_bwd_saved`` with the same inputs."""
    _require_cuda(q, k, v, g, beta, initial_state, cu_seqlens)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(g.shape) != (B, T, H):
        raise ValueError(f"gdn_chunk_fwd_save: g has shape {tuple(g.shape)}")
    num_seqs = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    N = num_seqs if cu_seqlens is not None else B
    o = torch.empty(B, T, H, dv, dtype=q.dtype, device=q.device) if out is None else out
    fs = (torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
          if output_final_state else None)
    need = bwd_workspace_size(B, T, H, dk, dv, num_seqs, q.dtype)
    if need == 0:
        raise GdnError(ERR_INVALID_ARG, "gdn_chunk_bwd_workspace_size")
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    rc = lib().gdn_chunk_fwd_save(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  _ptr(initial_state), _ptr(cu_seqlens), B, T, H, dk, dv,
                                  num_seqs, _dtype_code(q.dtype), _ptr(o), _ptr(fs),
                                  _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc, "gdn_chunk_fwd_save")
    return o, fs, workspace


def chunk_bwd_saved(q, k, v, g, beta, d_o, saved, initial_state=None, cu_seqlens=None,
                    d_final_state=None, stream=None):
    """``chunk_bwd`` from the workspace ``saved`` that ``chunk_fwd_save`` filled
    for the same inputs: the forward replay is skipped. Returns the same dict
    of fp32 gradients."""
    return chunk_bwd(q, k, v, g, beta, d_o, initial_state, cu_seqlens, d_final_state,
                     workspace=saved, stream=stream, _saved=True)


def get_status(workspace=None, stream=None) -> int:
    """Synchronise the stream and return the first recorded error code."""
    return int(lib().gdn_get_status(_ptr(workspace), _stream_ptr(stream)))


def decode_step(q, k, v, g, beta, state, out=None, stream=None):
    """One recurrent step, updating ``state`` [N,H,d_k,d_v] fp32 in place.

    q, k: [N,H,d_k]; v: [N,H,d_v]; g, beta: [N,H] fp32. Returns o [N,H,d_v].
    """
    return _decode_call(lib().gdn_decode_step, "gdn_decode_step", q, k, v, g, beta, state,
                        out, stream, channel_gate=False)


def kda_decode_step(q, k, v, g, beta, state, out=None, stream=None):
    """One channel-wise-gated step (g: [N,H,d_k] fp32), ``state`` updated in place."""
    return _decode_call(lib().gdn_kda_decode_step, "gdn_kda_decode_step", q, k, v, g, beta,
                        state, out, stream, channel_gate=True)


def _decode_call(fn, name, q, k, v, g, beta, state, out, stream, channel_gate):
    _require_cuda(q, k, v, g, beta, state)
    N, H, dk = q.shape
    dv = v.shape[-1]
    if tuple(g.shape) != ((N, H, dk) if channel_gate else (N, H)):
        raise ValueError(f"{name}: g has shape {tuple(g.shape)}")
    o = torch.empty(N, H, dv, dtype=q.dtype, device=q.device) if out is None else out
    rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state), _ptr(o), N, H, dk, dv,
            _dtype_code(q.dtype), _stream_ptr(stream))
    _check(rc, name)
    return o


# ---------------------------------------------------------------- states of many requests

def status_block(device=None) -> torch.Tensor:
    """A zeroed control block for the ``status`` argument of ``recurrent_fwd``;
    hand it to ``get_status`` to read (and clear) what its calls recorded."""
    return torch.zeros(256, dtype=torch.uint8, device=device or "cuda")


def recurrent_fwd(q, k, v, g, beta, pool, slots=None, cu_seqlens=None, keep=None, reset=None,
                  out=None, status=None, stream=None):
    """Runs of new tokens of many sequences against a pool of states, which is
    updated in place. Returns o [T,H_v,d_v].

    q, k: [T,H_k,d_k]; v: [T,H_v,d_v] (bf16 or fp32, one dtype; tokens may be
    apart, as in slices of a wider projection output); g (= log alpha): [T,H_v],
    or [T,H_v,d_k] for the channel-wise gate; beta: [T,H_v] (fp32); pool:
    [num_slots,H_v,d_k,d_v] fp32 or bf16. H_v is a multiple of H_k.

    Run n has tokens cu_seqlens[n] to cu_seqlens[n+1] (int32 [N+1]; without it
    all N runs have T/N) and its state in slot slots[n] (int32 [N]; without it
    slot n; negative: padding, whose boundaries are not looked at). The state
    kept is that after its first keep[n] tokens (int32 [N]; without it all; 0
    leaves the slot alone); reset[n] (bool [N]) starts it from zero. Tokens of no
    run keep what ``out`` held; ``out`` may not overlap an input.
    A run the device finds wrong (see gdn.h) leaves its state alone and has NaN
    outputs; ``status`` (see ``status_block``) then tells get_status."""
    name = "gdn_recurrent_fwd"
    dev = q.get_device()
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        with _on(name, dev, stream, q, k, v, g, beta, pool, slots, cu_seqlens, keep, reset, out,
                 status):
            return recurrent_fwd(q, k, v, g, beta, pool, slots, cu_seqlens, keep, reset, out, status)
    T, Hk, dk = q.shape
    _, Hv, dv = v.shape
    P = pool.shape[0]
    channel = g.dim() == 3
    dt, st = q.dtype, pool.dtype
    if cu_seqlens is not None:
        N = cu_seqlens.numel() - 1
    else:
        N = slots.numel() if slots is not None else P
    if out is None:
        out = torch.empty_like(v)
        if not out.is_contiguous():
            out = torch.empty((T, Hv, dv), dtype=dt, device="cuda")
    (qs, qh, qe), (ks, kh, ke), (vs, vh, ve) = q.stride(), k.stride(), v.stride()
    f32 = torch.float32
    if not (dt in _DTYPES and st in _DTYPES and k.dtype == dt and v.dtype == dt and out.dtype == dt and
            g.dtype == f32 and beta.dtype == f32 and
            k.shape == q.shape and v.shape[0] == T and out.shape == (T, Hv, dv) and
            g.shape == ((T, Hv, dk) if channel else (T, Hv)) and beta.shape == (T, Hv) and
            pool.shape == (P, Hv, dk, dv) and max(T, N, Hk, Hv, dk, dv) <= _INT32_MAX and
            (qe == 1 or dk == 1) and (ke == 1 or dk == 1) and (ve == 1 or dv == 1) and
            (qh == dk or Hk == 1) and (kh == dk or Hk == 1) and (vh == dv or Hv == 1) and
            g.is_contiguous() and beta.is_contiguous() and pool.is_contiguous() and
            out.is_contiguous() and
            _same_device(dev, k, v, g, beta, pool, slots, cu_seqlens, keep, reset, out, status) and
            _index(slots, torch.int32, N) and _index(cu_seqlens, torch.int32, N + 1) and
            _index(keep, torch.int32, N) and _index(reset, torch.bool, N) and
            (status is None or status.nbytes >= 256 and status.is_contiguous())):
        raise ValueError(
            f"{name}: q, k [T,H_k,d_k], v [T,H_v,d_v] and out of one type (bf16 or fp32), heads of a "
            "token next to each other; g [T,H_v] or [T,H_v,d_k] and beta [T,H_v] contiguous fp32; "
            "pool [num_slots,H_v,d_k,d_v] contiguous, bf16 or fp32; slots, keep [N] and cu_seqlens "
            "[N+1] int32, reset [N] bool; status of 256 bytes in a row; all on one CUDA device; sizes below 2^31")
    if T <= 1:                    # the stride of one token is of no account
        qs, ks, vs = max(qs, Hk * dk), max(ks, Hk * dk), max(vs, Hv * dv)
    rc = lib().gdn_recurrent_fwd(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), pool.data_ptr(),
        _at(slots), _at(cu_seqlens), _at(keep), _at(reset), N, T, Hk, Hv, dk, dv, P, qs, ks, vs,
        channel, _DTYPES[dt], _DTYPES[st], out.data_ptr(), _at(status), _raw_stream(dev))
    if rc != OK:
        _check(rc, name)
    return out


_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}
_INT32_MAX = 2 ** 31 - 1          # ctypes would pass the low 32 bits of a larger size
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


@contextlib.contextmanager
def _on(name, dev, stream, *used):
    """The tensors' device and the caller's stream as the current ones: outputs
    are allocated on the stream that writes them, and the memory of what the
    call uses is not given away before that stream has run it."""
    if dev < 0:
        raise ValueError(f"{name}: all tensors must be CUDA tensors")
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"{name}: the stream is on device {stream.device_index}, the tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        yield
    if stream is not None:
        for t in used:
            for x in t if isinstance(t, tuple) else (t,):
                if isinstance(x, tuple):
                    for y in x:
                        y.record_stream(stream)
                elif isinstance(x, torch.Tensor):
                    x.record_stream(stream)


def _at(t):
    return None if t is None else t.data_ptr()


def _same_device(dev, *ts):
    for t in ts:
        if t is not None and t.get_device() != dev:
            return False
    return dev >= 0


def _scratch(name, t, need, dev):
    """Whether the caller's workspace is to be used: it may be too small or None,
    but what is written to must be one piece of this device's memory."""
    if t is None or t.nbytes < need:
        return False
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: workspace not contiguous or on another device")
    return True


def _index(t, dtype, n):
    return t is None or (t.dtype == dtype and t.numel() == n and t.is_contiguous())


# ---------------------------------------------------------------- queries and keys

class Packed(NamedTuple):
    """Rows in 8 bits: codes [T,H,d] float8_e4m3fn and scales [T,H,ceil(d/32)]
    uint8; element e stands for codes[e] * 2^(scales[e // 32] - 127)."""
    codes: torch.Tensor
    scales: torch.Tensor


def _new_rows(x, dtype):
    """A contiguous tensor of x's shape, and its rows."""
    if x is None:
        return None, None
    y = torch.empty_like(x) if x.dtype == dtype else torch.empty_like(x, dtype=dtype)
    if not y.is_contiguous():
        y = torch.empty(x.shape, dtype=dtype, device="cuda")
    _, H, d = y.shape
    return y, _Rows(y.data_ptr(), H * d, d)


def _new_packed(x):
    """Packed rows for x, and their pointers."""
    T, H, d = x.shape
    y = Packed(x.new_empty((T, H, d), dtype=torch.float8_e4m3fn),
               x.new_empty((T, H, (d + 31) // 32), dtype=torch.uint8))
    return y, _PackedRows(y.codes.data_ptr(), y.scales.data_ptr())


def _packed_arg(name, x, dev, shape=None):
    if x is None:
        return None
    codes, scales = x
    T, H, d = codes.shape
    if not (codes.dtype == torch.float8_e4m3fn and scales.dtype == torch.uint8 and
            scales.shape == (T, H, (d + 31) // 32) and codes.is_contiguous() and
            scales.is_contiguous() and (shape is None or codes.shape == shape) and
            codes.get_device() == dev and scales.get_device() == dev):
        raise ValueError(f"{name}: packed rows are codes [T,H,d] float8_e4m3fn and scales "
                         "[T,H,ceil(d/32)] uint8, contiguous, on one CUDA device")
    return _PackedRows(codes.data_ptr(), scales.data_ptr())


def _rows_arg(name, x, dev, shape, dtype):
    if x is None:
        return None
    (T, H, d), (ts, hs, es) = x.shape, x.stride()
    if not (x.dtype == dtype and x.shape == shape and (es == 1 or d <= 1) and x.get_device() == dev):
        raise ValueError(f"{name}: rows of shape {tuple(x.shape)} and {x.dtype}, expected "
                         f"{tuple(shape)} and {dtype}, channels contiguous, on one CUDA device")
    if H <= 1:
        hs = d
    return _Rows(x.data_ptr(), ts if T > 1 else (H - 1) * hs + d, hs)


def _qk_params(name, dev, qs, ks, dtype, w_q, w_k, positions, inv_freq, norm, eps, interleaved,
               weight_offset, q_scale, rope_scale):
    """qs, ks: shapes of q and k (ks None without k)."""
    T, Hq, d = qs
    Hk = 0 if ks is None else ks[1]
    if max(T, Hq, Hk, d) > _INT32_MAX:
        raise ValueError(f"{name}: sizes of 2^31 and more")
    if not (dtype in _DTYPES and norm in _NORMS and (ks is None or (ks[0] == T and ks[2] == d)) and
            (positions is None) == (inv_freq is None) and (ks is not None or w_k is None)):
        raise ValueError(f"{name}: q and k [T,H,d] of bf16 or fp32, norm one of {sorted(_NORMS)}, "
                         "positions together with inv_freq, w_k only with k")
    rot = 0
    if positions is not None:
        rot = 2 * inv_freq.numel()
        if not (_index(positions, torch.int32, T) and positions.get_device() == dev and rot <= d and
                _index(inv_freq, torch.float64, rot // 2) and inv_freq.get_device() == dev):
            raise ValueError(f"{name}: positions int32 [T], inv_freq float64 [rot/2] with rot <= d, "
                             "contiguous, on the rows' device")
    for w in (w_q, w_k):
        if w is not None and not (_index(w, dtype, d) and w.get_device() == dev):
            raise ValueError(f"{name}: w_q and w_k [d] of the rows' dtype, contiguous, on their device")
    return _QkParams(T, Hq, Hk, d, rot, interleaved, _NORMS[norm], _DTYPES[dtype], eps, weight_offset,
                     q_scale, rope_scale, _at(positions) if rot else None,
                     _at(inv_freq) if rot else None, _at(w_q), _at(w_k))


def _qk_source(name, q, k):
    """(packed?, the tensor whose shape is q's, k's or None)."""
    if isinstance(q, tuple):
        if k is not None and not isinstance(k, tuple):
            raise ValueError(f"{name}: q and k both packed, or neither")
        return True, q[0], None if k is None else k[0]
    if isinstance(k, tuple):
        raise ValueError(f"{name}: q and k both packed, or neither")
    return False, q, k


def qk_norm_rope_fwd(q, k, w_q=None, w_k=None, positions=None, inv_freq=None, norm="l2", eps=1e-6,
                     interleaved=False, weight_offset=0.0, q_scale=1.0, rope_scale=1.0, pack=False,
                     dtype=None, out=None, stream=None):
    """Norm of each head's row of q and k and the position rotation, one pass.
    Returns ``(q_out, k_out)``, with pack=True ``(q_out, k_out, q_packed,
    k_packed)``: the raw q and k in 8 bits, for the backward pass.

    q: [T,H_q,d], k: [T,H_k,d] or None (bf16 or fp32; tokens and heads may be
    apart), or both ``Packed`` (then dtype is that of the outputs, bfloat16 if
    not given). norm: "l2", "rms" or "none"; w_q, w_k: [d] weights (the
    rows' dtype) or None, to which weight_offset is added; inv_freq: fp64
    [rot/2] and positions: int32 [T] rotate the first rot elements, by halves
    or interleaved pairs, times rope_scale; q_scale multiplies q's outputs.
    out: ``(q_out, k_out)`` to write to; an output may be its own input, and
    with pack=True None, to write the 8-bit rows alone."""
    name = "gdn_qk_norm_rope_fwd"
    packed, qx, kx = _qk_source(name, q, k)
    dev = qx.get_device()
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        with _on(name, dev, stream, q, k, w_q, w_k, positions, inv_freq, out):
            return qk_norm_rope_fwd(q, k, w_q, w_k, positions, inv_freq, norm, eps, interleaved,
                                    weight_offset, q_scale, rope_scale, pack, dtype, out)
    if packed:
        if pack:
            raise ValueError(f"{name}: the rows are packed already")
        dtype = dtype or torch.bfloat16
    else:
        dtype = qx.dtype
    qs, ks = qx.shape, None if kx is None else kx.shape
    p = _qk_params(name, dev, qs, ks, dtype, w_q, w_k, positions, inv_freq, norm, eps, interleaved,
                   weight_offset, q_scale, rope_scale)
    if out is None:
        (qo, qr), (ko, kr) = _new_rows(qx, dtype), _new_rows(kx, dtype)
    else:
        qo, ko = out
        qr, kr = _rows_arg(name, qo, dev, qs, dtype), _rows_arg(name, ko, dev, ks, dtype)
    s = _raw_stream(dev)
    if packed:
        rc = lib().gdn_qk_norm_rope_fwd_packed(p, _packed_arg(name, q, dev), _packed_arg(name, k, dev),
                                               qr, kr, s)
        if rc != OK:
            _check(rc, name + "_packed")
        return qo, ko
    q8, q8p = _new_packed(q) if pack else (None, None)
    k8, k8p = _new_packed(k) if pack and k is not None else (None, None)
    rc = lib().gdn_qk_norm_rope_fwd(p, _rows_arg(name, q, dev, qs, dtype),
                                    _rows_arg(name, k, dev, ks, dtype), qr, kr,
                                    q8p, k8p, s)
    if rc != OK:
        _check(rc, name)
    return (qo, ko, q8, k8) if pack else (qo, ko)


def qk_norm_rope_bwd(dq_out, dk_out, q, k, w_q=None, w_k=None, positions=None, inv_freq=None,
                     norm="l2", eps=1e-6, interleaved=False, weight_offset=0.0, q_scale=1.0,
                     rope_scale=1.0, dtype=None, out=None, workspace=None, stream=None):
    """Gradients of ``qk_norm_rope_fwd``, whose inputs come again (q, k as they
    were, or ``Packed``: then at the point the 8-bit rows stand for). dq_out,
    dk_out: gradients of its outputs (fp32, or the rows' dtype). Returns a dict:
    dq, dk (the rows' dtype; for packed rows ``dtype``, bfloat16 if not given),
    dw_q, dw_k ([d] fp32, None without weights). out: ``(dq, dk)`` to write; each
    may be its own raw rows, or its gradients if they have the rows' type. Rows
    may not overlap, so a broadcast gradient (of a sum, say) is refused: give a
    ``.contiguous()`` one."""
    name = "gdn_qk_norm_rope_bwd"
    packed, qx, kx = _qk_source(name, q, k)
    dev = qx.get_device()
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        with _on(name, dev, stream, dq_out, dk_out, q, k, w_q, w_k, positions, inv_freq, out,
                 workspace):
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, w_q, w_k, positions, inv_freq, norm, eps,
                                    interleaved, weight_offset, q_scale, rope_scale, dtype, out,
                                    workspace)
    dtype = (dtype or torch.bfloat16) if packed else qx.dtype
    qs, ks = qx.shape, None if kx is None else kx.shape
    p = _qk_params(name, dev, qs, ks, dtype, w_q, w_k, positions, inv_freq, norm, eps, interleaved,
                   weight_offset, q_scale, rope_scale)
    gt = dq_out.dtype
    if gt not in _DTYPES or (ks is None) != (dk_out is None):
        raise ValueError(f"{name}: dq_out, dk_out like the outputs, fp32 or the rows' dtype")
    dyq, dyk = _rows_arg(name, dq_out, dev, qs, gt), _rows_arg(name, dk_out, dev, ks, gt)
    if out is None:
        (dq, qr), (dk, kr) = _new_rows(qx, dtype), _new_rows(kx, dtype)
    else:
        dq, dk = out
        qr, kr = _rows_arg(name, dq, dev, qs, dtype), _rows_arg(name, dk, dev, ks, dtype)
    dwq = None if w_q is None else torch.empty_like(w_q, dtype=torch.float32)
    dwk = None if w_k is None else torch.empty_like(w_k, dtype=torch.float32)
    need = 0
    if dwq is not None or dwk is not None:
        need = lib().gdn_qk_norm_rope_bwd_workspace_size(p)
        if not _scratch(name, workspace, need, dev):
            workspace = dq_out.new_empty(need, dtype=torch.uint8)
    s = _raw_stream(dev)
    if packed:
        rc = lib().gdn_qk_norm_rope_bwd_packed(
            p, dyq, dyk, _DTYPES[gt], _packed_arg(name, q, dev), _packed_arg(name, k, dev), qr, kr,
            _at(dwq), _at(dwk), _at(workspace), need, s)
    else:
        rc = lib().gdn_qk_norm_rope_bwd(
            p, dyq, dyk, _DTYPES[gt], _rows_arg(name, q, dev, qs, dtype),
            _rows_arg(name, k, dev, ks, dtype), qr, kr, _at(dwq), _at(dwk), _at(workspace), need, s)
    if rc != OK:
        _check(rc, name + ("_packed" if packed else ""))
    return dict(dq=dq, dk=dk, dw_q=dwq, dw_k=dwk)


def pack(x, stream=None) -> Packed:
    """Rows [T,H,d] in 8 bits (see ``Packed``)."""
    return qk_norm_rope_fwd(x, None, norm="none", pack=True, out=(None, None), stream=stream)[2]


def unpack(x: Packed, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The rows that 8-bit rows stand for: exact in fp32, and in bf16 but for fp32
    rows below 2^-115 or so, whose codes reach under bf16's smallest number."""
    return qk_norm_rope_fwd(x, None, norm="none", dtype=dtype, stream=stream)[0]


# ---------------------------------------------------------------- a training step on 8-bit checkpoints

class Checkpoint(NamedTuple):
    """What ``chunk_fwd_packed`` keeps for the backward pass: the raw q, k and v
    in 8 bits (with scales: 3.1 bytes a token, head and channel of d = 128,
    against 6 for q, k, v in bf16 or 10 with the normed q and k)."""
    q: Packed
    k: Packed
    v: Packed
    shape: tuple
    dtype: torch.dtype


def _step_args(name, dev, shape, dtype, g, beta, initial_state, cu_seqlens, d_final_state=None,
               **rows):
    """Refuses what the chunked passes would read as something else, or past its end.
    shape: (B, T, H, d_k, d_v); rows: tensors of the step by name."""
    B, T, H, dk, dv = shape
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1

    def fits(t, want, want_dtype):
        return t is None or (t.shape == want and t.dtype == want_dtype and t.get_device() == dev)

    for what, t in rows.items():
        if not fits(t, (B, T, H, dk if what in "qk" else dv), dtype):
            raise ValueError(f"{name}: {what} has shape {tuple(t.shape)} and {t.dtype}")
    f32 = torch.float32
    if g is None or beta is None or not (
            fits(g, (B, T, H), f32) and fits(beta, (B, T, H), f32) and
            fits(initial_state, (N, H, dk, dv), f32) and fits(d_final_state, (N, H, dk, dv), f32) and
            fits(cu_seqlens, (N + 1,), torch.int32)):
        raise ValueError(f"{name}: g and beta [B,T,H], states [N,H,d_k,d_v] (fp32) and cu_seqlens [N+1] "
                         "(int32) on the rows' device")


def chunk_fwd_packed(q, k, v, g, beta, initial_state=None, cu_seqlens=None, chunk=64,
                     output_final_state=True, stream=None, **norm):
    """``qk_norm_rope_fwd`` (its keywords in ``norm``; positions [B*T]) and
    ``chunk_fwd`` of the result, keeping q, k and v in 8 bits for
    ``chunk_bwd_packed``. q, k, v: [B,T,H,d] of one type, with equally many heads
    (repeat q and k where value heads share them). Returns ``(o, final_state or None,
    Checkpoint)``; o and the state are those of the exact q, k, v."""
    dev = q.get_device()
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        with _on("chunk_fwd_packed", dev, stream, q, k, v, g, beta, initial_state, cu_seqlens,
                 *norm.values()):
            return chunk_fwd_packed(q, k, v, g, beta, initial_state, cu_seqlens, chunk,
                                    output_final_state, **norm)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    _step_args("chunk_fwd_packed", dev, (B, T, H, dk, dv), q.dtype, g, beta, initial_state, cu_seqlens,
               q=q, k=k, v=v)
    flat = [x.reshape(B * T, H, x.shape[-1]) for x in (q, k, v)]
    qn, kn, q8, k8 = qk_norm_rope_fwd(flat[0], flat[1], pack=True, **norm)
    v8 = pack(flat[2])
    o, fs = chunk_fwd(qn.view(B, T, H, dk), kn.view(B, T, H, dk), flat[2].contiguous().view(B, T, H, dv),
                      g, beta, initial_state, cu_seqlens, chunk, output_final_state)
    return o, fs, Checkpoint(q8, k8, v8, (B, T, H, dk, dv), q.dtype)


def chunk_bwd_packed(ckpt: Checkpoint, g, beta, d_o, initial_state=None, cu_seqlens=None,
                     d_final_state=None, workspace=None, stream=None, exact=False, **norm):
    """Gradients of ``chunk_fwd_packed`` from its checkpoint, at the q, k and v
    that the 8-bit rows stand for. Arguments as there and for ``chunk_bwd``.
    Returns a dict: dq, dk (of the raw q, k; their dtype), dw_q, dw_k (fp32 or
    None), dv, dg, dbeta, d_initial_state (fp32). Repeated calls give the same
    bits, but for dg and dbeta of the chunkwise path: they agree to rounding."""
    dev = ckpt.q.codes.get_device()
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        with _on("chunk_bwd_packed", dev, stream, ckpt[:3], g, beta, d_o, initial_state, cu_seqlens,
                 d_final_state, workspace, *norm.values()):
            return chunk_bwd_packed(ckpt, g, beta, d_o, initial_state, cu_seqlens, d_final_state,
                                    workspace, exact=exact, **norm)
    B, T, H, dk, dv = ckpt.shape
    _scratch("chunk_bwd_packed", workspace, 0, dev)
    _step_args("chunk_bwd_packed", dev, ckpt.shape, ckpt.dtype, g, beta, initial_state, cu_seqlens,
               d_final_state, d_o=d_o)
    qn, kn = qk_norm_rope_fwd(ckpt.q, ckpt.k, dtype=ckpt.dtype, **norm)
    v = unpack(ckpt.v, ckpt.dtype)
    out = chunk_bwd(qn.view(B, T, H, dk), kn.view(B, T, H, dk), v.view(B, T, H, dv), g, beta, d_o,
                    initial_state, cu_seqlens, d_final_state, workspace, None, exact)
    raw = qk_norm_rope_bwd(out["dq"].view(B * T, H, dk), out["dk"].view(B * T, H, dk), ckpt.q, ckpt.k,
                           dtype=ckpt.dtype, **norm)
    out.update(dq=raw["dq"].view(B, T, H, dk), dk=raw["dk"].view(B, T, H, dk), dw_q=raw["dw_q"],
               dw_k=raw["dw_k"])
    return out
