"""MI355X-native Gated DeltaNet chunked forward.

A thin Python binding over ``libgdn.so`` (C ABI declared in include/gdn.h).
Every step of the computation runs in the library's HIP kernels; this module
only checks tensors, allocates outputs and workspace with torch and passes
device pointers plus torch's current HIP stream.  There is no fallback: if the
library is not built, every call raises.

Functions (same names as the C entry points, without the ``gdn_`` prefix):
  chunk_fwd(q, k, v, g, beta, h0=None, chunk=128, n_groups=0, ...) -> (o, h_T)
  chunk_fold(k, v, g, beta, n_groups, chunk=128)                 -> (A, Bm)
  compose_prefix(A, Bm, h_init=None, split_bf16=False)          -> (h_in, h_final)
  chunk_transform(k, v, g, beta, chunk=128, want_T=False)       -> (G, T, W, U)
  workspace_size(...), validate(...)
Linear attention with a decay per head (the rule without the correction):
  linear_chunk_fwd(q, k, v, g, h0=None)                         -> (o, h_T)
  linear_chunk_fwd_varlen(q, k, v, g, cu_seqlens, h0=None)      -> (o, h_T)
  linear_chunk_bwd(q, k, v, g, dO, h0=None, dh_T=None)          -> gradients
States in a pool [n_slots,H_v,d_k,d_v], for serving (beta=None: the linear rule):
  step(q, k, v, g, beta, state, slots=None)                     -> o
  tree_fwd(q, k, v, g, beta, parents, state, slots=None)        -> (o, u)
  tree_commit(k, u, g, parents, last, state, slots=None)        -> state
Outputs and a workspace that a caller passes to these (out, final_state,
values, workspace) are refused where they overlap an input or each other.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

F32, BF16 = 0, 1
PREFIX_SPLIT_BF16, PREFIX_SEQUENTIAL, PREFIX_BLOCKED = 1, 2, 4
STATUS = {0: "ok", -1: "null pointer", -2: "unsupported or inconsistent sizes",
          -3: "unsupported dtype", -4: "misaligned pointer", -5: "workspace too small",
          -6: "kernel launch failed"}


class GdnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H_qk", "H_v", "d_k", "d_v", "chunk", "n_groups", "dtype", "o_dtype")]


class GdnPoolShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "n", "H_qk", "H_v", "d_k", "d_v", "n_slots", "g_fixed", "dtype", "o_dtype")]


class GdnLinearShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "T", "H_qk", "H_v", "d_k", "d_v", "g_fixed", "dtype", "o_dtype")]


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} (status {status})")
        self.status = status


_lib = None

SYMBOLS = ("gdn_status_str", "gdn_validate", "gdn_workspace_size", "gdn_workspace_size_varlen",
           "gdn_chunk_fwd", "gdn_chunk_fwd_varlen",
           "gdn_chunk_fwd_stages", "gdn_chunk_fwd_timed", "gdn_chunk_fold", "gdn_compose_prefix",
           "gdn_chunk_transform", "gdn_chunk_fwd_noalloc", "gdn_chunk_fwd_affine",
           "gdn_workspace_size_bwd", "gdn_chunk_bwd_state", "gdn_workspace_size_bwd_grads", "gdn_chunk_bwd",
           "gdn_step", "gdn_tree_fwd", "gdn_tree_commit", "gdn_workspace_size_linear", "gdn_linear_chunk_fwd",
           "gdn_linear_chunk_fwd_varlen", "gdn_linear_chunk_bwd")
STAGE_PREP, STAGE_FOLD, STAGE_PREFIX, STAGE_WALK, STAGE_OUT, STAGE_ALL = 1, 2, 4, 8, 16, 31


def lib():
    """Load libgdn.so (raises if it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                               "(there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        SP = ctypes.POINTER(GdnShape)
        L.gdn_status_str.argtypes = [I]
        L.gdn_status_str.restype = ctypes.c_char_p
        L.gdn_validate.argtypes = [SP]
        L.gdn_validate.restype = I
        L.gdn_workspace_size.argtypes = [SP, ctypes.POINTER(SZ)]
        L.gdn_workspace_size.restype = I
        L.gdn_workspace_size_varlen.argtypes = [SP, ctypes.POINTER(SZ)]
        L.gdn_workspace_size_varlen.restype = I
        L.gdn_chunk_fwd_varlen.argtypes = [SP] + [P] * 10 + [SZ, P]
        L.gdn_chunk_fwd_varlen.restype = I
        L.gdn_chunk_fwd.argtypes = [SP] + [P] * 9 + [SZ, P]
        L.gdn_chunk_fwd.restype = I
        L.gdn_chunk_fwd_stages.argtypes = [SP, I] + [P] * 9 + [SZ, P]
        L.gdn_chunk_fwd_stages.restype = I
        L.gdn_chunk_fwd_timed.argtypes = [SP, I] + [P] * 9 + [SZ, P, P, P]
        L.gdn_chunk_fwd_timed.restype = I
        L.gdn_chunk_fold.argtypes = [SP] + [P] * 7 + [SZ, P]
        L.gdn_chunk_fold.restype = I
        L.gdn_compose_prefix.argtypes = [I, I, I, I] + [P] * 5 + [I, P]
        L.gdn_compose_prefix.restype = I
        L.gdn_chunk_transform.argtypes = [SP] + [P] * 8 + [P]
        L.gdn_chunk_transform.restype = I
        L.gdn_chunk_fwd_noalloc.argtypes = [SP] + [P] * 9
        L.gdn_chunk_fwd_noalloc.restype = I
        L.gdn_chunk_fwd_affine.argtypes = [SP] + [P] * 10 + [SZ, P]
        L.gdn_chunk_fwd_affine.restype = I
        L.gdn_workspace_size_bwd.argtypes = [SP, ctypes.POINTER(SZ)]
        L.gdn_workspace_size_bwd.restype = I
        L.gdn_chunk_bwd_state.argtypes = [SP] + [P] * 9 + [SZ, P]
        L.gdn_chunk_bwd_state.restype = I
        L.gdn_workspace_size_bwd_grads.argtypes = [SP, ctypes.POINTER(SZ)]
        L.gdn_workspace_size_bwd_grads.restype = I
        L.gdn_chunk_bwd.argtypes = [SP] + [P] * 15 + [SZ, P]
        L.gdn_chunk_bwd.restype = I
        PP = ctypes.POINTER(GdnPoolShape)
        L.gdn_step.argtypes = [PP] + [P] * 9
        L.gdn_step.restype = I
        L.gdn_tree_fwd.argtypes = [PP] + [P] * 11
        L.gdn_tree_fwd.restype = I
        L.gdn_tree_commit.argtypes = [PP] + [P] * 8
        L.gdn_tree_commit.restype = I
        LP = ctypes.POINTER(GdnLinearShape)
        L.gdn_workspace_size_linear.argtypes = [LP, I, ctypes.POINTER(SZ)]
        L.gdn_workspace_size_linear.restype = I
        L.gdn_linear_chunk_fwd.argtypes = [LP] + [P] * 8 + [SZ, P]
        L.gdn_linear_chunk_fwd.restype = I
        L.gdn_linear_chunk_fwd_varlen.argtypes = [LP] + [P] * 9 + [SZ, P]
        L.gdn_linear_chunk_fwd_varlen.restype = I
        L.gdn_linear_chunk_bwd.argtypes = [LP] + [P] * 13 + [SZ, P]
        L.gdn_linear_chunk_bwd.restype = I
        _lib = L
    return _lib


def _check(st: int, where: str):
    if st != 0:
        raise GdnError(st, where)


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t}")


def make_shape(B, T, H_qk, H_v, d_k=128, d_v=128, chunk=128, n_groups=0,
               dtype=torch.bfloat16, o_dtype=torch.float32) -> GdnShape:
    return GdnShape(B, T, H_qk, H_v, d_k, d_v, chunk, n_groups, _dt(dtype), _dt(o_dtype))


def validate(shape: GdnShape) -> int:
    """Host-only check; returns the status code (0 = supported)."""
    return int(lib().gdn_validate(ctypes.byref(shape)))


def workspace_size(shape: GdnShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_size(ctypes.byref(shape), ctypes.byref(n)), "gdn_workspace_size")
    return int(n.value)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _inputs(q, k, v, g, beta):
    B, T, Hqk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = k.device
    if q is not None:
        _need(q, "q", k.dtype, (B, T, Hqk, dk), dev)
    _need(k, "k", None, None, dev)
    _need(v, "v", k.dtype, (B, T, Hv, dv), dev)
    _need(g, "g", torch.float32, (B, T, Hv), dev)
    _need(beta, "beta", torch.float32, (B, T, Hv), dev)
    return B, T, Hqk, Hv, dk, dv, dev


def chunk_fwd(q, k, v, g, beta, h0=None, chunk=128, n_groups=0, o_dtype=torch.float32,
              output_final_state=True, workspace=None, out=None, final_state=None, stream=None,
              stages=None, events=None):
    """Gated DeltaNet chunked forward (gdn_chunk_fwd; gdn_chunk_fwd_stages when
    ``stages`` is a mask of STAGE_* bits; gdn_chunk_fwd_timed when ``events`` =
    (starts, stops) gives, per stage bit b = 0..4, timing torch.cuda.Event
    objects (already recorded once, so that they exist) or None).

    q, k [B,T,H_qk,d_k]; v [B,T,H_v,d_v] (bf16 or fp32); g, beta [B,T,H_v] fp32;
    h0 [B,H_v,d_k,d_v] fp32 or None.  Returns (o [B,T,H_v,d_v] o_dtype, h_T or None)."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(q, k, v, g, beta)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, n_groups, k.dtype, o_dtype)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, Hv, dk, dv), dev)
    need = workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    o = out if out is not None else torch.empty((B, T, Hv, dv), dtype=o_dtype, device=dev)
    _need(o, "o", o_dtype, (B, T, Hv, dv), dev)
    hT = None
    if output_final_state:
        hT = final_state if final_state is not None else torch.empty((B, Hv, dk, dv),
                                                                    dtype=torch.float32, device=dev)
        _need(hT, "h_T", torch.float32, (B, Hv, dk, dv), dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT),
            _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream))
    if events is not None:
        arr = [(ctypes.c_void_p * 5)(*[e.cuda_event if e is not None else None for e in evs])
               for evs in events]
        _check(lib().gdn_chunk_fwd_timed(ctypes.byref(shape), int(STAGE_ALL if stages is None else stages),
                                         *args, arr[0], arr[1]), "gdn_chunk_fwd_timed")
    elif stages is None:
        _check(lib().gdn_chunk_fwd(ctypes.byref(shape), *args), "gdn_chunk_fwd")
    else:
        _check(lib().gdn_chunk_fwd_stages(ctypes.byref(shape), int(stages), *args),
               "gdn_chunk_fwd_stages")
    return o, hT


NOALLOC_SCRATCH_BYTES = 256 << 20


def chunk_fwd_noalloc(q, k, v, g, beta, h0, out, final_state=None, chunk=128, n_groups=0,
                      stream=None):
    """gdn_chunk_fwd_noalloc: the forward with the library's static device
    scratch as its workspace (nothing is allocated by the library; the caller
    passes the outputs).  out [B,T,H_v,d_v] (fp32 or bf16: the output dtype),
    final_state [B,H_v,d_k,d_v] fp32 or None.  Returns (out, final_state)."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(q, k, v, g, beta)
    _need(out, "o", None, (B, T, Hv, dv), dev)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, n_groups, k.dtype, out.dtype)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, Hv, dk, dv), dev)
    if final_state is not None:
        _need(final_state, "h_T", torch.float32, (B, Hv, dk, dv), dev)
    _check(lib().gdn_chunk_fwd_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                       _ptr(h0), _ptr(out), _ptr(final_state), _stream(stream)),
           "gdn_chunk_fwd_noalloc")
    return out, final_state


def chunk_fwd_affine(q, k, v, g, beta, h0=None, chunk=128, o_dtype=torch.float32, workspace=None,
                     out=None, final_state=None, affine=None, stream=None):
    """The forward that also returns the affine map of the whole sequence
    (gdn_chunk_fwd_affine): (o, h_T, A) with A [B,H_v,d_k,d_k] fp32 and
    h_T = A h0 + B (B = h_T when h0 is None)."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(q, k, v, g, beta)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, 0, k.dtype, o_dtype)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, Hv, dk, dv), dev)
    need = workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    o = out if out is not None else torch.empty((B, T, Hv, dv), dtype=o_dtype, device=dev)
    _need(o, "o", o_dtype, (B, T, Hv, dv), dev)
    hT = final_state if final_state is not None else torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev)
    _need(hT, "h_T", torch.float32, (B, Hv, dk, dv), dev)
    A = affine if affine is not None else torch.empty((B, Hv, dk, dk), dtype=torch.float32, device=dev)
    _need(A, "A", torch.float32, (B, Hv, dk, dk), dev)
    _check(lib().gdn_chunk_fwd_affine(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                      _ptr(h0), _ptr(o), _ptr(hT), _ptr(A), _ptr(workspace),
                                      ctypes.c_size_t(workspace.numel()), _stream(stream)),
           "gdn_chunk_fwd_affine")
    return o, hT, A


def chunk_bwd_state(q, k, g, beta, dO, dh_T=None, chunk=128, want_chunks=True, workspace=None, stream=None):
    """The chunked backward's state cotangents (gdn_chunk_bwd_state): the
    reverse chunk walk dh_n = e^{G_last} dh_{n+1} - W^T (K_g dh_{n+1}) + ddh_n
    from dh_T.  q, k [B,T,H_qk,d_k]; g, beta [B,T,H_v] fp32; dO [B,T,H_v,d_v]
    fp32; dh_T [B,H_v,d_k,d_v] fp32 or None.  Returns (dh_chunks
    [B,H_v,N,d_k,d_v] or None, dh0 [B,H_v,d_k,d_v])."""
    B, T, Hqk, dk = k.shape
    Hv, dv = dO.shape[2], dO.shape[3]
    dev = k.device
    _need(q, "q", k.dtype, (B, T, Hqk, dk), dev)
    _need(k, "k", None, None, dev)
    _need(g, "g", torch.float32, (B, T, Hv), dev)
    _need(beta, "beta", torch.float32, (B, T, Hv), dev)
    _need(dO, "dO", torch.float32, (B, T, Hv, dv), dev)
    if dh_T is not None:
        _need(dh_T, "dh_T", torch.float32, (B, Hv, dk, dv), dev)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, 0, k.dtype, torch.float32)
    n = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_size_bwd(ctypes.byref(shape), ctypes.byref(n)), "gdn_workspace_size_bwd")
    if workspace is None:
        workspace = torch.empty(max(int(n.value), 1), dtype=torch.uint8, device=dev)
    N = -(-T // chunk)
    dhc = torch.empty((B, Hv, N, dk, dv), dtype=torch.float32, device=dev) if want_chunks else None
    dh0 = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev)
    _check(lib().gdn_chunk_bwd_state(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(g), _ptr(beta), _ptr(dO),
                                     _ptr(dh_T), _ptr(dhc), _ptr(dh0), _ptr(workspace),
                                     ctypes.c_size_t(workspace.numel()), _stream(stream)),
           "gdn_chunk_bwd_state")
    return dhc, dh0


def workspace_size_bwd_grads(shape: GdnShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_size_bwd_grads(ctypes.byref(shape), ctypes.byref(n)), "gdn_workspace_size_bwd_grads")
    return int(n.value)


def chunk_bwd(q, k, v, g, beta, dO, h0=None, dh_T=None, chunk=128, workspace=None, out=None, stream=None):
    """Gradients of sum_t <o_t, dO_t> + <h_T, dh_T> through the chunked
    forward (gdn_chunk_bwd).  q, k [B,T,H_qk,d_k]; v [B,T,H_v,d_v]; g, beta
    [B,T,H_v] fp32; dO [B,T,H_v,d_v] fp32; h0, dh_T [B,H_v,d_k,d_v] fp32 or
    None.  Returns a dict of fp32 tensors dq, dk [B,T,H_qk,d_k], dv
    [B,T,H_v,d_v], dg, dbeta [B,T,H_v], dh0 [B,H_v,d_k,d_v] (``out``: such a
    dict to write into)."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(q, k, v, g, beta)
    _need(dO, "dO", torch.float32, (B, T, Hv, dv), dev)
    for name, x in (("h0", h0), ("dh_T", dh_T)):
        if x is not None:
            _need(x, name, torch.float32, (B, Hv, dk, dv), dev)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, 0, q.dtype, torch.float32)
    if workspace is None:
        workspace = torch.empty(max(workspace_size_bwd_grads(shape), 1), dtype=torch.uint8, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    want = dict(dq=(B, T, Hqk, dk), dk=(B, T, Hqk, dk), dv=(B, T, Hv, dv), dg=(B, T, Hv), dbeta=(B, T, Hv),
                dh0=(B, Hv, dk, dv))
    if out is None:
        out = {kk: torch.empty(sh, **f32) for kk, sh in want.items()}
    for kk, sh in want.items():
        _need(out[kk], kk, torch.float32, sh, dev)
    _check(lib().gdn_chunk_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                               _ptr(dO), _ptr(dh_T), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]),
                               _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]), _ptr(workspace),
                               ctypes.c_size_t(workspace.numel()), _stream(stream)), "gdn_chunk_bwd")
    return out


def workspace_size_varlen(shape: GdnShape) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_size_varlen(ctypes.byref(shape), ctypes.byref(n)), "gdn_workspace_size_varlen")
    return int(n.value)


def chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, h0=None, chunk=128, o_dtype=torch.float32,
                     output_final_state=True, workspace=None, out=None, final_state=None, stream=None):
    """Chunked forward over packed variable-length sequences
    (gdn_chunk_fwd_varlen).  q, k [1,T,H_qk,d_k]; v [1,T,H_v,d_v]; g, beta
    [1,T,H_v]; cu_seqlens int32 [n+1] on the device, or a Python sequence of
    the n+1 offsets (sequence s = tokens cu[s]..cu[s+1]); h0 [n,H_v,d_k,d_v]
    or None.  Returns (o, h_T [n,...] or None)."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(q, k, v, g, beta)
    if B != 1:
        raise ValueError("packed sequences: the batch dimension of q, k, v, g, beta must be 1")
    if not isinstance(cu_seqlens, torch.Tensor):   # a sequence of offsets
        cu_seqlens = torch.tensor(list(cu_seqlens), dtype=torch.int32, device=dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, None, dev)
    nseq = cu_seqlens.numel() - 1
    if nseq < 1:
        raise ValueError("cu_seqlens must hold at least two offsets")
    shape = make_shape(nseq, T, Hqk, Hv, dk, dv, chunk, 0, k.dtype, o_dtype)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (nseq, Hv, dk, dv), dev)
    need = workspace_size_varlen(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    o = out if out is not None else torch.empty((1, T, Hv, dv), dtype=o_dtype, device=dev)
    _need(o, "o", o_dtype, (1, T, Hv, dv), dev)
    hT = None
    if output_final_state:
        hT = final_state if final_state is not None else torch.empty((nseq, Hv, dk, dv),
                                                                    dtype=torch.float32, device=dev)
        _need(hT, "h_T", torch.float32, (nseq, Hv, dk, dv), dev)
    _check(lib().gdn_chunk_fwd_varlen(ctypes.byref(shape), _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                      _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT), _ptr(workspace),
                                      ctypes.c_size_t(workspace.numel()), _stream(stream)),
           "gdn_chunk_fwd_varlen")
    return o, hT


def chunk_fold(k, v, g, beta, n_groups, chunk=128, workspace=None, stream=None):
    """Per-group affine pairs (gdn_chunk_fold): A [B,H_v,G,d_k,d_k], Bm [B,H_v,G,d_k,d_v]."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(None, k, v, g, beta)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, n_groups, k.dtype, torch.float32)
    Gn = max(int(n_groups), 1)
    need = workspace_size(shape)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    A = torch.empty((B, Hv, Gn, dk, dk), dtype=torch.float32, device=dev)
    Bm = torch.empty((B, Hv, Gn, dk, dv), dtype=torch.float32, device=dev)
    st = lib().gdn_chunk_fold(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(A),
                              _ptr(Bm), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                              _stream(stream))
    _check(st, "gdn_chunk_fold")
    return A, Bm


def compose_prefix(A, Bm, h_init=None, split_bf16=False, want_h_in=True, stream=None, form=None):
    """Exclusive prefix of affine pairs (gdn_compose_prefix).  ``form``: None
    lets the library choose, "sequential" or "blocked" force one.
    A [BH,n,d_k,d_k], Bm [BH,n,d_k,d_v] fp32; h_init [BH,d_k,d_v] or None.
    Returns (h_in [BH,n,d_k,d_v] or None, h_final [BH,d_k,d_v])."""
    BH, n, dk, _ = A.shape
    dv = Bm.shape[3]
    dev = A.device
    _need(A, "A", torch.float32, None, dev)
    _need(Bm, "Bm", torch.float32, (BH, n, dk, dv), dev)
    if h_init is not None:
        _need(h_init, "h_init", torch.float32, (BH, dk, dv), dev)
    h_in = torch.empty((BH, n, dk, dv), dtype=torch.float32, device=dev) if want_h_in else None
    h_fin = torch.empty((BH, dk, dv), dtype=torch.float32, device=dev)
    st = lib().gdn_compose_prefix(BH, n, dk, dv, _ptr(A), _ptr(Bm), _ptr(h_init), _ptr(h_in),
                                  _ptr(h_fin), (PREFIX_SPLIT_BF16 if split_bf16 else 0) |
                                  {None: 0, "sequential": PREFIX_SEQUENTIAL,
                                   "blocked": PREFIX_BLOCKED}[form],
                                  _stream(stream))
    _check(st, "gdn_compose_prefix")
    return h_in, h_fin


def chunk_transform(k, v, g, beta, chunk=128, want_T=False, stream=None):
    """Intra-chunk transform (gdn_chunk_transform): G [B,H_v,N,C], T [B,H_v,N,C,C] or None,
    W [B,H_v,N,C,d_k], U [B,H_v,N,C,d_v], all fp32."""
    B, T, Hqk, Hv, dk, dv, dev = _inputs(None, k, v, g, beta)
    shape = make_shape(B, T, Hqk, Hv, dk, dv, chunk, 0, k.dtype, torch.float32)
    _check(validate(shape), "gdn_chunk_transform")
    N = -(-T // chunk)   # a partial last chunk is padded with identity steps
    f = dict(dtype=torch.float32, device=dev)
    G = torch.empty((B, Hv, N, chunk), **f)
    Tm = torch.empty((B, Hv, N, chunk, chunk), **f) if want_T else None
    W = torch.empty((B, Hv, N, chunk, dk), **f)
    U = torch.empty((B, Hv, N, chunk, dv), **f)
    st = lib().gdn_chunk_transform(ctypes.byref(shape), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                   _ptr(G), _ptr(Tm), _ptr(W), _ptr(U), _stream(stream))
    _check(st, "gdn_chunk_transform")
    return G, Tm, W, U


# ---------------------------------------------------------------------------
# states in a pool: the single-token step, drafted trees


# The current stream's handle of a device, without building a Stream object
# (a single-token step takes the GPU a few microseconds: so may its checks).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """A call on a stream of the caller's, or on a device that is not the
    current one (which is made current for the launch).  Outputs and workspace
    allocated inside belong to that stream."""
    __slots__ = ("dev", "ctx")

    def __init__(self, dev, stream):
        if stream is not None and stream.device != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
        self.dev = dev
        self.ctx = torch.cuda.device(dev) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()
        return _raw_stream(self.dev.index)

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


class _Here:
    """The current stream of the current device."""
    __slots__ = ("handle",)

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        pass


def _on(dev, stream):
    """Context of a launch: enters the stream the call goes to (``stream``, or
    the current stream of the tensors' device) and gives its handle."""
    index = dev.index
    if stream is None and index == torch.cuda.current_device():
        return _Here(_raw_stream(index))
    return _On(dev, stream)


def _check_tensors(dev, *items):
    """Each item: (tensor, name, dtype, shape); raises what _need raises."""
    index = dev.index
    for t, name, dtype, shape in items:
        if not (type(t) is torch.Tensor and t.get_device() == index and t.dtype is dtype and t.shape == shape
                and t.is_contiguous()):
            _need(t, name, dtype, shape, dev)   # (a subclass of Tensor that fits passes here)


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_apart(outputs, inputs):
    """Outputs (and a workspace) that the caller passed must lie apart from
    the inputs and from each other: workgroups that still read an input run
    beside those that write.  Both are (tensor or None, name) pairs of
    contiguous tensors."""
    def span(t, name):
        at = t.data_ptr()
        return at, at + t.numel() * t.element_size(), name

    taken = [span(t, name) for t, name in inputs if t is not None and t.numel()]
    for t, name in outputs:
        if t is None or not t.numel():
            continue
        lo, hi, _ = here = span(t, name)
        for a, b, other in taken:
            if a < hi and lo < b:
                raise ValueError(f"{name} overlaps {other}")
        taken.append(here)


@functools.lru_cache(maxsize=256)
def _pool_shape(*sizes):
    return GdnPoolShape(*sizes)


def _pool_dims(k, Hv_of, state, slots, lead):
    """Sizes of a call on a pool, and what is to be checked of k, the pool and
    the slots; ``lead``: leading dimensions before the heads (1: rows, 2: rows
    and nodes)."""
    if not isinstance(k, torch.Tensor) or not isinstance(Hv_of, torch.Tensor) or not isinstance(state, torch.Tensor):
        raise TypeError("k, v (u) and state must be tensors")
    ks, vs, ss = k.shape, Hv_of.shape, state.shape
    if len(ks) != lead + 2 or len(vs) != lead + 2 or len(ss) != 4:
        raise ValueError(f"k and v (u) must have {lead + 2} dimensions and state 4")
    dt = k.dtype
    _dt(dt)
    Hv, dv, dk = vs[-2], vs[-1], ks[-1]
    items = [(k, "k", dt, ks), (state, "state", torch.float32, (ss[0], Hv, dk, dv))]
    if slots is not None:
        items.append((slots, "slots", torch.int32, ks[:1]))
    return ks[0], (ks[1] if lead == 2 else 1), ks[-2], Hv, dk, dv, ss[0], k.device, items


def _decay_shape(g, per_token):
    return (1, per_token[-1:]) if isinstance(g, torch.Tensor) and g.dim() == 1 else (0, per_token)


def step(q, k, v, g, beta, state, slots=None, o_dtype=torch.float32, out=None, stream=None):
    """One token of every row (gdn_step): the recurrent form, for decoding.

    q, k [B,H_qk,d_k]; v [B,H_v,d_v] (bf16 or fp32); g [B,H_v] or [H_v] fp32;
    beta [B,H_v] fp32, or None for the linear rule (S = e^g S + k v^T); state
    [n_slots,H_v,d_k,d_v] fp32, advanced in place; slots [B] int32 on the
    device (None: row b has slot b).  A row whose slot is outside the pool,
    or is an earlier row's slot, gets a zero output and writes no state.
    Returns o [B,H_v,d_v] o_dtype."""
    B, n, Hqk, Hv, dk, dv, n_slots, dev, items = _pool_dims(k, v, state, slots, 1)
    fixed, gshape = _decay_shape(g, (B, Hv))
    items += ((q, "q", k.dtype, (B, Hqk, dk)), (v, "v", k.dtype, (B, Hv, dv)), (g, "g", torch.float32, gshape))
    if beta is not None:
        items.append((beta, "beta", torch.float32, (B, Hv)))
    if out is not None:
        items.append((out, "o", o_dtype, (B, Hv, dv)))
    _check_tensors(dev, *items)
    if out is not None:
        _check_apart(((out, "o"),), ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (state, "state"), (slots, "slots")))
    shape = _pool_shape(B, 1, Hqk, Hv, dk, dv, n_slots, fixed, _dt(k.dtype), _dt(o_dtype))
    with _on(dev, stream) as st:
        o = out if out is not None else torch.empty((B, Hv, dv), dtype=o_dtype, device=dev)
        _check(lib().gdn_step(shape, _addr(q), _addr(k), _addr(v), _addr(g), _addr(beta), _addr(slots), _addr(state),
                              _addr(o), st), "gdn_step")
    return o


def tree_fwd(q, k, v, g, beta, parents, state, slots=None, o_dtype=torch.float32, out=None, values=None, stream=None):
    """The check of a tree of drafted tokens (gdn_tree_fwd): every node's
    output from its parent's state; the pool is only read.

    q, k [B,n,H_qk,d_k]; v [B,n,H_v,d_v]; g [B,n,H_v] or [H_v] fp32; beta
    [B,n,H_v] fp32 or None (the linear rule); parents [B,n] int32: an earlier
    node, or -1 for the row's state (any other value: an absent node, zero
    outputs); n <= 64; state [n_slots,H_v,d_k,d_v] fp32; slots as in step (rows
    may share a slot).  Returns (o [B,n,H_v,d_v] o_dtype, u [B,n,H_v,d_v] fp32,
    the values the nodes write, for tree_commit)."""
    B, n, Hqk, Hv, dk, dv, n_slots, dev, items = _pool_dims(k, v, state, slots, 2)
    fixed, gshape = _decay_shape(g, (B, n, Hv))
    items += ((q, "q", k.dtype, (B, n, Hqk, dk)), (v, "v", k.dtype, (B, n, Hv, dv)),
              (g, "g", torch.float32, gshape), (parents, "parents", torch.int32, (B, n)))
    if beta is not None:
        items.append((beta, "beta", torch.float32, (B, n, Hv)))
    if out is not None:
        items.append((out, "o", o_dtype, (B, n, Hv, dv)))
    if values is not None:
        items.append((values, "u", torch.float32, (B, n, Hv, dv)))
    _check_tensors(dev, *items)
    if not (out is None and values is None):
        _check_apart(((out, "o"), (values, "u")),
                     ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta"), (parents, "parents"), (state, "state"),
                      (slots, "slots")))
    shape = _pool_shape(B, n, Hqk, Hv, dk, dv, n_slots, fixed, _dt(k.dtype), _dt(o_dtype))
    with _on(dev, stream) as st:
        o = out if out is not None else torch.empty((B, n, Hv, dv), dtype=o_dtype, device=dev)
        u = values if values is not None else torch.empty((B, n, Hv, dv), dtype=torch.float32, device=dev)
        _check(lib().gdn_tree_fwd(shape, _addr(q), _addr(k), _addr(v), _addr(g), _addr(beta), _addr(parents),
                                  _addr(slots), _addr(state), _addr(o), _addr(u), st), "gdn_tree_fwd")
    return o, u


def tree_commit(k, u, g, parents, last, state, slots=None, stream=None):
    """The commit of an accepted path (gdn_tree_commit): row b's state becomes
    the state of node last[b], in place (last[b] outside the tree, or an absent
    node: nothing is committed and the state is left as it is).  k, g, parents
    as given to tree_fwd, u as returned by it; last [B] int32.  Rows naming one
    slot: the first one that commits a node is run.  Returns state."""
    B, n, Hqk, Hv, dk, dv, n_slots, dev, items = _pool_dims(k, u, state, slots, 2)
    fixed, gshape = _decay_shape(g, (B, n, Hv))
    _check_tensors(dev, *items, (u, "u", torch.float32, (B, n, Hv, dv)), (g, "g", torch.float32, gshape),
                   (parents, "parents", torch.int32, (B, n)), (last, "last", torch.int32, (B,)))
    shape = _pool_shape(B, n, Hqk, Hv, dk, dv, n_slots, fixed, _dt(k.dtype), F32)
    with _on(dev, stream) as st:
        _check(lib().gdn_tree_commit(shape, _addr(k), _addr(u), _addr(g), _addr(parents), _addr(last), _addr(slots),
                                     _addr(state), st), "gdn_tree_commit")
    return state


# ---------------------------------------------------------------------------
# linear attention with a decay per head, in chunks

LINEAR_FWD, LINEAR_VARLEN, LINEAR_BWD = 0, 1, 2


@functools.lru_cache(maxsize=256)
def _linear_plan(kind, *sizes):
    """(shape, workspace bytes) of a call's sizes."""
    shape = GdnLinearShape(*sizes)
    return shape, workspace_size_linear(shape, kind)


def workspace_size_linear(shape: GdnLinearShape, kind: int) -> int:
    """Workspace bytes of linear_chunk_fwd (LINEAR_FWD), linear_chunk_fwd_varlen
    (LINEAR_VARLEN; shape.B = sequences) or linear_chunk_bwd (LINEAR_BWD)."""
    n = ctypes.c_size_t(0)
    _check(lib().gdn_workspace_size_linear(shape, kind, ctypes.byref(n)), "gdn_workspace_size_linear")
    return int(n.value)


def _linear_inputs(q, k, v, g):
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (g, "g")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must have 4 dimensions")
    _dt(k.dtype)
    B, T, Hqk, dk = k.shape
    Hv, dv = v.shape[2:]
    dev = k.device
    fixed, gshape = _decay_shape(g, (B, T, Hv))
    _check_tensors(dev, (q, "q", k.dtype, (B, T, Hqk, dk)), (k, "k", k.dtype, k.shape), (v, "v", k.dtype, (B, T, Hv, dv)),
                   (g, "g", torch.float32, gshape))
    return B, T, Hqk, Hv, dk, dv, fixed, dev


def _linear_fwd(rows, cu, q, k, v, g, h0, o_dtype, output_final_state, workspace, out, final_state, stream):
    B, T, Hqk, Hv, dk, dv, fixed, dev = _linear_inputs(q, k, v, g)
    n = B if rows is None else rows
    state = (n, Hv, dk, dv)
    if h0 is not None:
        _check_tensors(dev, (h0, "h0", torch.float32, state))
    if out is not None:
        _check_tensors(dev, (out, "o", o_dtype, (B, T, Hv, dv)))
    if final_state is not None:
        _check_tensors(dev, (final_state, "h_T", torch.float32, state))
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, None, dev)
    if not (out is None and final_state is None and workspace is None):
        _check_apart(((out, "o"), (final_state, "h_T"), (workspace, "workspace")),
                     ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (h0, "h0"), (cu, "cu_seqlens")))
    shape, need = _linear_plan(LINEAR_FWD if rows is None else LINEAR_VARLEN, n, T, Hqk, Hv, dk, dv, fixed, _dt(k.dtype),
                               _dt(o_dtype))
    with _on(dev, stream) as st:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev) if workspace is None else workspace
        o = out if out is not None else torch.empty((B, T, Hv, dv), dtype=o_dtype, device=dev)
        hT = None
        if output_final_state:
            hT = final_state if final_state is not None else torch.empty(state, dtype=torch.float32, device=dev)
        args = (_addr(q), _addr(k), _addr(v), _addr(g), _addr(h0), _addr(o), _addr(hT), _addr(ws), ws.numel(), st)
        if rows is None:
            _check(lib().gdn_linear_chunk_fwd(shape, *args), "gdn_linear_chunk_fwd")
        else:
            _check(lib().gdn_linear_chunk_fwd_varlen(shape, _addr(cu), *args), "gdn_linear_chunk_fwd_varlen")
    return o, hT


def linear_chunk_fwd(q, k, v, g, h0=None, o_dtype=torch.float32, output_final_state=True, workspace=None, out=None,
                     final_state=None, stream=None):
    """Linear attention with a decay per head (gdn_linear_chunk_fwd):
    S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

    q, k [B,T,H_qk,d_k]; v [B,T,H_v,d_v] (bf16 or fp32); g [B,T,H_v] fp32, or
    [H_v] for decays that do not depend on the token; h0 [B,H_v,d_k,d_v] fp32
    or None.  Returns (o [B,T,H_v,d_v] o_dtype, h_T or None)."""
    return _linear_fwd(None, None, q, k, v, g, h0, o_dtype, output_final_state, workspace, out, final_state, stream)


def linear_chunk_fwd_varlen(q, k, v, g, cu_seqlens, h0=None, o_dtype=torch.float32, output_final_state=True,
                            workspace=None, out=None, final_state=None, stream=None):
    """linear_chunk_fwd over packed sequences (gdn_linear_chunk_fwd_varlen):
    the batch dimension of q, k, v (and g) is 1; cu_seqlens as in
    chunk_fwd_varlen (n + 1 int32 offsets on the device, or a Python
    sequence); h0 and h_T [n,H_v,d_k,d_v]."""
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a tensor")
    if k.dim() == 4 and k.shape[0] != 1:
        raise ValueError("packed sequences: the batch dimension of q, k, v, g must be 1")
    if not isinstance(cu_seqlens, torch.Tensor):
        if not k.is_cuda:
            raise ValueError("k must be a device tensor")
        # on the call's stream, so that the memory is not given to other work
        # of the current stream while the call still reads it
        with _on(k.device, stream):
            cu_seqlens = torch.tensor(list(cu_seqlens), dtype=torch.int32, device=k.device)
    n = cu_seqlens.numel() - 1
    if n < 1:
        raise ValueError("cu_seqlens must hold at least two offsets")
    _check_tensors(k.device, (cu_seqlens, "cu_seqlens", torch.int32, (n + 1,)))
    return _linear_fwd(n, cu_seqlens, q, k, v, g, h0, o_dtype, output_final_state, workspace, out, final_state, stream)


def linear_chunk_bwd(q, k, v, g, dO, h0=None, dh_T=None, workspace=None, out=None, stream=None):
    """Gradients of sum_t <o_t, dO_t> + <h_T, dh_T> through linear_chunk_fwd
    (gdn_linear_chunk_bwd).  dO [B,T,H_v,d_v] in the inputs' dtype; h0, dh_T
    [B,H_v,d_k,d_v] fp32 or None.  Returns a dict (``out``: such a dict to
    write into): dq, dk [B,T,H_qk,d_k], dv [B,T,H_v,d_v] in the inputs' dtype,
    dg fp32 shaped as g, dh0 [B,H_v,d_k,d_v] fp32."""
    B, T, Hqk, Hv, dk, dv, fixed, dev = _linear_inputs(q, k, v, g)
    state = (B, Hv, dk, dv)
    _check_tensors(dev, (dO, "dO", k.dtype, (B, T, Hv, dv)))
    for name, x in (("h0", h0), ("dh_T", dh_T)):
        if x is not None:
            _check_tensors(dev, (x, name, torch.float32, state))
    want = dict(dq=(k.dtype, (B, T, Hqk, dk)), dk=(k.dtype, (B, T, Hqk, dk)), dv=(k.dtype, (B, T, Hv, dv)),
                dg=(torch.float32, tuple(g.shape)), dh0=(torch.float32, state))
    if out is not None:
        for name, (dt, sh) in want.items():
            _check_tensors(dev, (out[name], name, dt, sh))
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, None, dev)
    if not (out is None and workspace is None):
        _check_apart([(out[name], name) for name in want if out is not None] + [(workspace, "workspace")],
                     ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (dO, "dO"), (h0, "h0"), (dh_T, "dh_T")))
    shape, need = _linear_plan(LINEAR_BWD, B, T, Hqk, Hv, dk, dv, fixed, _dt(k.dtype), F32)
    with _on(dev, stream) as st:
        ws = torch.empty(max(need, 1), dtype=torch.uint8, device=dev) if workspace is None else workspace
        if out is None:
            out = {name: torch.empty(sh, dtype=dt, device=dev) for name, (dt, sh) in want.items()}
        _check(lib().gdn_linear_chunk_bwd(shape, _addr(q), _addr(k), _addr(v), _addr(g), _addr(h0), _addr(dO),
                                          _addr(dh_T), _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]),
                                          _addr(out["dg"]), _addr(out["dh0"]), _addr(ws), ws.numel(), st),
               "gdn_linear_chunk_bwd")
    return out
