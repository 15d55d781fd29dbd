"""The gated block's operators (``include/mg_block.h``): a gated linear
recurrence whose state is a matrix per head, and the root-mean-square norm with
the residual's addition, for prompts, for training and for single tokens.

* ``gated_scan_fwd(q, k, v, g, S0=None, scale=1.0) -> (o, S_last, saved)``,
  ``gated_scan_bwd(do, saved, q, k, v, g, S0=None, dS_last=None, ...) -> (dq, dk, dv, dg, dS0)``,
  ``gated_scan_step(q, k, v, g, state, slots=None, scale=1.0) -> o``
* ``rms_norm_fwd(x, w, residual=None, eps=1e-5) -> (y, r, rstd)``,
  ``rms_norm_quant(x, w, residual=None, eps=1e-5, block=None) -> (q, scale, r)``,
  ``rms_norm_bwd(dy, rstd, r, w, dr=None) -> (dx, dw)``

Activations are float32 or bf16, all of a call the same; gates, states, norm
weights and scales are float32.  Rows, ``cu_seqlens``, ``out=``, ``ws=`` and
``stream=`` are as in ``ssm.py``.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import struct

import torch
from torch import Tensor

from . import _DT, MG_ERR_INVALID_ARG, MG_OK, _check, _workspace, load
from .ssm import _ACTIVATIONS, _CONTROL_BYTES, _F32, _new, _param, _rows, _sequences, _slots, _state, _stream

__all__ = [
    "mg_gated_scan_fwd", "mg_gated_scan_bwd", "mg_gated_scan_step",
    "mg_rms_norm_fwd", "mg_rms_norm_quant", "mg_rms_norm_bwd",
    "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step",
    "rms_norm_fwd", "rms_norm_quant", "rms_norm_bwd",
]

SYMBOLS = (
    "mg_gated_scan_workspace_size", "mg_gated_scan_saved_size", "mg_gated_scan_fwd",
    "mg_gated_scan_bwd", "mg_gated_scan_step", "mg_rms_norm_workspace_size", "mg_rms_norm_fwd",
    "mg_rms_norm_quant", "mg_rms_norm_bwd", "mg_block_call",
)

MAX_HEAD = 128                      # values of a head's q, k and v
BLOCKS = (32, 64, 128, 256)         # channels that may share a scale
_E4M3 = torch.float8_e4m3fn


def _on_its_device(f):
    """Makes a call on its stream, where one is given, and with its first
    tensor's device current; adds the argument `stream`."""
    shown = inspect.signature(f)
    first = next(iter(shown.parameters))

    @functools.wraps(f)
    def call(*args, stream=None, **more):
        x = args[0] if args else more.get(first)
        if stream is not None:
            if isinstance(x, Tensor) and x.is_cuda and stream.device != x.device:
                raise ValueError("the stream must be on the tensors' device")
            with torch.cuda.stream(stream):
                return call(*args, **more)
        if isinstance(x, Tensor) and x.is_cuda and x.get_device() != torch.cuda.current_device():
            with torch.cuda.device(x.device):
                return f(*args, **more)
        return f(*args, **more)
    call.__signature__ = shown.replace(parameters=[*shown.parameters.values(),
                                                   inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _together(first, *others):
    """Refuses tensors of another device than the first one's."""
    at = first.get_device()
    for x in others:
        if x is not None and x.get_device() != at:
            raise ValueError("the tensors of a call must be on one device")


# The calls' argument blocks (mg_block_call): q an integer or a pointer, d a double.
_OPS = {name: (op, struct.Struct(words).pack, len(words)) for op, (name, words) in enumerate({
    "mg_gated_scan_fwd": "q" * 9 + "d" + "q" * 15, "mg_gated_scan_bwd": "q" * 12 + "d" + "q" * 17,
    "mg_gated_scan_step": "q" * 9 + "d" + "q" * 10,
    "mg_rms_norm_fwd": "q" * 6 + "d" + "q" * 6, "mg_rms_norm_quant": "q" * 6 + "d" + "q" * 7,
    "mg_rms_norm_bwd": "q" * 16,
}.items())}
_call = None


def declare(lib):
    """Argument types of the entry points of mg_block.h that are called."""
    global _call
    vp, i64, i32, sz, f64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    sizes = {"mg_gated_scan_workspace_size": [i64] * 7 + [i32] * 3,
             "mg_gated_scan_saved_size": [i64] * 6 + [i32] * 2,
             "mg_rms_norm_workspace_size": [i64] * 2}
    for name, args in sizes.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, sz
    row = [vp, i64]
    calls = {
        "mg_gated_scan_fwd": row * 4 + [i32, f64, vp, vp, i64, vp, vp, vp] + [i64] * 6 + [vp, sz, vp],
        "mg_gated_scan_bwd": row + [vp] + row * 4 + [i32, f64, vp, vp, i64] + [vp] * 5 + [i64] * 6 + [vp, sz, vp],
        "mg_gated_scan_step": row * 4 + [i32, f64, vp, i64, vp, vp] + [i64] * 5 + [vp],
        "mg_rms_norm_fwd": row * 2 + [i32, vp, f64, vp, vp, vp, i64, i64, vp],
        "mg_rms_norm_quant": row * 2 + [i32, vp, f64, vp, vp, vp, i64, i64, i64, vp],
        "mg_rms_norm_bwd": row + [vp] + row * 2 + [i32, vp, vp, vp, i64, i64, vp, sz, vp],
    }
    for name, args in calls.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, i32
    lib.mg_block_call.argtypes, lib.mg_block_call.restype = [i32, ctypes.c_char_p, i32], i32
    _call = lib.mg_block_call


def _run(name, *words):
    """The C call `name`; `words` are its arguments."""
    op, pack, n = _OPS[name]
    st = (_call or load().mg_block_call)(op, pack(*words), n)
    if st != MG_OK:
        _check(st, name)


def _run_ws(name, need, device, ws, words, sh):
    """The C call `name` with a workspace; need() is asked only when the
    stream's cached workspace does not do."""
    op, pack, n = _OPS[name]
    buf = _workspace(_CONTROL_BYTES, device, sh, ws)
    st = (_call or load().mg_block_call)(op, pack(*words, buf.data_ptr(), buf.numel(), sh), n)
    if st == MG_ERR_INVALID_ARG and ws is None:
        size = need()
        if size > buf.numel():
            buf = _workspace(size, device, sh, None)
            st = _call(op, pack(*words, buf.data_ptr(), buf.numel(), sh), n)
    if st != MG_OK:
        _check(st, name)


# -------------------------------------------------------------- gated scan

def _scan_args(q, k, v, g, lead):
    """The arguments that the recurrence's three calls share; v has `lead`
    leading dimensions.  q and k may leave out the group dimension.  The tensors
    (kept alive until the call is made), the words of the C calls from q to
    the type, the sizes (H, G, N, P), and q's shape."""
    v, pv, ldv = _rows(v, "v", _ACTIVATIONS, 2)
    shape, ty = v.shape, v.dtype
    if len(shape) != lead + 2:
        raise ValueError("v must be (B, T, H, P)" if lead == 2 else "v must be (B, H, P)")
    H, P = shape[-2:]
    qshape = q.shape if isinstance(q, Tensor) else ()
    dims = len(qshape) - lead
    if dims not in (1, 2) or qshape[:lead] != shape[:lead] or not isinstance(k, Tensor) or k.shape != qshape:
        raise ValueError("q and k must both be v's leading dimensions and (G, N), or (N)")
    N, G = qshape[-1], qshape[-2] if dims == 2 else 1
    if not 1 <= N <= MAX_HEAD or not 1 <= P <= MAX_HEAD:
        raise ValueError(f"q, k and v must have 1 to {MAX_HEAD} values a head")
    if G < 1 or H % G:
        raise ValueError("the heads of v must be a multiple of the groups of q and k")
    q, pq, ldq = _rows(q, "q", (ty,), dims)
    k, pk, ldk = _rows(k, "k", (ty,), dims)
    g, pg, ldg = _rows(g, "g", (_F32,))
    if g.shape != shape[:-1]:
        raise ValueError("g must have v's leading dimensions and a value for each head")
    return (q, k, v, g), (pq, ldq, pk, ldk, pv, ldv, pg, ldg, _DT[ty]), (H, G, N, P), qshape


@functools.lru_cache(maxsize=256)
def _saved_numel(B, T, H, N, P, nseq, packed, dt):
    return load().mg_gated_scan_saved_size(B, T, H, N, P, nseq, packed, dt) // 4


@_on_its_device
def mg_gated_scan_fwd(q, k, v, g, S0=None, *, scale=1.0, cu_seqlens=None, save=False, out=None, ws=None):
    """(o (B,T,H,P), S_last (sequences,H,N,P), saved): per head
      S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,
    from S0.  q, k (B,T,G,N), or (B,T,N) for one group; v (B,T,H,P); N, P <=
    128; g (B,T,H) float32, the logarithms of the decays; head h reads group
    h // (H/G).  saved, with save=True, is what mg_gated_scan_bwd needs of
    this call; else None."""
    keep, words, (H, G, N, P), _ = _scan_args(q, k, v, g, 2)
    v = keep[2]
    B, T = v.shape[:2]
    cu, pcu, nseq = _sequences(cu_seqlens, v, B)
    states, packed = (nseq, H, N, P), 0 if cu is None else 1
    S0, pS0 = _param(S0, "S0", states)
    _together(v, *keep, cu, S0, ws, *(out or ()))
    o, po = _new(out, 0, v.shape, v, v.dtype)
    S_last, pl = _new(out, 1, states, v, _F32)
    saved, psv = _new(out, 2, (_saved_numel(B, T, H, N, P, nseq, packed, words[-1]),), v, _F32) if save else (None, 0)
    sh = _stream(v)
    _run_ws("mg_gated_scan_fwd",
            lambda: load().mg_gated_scan_workspace_size(B, T, H, G, N, P, nseq, packed, words[-1], 0), v.device, ws,
            (*words, float(scale), pS0, pcu, nseq, po, pl, psv, B, T, H, G, N, P), sh)
    return o, S_last, saved


@_on_its_device
def mg_gated_scan_bwd(do, saved, q, k, v, g, S0=None, dS_last=None, *, scale=1.0, cu_seqlens=None, out=None,
                      ws=None):
    """(dq, dk, dv, dg, dS0): gradients of sum(do*o) + sum(dS_last*S_last) for
    mg_gated_scan_fwd on the same inputs, with the `saved` that it returned.
    dS0 is None where S0 is."""
    keep, words, (H, G, N, P), qshape = _scan_args(q, k, v, g, 2)
    v, ty = keep[2], keep[2].dtype
    do, pdo, lddo = _rows(do, "do", (ty,), 2)
    if do.shape != v.shape:
        raise ValueError("do must have v's shape")
    B, T = v.shape[:2]
    cu, pcu, nseq = _sequences(cu_seqlens, v, B)
    states, packed = (nseq, H, N, P), 0 if cu is None else 1
    S0, _ = _param(S0, "S0", states)
    dS_last, pdl = _param(dS_last, "dS_last", states)
    if saved is None:
        raise ValueError("saved must be what mg_gated_scan_fwd returned with save=True")
    _together(v, *keep, do, cu, dS_last, saved, ws, *(out or ()))
    saved, psv = _param(saved, "saved", (_saved_numel(B, T, H, N, P, nseq, packed, words[-1]),))
    dq, pdq = _new(out, 0, qshape, v, ty)
    dk, pdk = _new(out, 1, qshape, v, ty)
    dv, pdv = _new(out, 2, v.shape, v, ty)
    dg, pdg = _new(out, 3, v.shape[:-1], v, _F32)
    dS0, pdS0 = _new(out, 4, states, v, _F32) if S0 is not None else (None, 0)
    sh = _stream(v)
    _run_ws("mg_gated_scan_bwd",
            lambda: load().mg_gated_scan_workspace_size(B, T, H, G, N, P, nseq, packed, words[-1], 1), v.device, ws,
            (pdo, lddo, psv, *words, float(scale), pdl, pcu, nseq, pdq, pdk, pdv, pdg, pdS0, B, T, H, G, N, P), sh)
    return dq, dk, dv, dg, dS0


@_on_its_device
def mg_gated_scan_step(q, k, v, g, state, *, slots=None, scale=1.0, out=None):
    """o (B,H,P): one token a row through mg_gated_scan_fwd's recurrence.  q, k
    (B,G,N) or (B,N); v (B,H,P); g (B,H).  Row i's state is state[slots[i]]
    (state[i] without slots) of (states,H,N,P) float32, updated in place; a row
    whose slot is not in the pool is idle: o 0, no state written."""
    keep, words, (H, G, N, P), _ = _scan_args(q, k, v, g, 1)
    v = keep[2]
    B = v.shape[0]
    ps = _state(state, "state", _F32, (H, N, P))
    slots, psl = _slots(slots, state, B)
    _together(v, *keep, state, slots, out)
    o, po = _new(None if out is None else (out,), 0, v.shape, v, v.dtype)
    _run("mg_gated_scan_step", *words, float(scale), ps, state.shape[0], psl, po, B, H, G, N, P, _stream(v))
    return o


# ---------------------------------------------------------------- rms norm

def _norm_in(x, w, residual, out):
    """(tensors, words from x to w, rows M, channels D)."""
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    D = x.shape[-1]
    pr, ldr = 0, D
    if residual is not None:
        if not isinstance(residual, Tensor) or residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        residual, pr, ldr = _rows(residual, "residual", (x.dtype,))
    w, pw = _param(w, "w", (D,))
    if w is None:
        raise ValueError("w must be (D,)")
    _together(x, residual, w, *(out or ()))
    return (x, residual, w), (px, ldx, pr, ldr, _DT[x.dtype], pw), x.shape[:-1].numel(), D


@_on_its_device
def mg_rms_norm_fwd(x, w, residual=None, *, eps=1e-5, out=None):
    """(y, r, rstd): r = x + residual, rounded to x's type (x itself without a
    residual), y = r w / sqrt(mean(r^2) + eps) over the last dimension, of at
    most 16384 channels.  rstd (x's leading dimensions) is for
    mg_rms_norm_bwd.  out's r may be the residual."""
    (x, res, w), words, M, D = _norm_in(x, w, residual, out)
    y, py = _new(out, 0, x.shape, x, x.dtype)
    r, pr = _new(out, 1, x.shape, x, x.dtype) if res is not None else (x, 0)
    rstd, ps = _new(out, 2, x.shape[:-1], x, _F32)
    _run("mg_rms_norm_fwd", *words, float(eps), py, pr, ps, M, D, _stream(x))
    return y, r, rstd


@_on_its_device
def mg_rms_norm_quant(x, w, residual=None, *, eps=1e-5, block=None, out=None):
    """(q, scale, r): mg_rms_norm_fwd's y in 8 bits, q = y / scale rounded to
    float8_e4m3fn, with scale = max(largest |y|, 1e-30) / 448 of each block of
    32, 64, 128 or 256 channels (None: of the row), scale (..., D/block)."""
    (x, res, w), words, M, D = _norm_in(x, w, residual, out)
    if block is not None and (block not in BLOCKS or D % block):
        raise ValueError(f"block must be one of {BLOCKS} and divide the channels, or None")
    q, pq = _new(out, 0, x.shape, x, _E4M3)
    scale, ps = _new(out, 1, (*x.shape[:-1], D // block if block else 1), x, _F32)
    r, pr = _new(out, 2, x.shape, x, x.dtype) if res is not None else (x, 0)
    _run("mg_rms_norm_quant", *words, float(eps), pq, ps, pr, block or 0, M, D, _stream(x))
    return q, scale, r


@_on_its_device
def mg_rms_norm_bwd(dy, rstd, r, w, dr=None, *, out=None, ws=None):
    """(dx, dw): gradients of sum(dy*y) + sum(dr*r) for mg_rms_norm_fwd, from
    the r and rstd that it returned; dx is the gradient of x and of the
    residual alike."""
    r, pr, ldr = _rows(r, "r", _ACTIVATIONS)
    shape, ty = r.shape, r.dtype
    if len(shape) < 1:
        raise ValueError("r must be (..., D)")
    dy, pdy, lddy = _rows(dy, "dy", (ty,))
    if dy.shape != shape:
        raise ValueError("dy must have r's shape")
    pdr, lddr = 0, shape[-1]
    if dr is not None:
        dr, pdr, lddr = _rows(dr, "dr", (ty,))
        if dr.shape != shape:
            raise ValueError("dr must have r's shape")
    D = shape[-1]
    M = r.numel() // D if D else 0
    w, pw = _param(w, "w", (D,))
    if w is None or rstd is None:
        raise ValueError("w must be (D,), and rstd what mg_rms_norm_fwd returned")
    rstd, ps = _param(rstd, "rstd", shape[:-1])
    _together(r, dy, dr, w, rstd, ws, *(out or ()))
    dx, pdx = _new(out, 0, shape, r, ty)
    dw, pdw = _new(out, 1, (D,), r, _F32)
    sh = _stream(r)
    _run_ws("mg_rms_norm_bwd", lambda: load().mg_rms_norm_workspace_size(M, D), r.device, ws,
            (pdy, lddy, ps, pr, ldr, pdr, lddr, _DT[ty], pw, pdx, pdw, M, D), sh)
    return dx, dw


gated_scan_fwd = mg_gated_scan_fwd
gated_scan_bwd = mg_gated_scan_bwd
gated_scan_step = mg_gated_scan_step
rms_norm_fwd = mg_rms_norm_fwd
rms_norm_quant = mg_rms_norm_quant
rms_norm_bwd = mg_rms_norm_bwd
