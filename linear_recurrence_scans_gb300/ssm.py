"""The selective state space mixer's operators (``include/mg_ssm.h``): the
short causal depthwise convolution, the selective scan and the gated group
norm, channels last, for prompts, for training and for single tokens.

* ``causal_conv_fwd(x, w, bias=None, x0=None) -> (y, x_last)``,
  ``causal_conv_bwd(dy, x, w, ...) -> (dx, dw, dbias, dx0)``,
  ``causal_conv_step(x, w, state, bias=None, slots=None) -> y``
* ``selective_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, h0=None) -> (y, h_last, saved)``,
  ``selective_scan_bwd(dy, saved, x, dt, A, B, C, ...) -> (dx, ddt, dA, dB, dC, dD, ddt_bias, dh0)``,
  ``selective_scan_step(x, dt, A, B, C, state, D=None, dt_bias=None, slots=None) -> y``
* ``group_norm_fwd(x, w, bias=None, z=None, groups=1) -> (y, stats)``,
  ``group_norm_bwd(dy, stats, x, w, ...) -> (dx, dw, dbias, dz)``

Activations are float32 or bf16, all of a call the same; parameters, states
and their gradients are float32 (the convolution's state has the activations'
type).  Activations may be slices of wider rows (last dimension contiguous);
anything else is copied first.  ``cu_seqlens`` (int64, on the device) packs
sequences of any lengths into a batch of one.  ``out=`` takes preallocated
outputs in the order of the results (``None`` where the call is to allocate),
``ws=`` a workspace and ``stream=`` a stream, on which copies and outputs are
then made too; a token call writes its state in place.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _DT, _check, _cu, _out, _prep, _stream_handle, _workspace, load

__all__ = [
    "mg_causal_conv_fwd", "mg_causal_conv_bwd", "mg_causal_conv_step",
    "mg_selective_scan_fwd", "mg_selective_scan_bwd", "mg_selective_scan_step",
    "mg_group_norm_fwd", "mg_group_norm_bwd",
    "causal_conv_fwd", "causal_conv_bwd", "causal_conv_step",
    "selective_scan_fwd", "selective_scan_bwd", "selective_scan_step",
    "group_norm_fwd", "group_norm_bwd",
]

SYMBOLS = (
    "mg_causal_conv_workspace_size", "mg_causal_conv_fwd", "mg_causal_conv_bwd",
    "mg_causal_conv_step", "mg_selective_scan_fwd_workspace_size",
    "mg_selective_scan_bwd_workspace_size", "mg_selective_scan_saved_size",
    "mg_selective_scan_saved_rows", "mg_selective_scan_fwd", "mg_selective_scan_bwd",
    "mg_selective_scan_step", "mg_group_norm_workspace_size", "mg_group_norm_fwd",
    "mg_group_norm_bwd",
)

MAX_STATES, MAX_TAPS = 64, 8
_ACTIVATIONS = (torch.float32, torch.bfloat16)
_CONTROL_BYTES = 256


def declare(lib):
    """Argument types of the entry points of mg_ssm.h."""
    vp, i64, i32, sz, f64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                             ctypes.c_double)
    sizes = {"mg_causal_conv_workspace_size": [i64, i64, i64, i32],
             "mg_selective_scan_fwd_workspace_size": [i64] * 6,
             "mg_selective_scan_bwd_workspace_size": [i64] * 6,
             "mg_selective_scan_saved_size": [i64] * 4,
             "mg_group_norm_workspace_size": [i64] * 3}
    for name, args in sizes.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, sz
    lib.mg_selective_scan_saved_rows.argtypes, lib.mg_selective_scan_saved_rows.restype = [], i32
    calls = {
        "mg_causal_conv_fwd": [vp, i64, i32, vp, vp, vp, vp, i64, i32, vp, vp, i64, i64, i64, i32,
                               vp, sz, vp],
        "mg_causal_conv_bwd": [vp, i64, vp, i64, i32, vp, vp, vp, vp, vp, i64, i32, vp, vp, vp, vp,
                               i64, i64, i64, i32, vp, sz, vp],
        "mg_causal_conv_step": [vp, i64, i32, vp, vp, vp, i64, vp, i32, vp, i64, i64, i32, vp],
        "mg_selective_scan_fwd": [vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, vp, vp, i32, vp, vp,
                                  i64, vp, vp, vp, i64, i64, i64, i64, i64, vp, sz, vp],
        "mg_selective_scan_bwd": [vp, i64, vp, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, vp, vp,
                                  i32, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                  i64, i64, i64, i64, i64, vp, sz, vp],
        "mg_selective_scan_step": [vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, vp, vp, i32, vp,
                                   i64, vp, vp, i64, i64, i64, i64, vp],
        "mg_group_norm_fwd": [vp, i64, vp, i64, i32, vp, vp, f64, i32, i32, i32, vp, vp,
                              i64, i64, i64, vp],
        "mg_group_norm_bwd": [vp, i64, vp, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32,
                              vp, vp, vp, vp, i64, i64, i64, vp, sz, vp],
    }
    for name, args in calls.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, i32


# ---------------------------------------------------------------- arguments

def _on_stream(f):
    """With stream=, everything the op does (copies of arguments and the
    allocation of outputs too) happens on that stream."""
    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return call


def _rows(x, name, dtypes, inner=1):
    """(tensor, row stride) of an activation whose rows are its last ``inner``
    dimensions: x itself where the kernels can read its rows in place, else a
    dense copy."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {x.dtype} not in {dtypes}")
    shape, stride = x.shape, x.stride()
    width = shape[-1] if inner == 1 else shape[-1] * shape[-2]
    ok, step = x.data_ptr() % 16 == 0, 1
    for i in range(1, inner + 1):
        ok = ok and (shape[-i] == 1 or stride[-i] == step)
        step *= shape[-i]
    ld, rows = 0, 1
    for i in range(len(shape) - inner - 1, -1, -1):
        n = shape[i]
        if n != 1:
            if ld == 0:
                ld = stride[i]   # rows is still 1 here
            elif stride[i] != ld * rows:
                ok = False
            rows *= n
    if ld == 0 and rows == 1:
        ld = width
    if ok and ld >= width:
        return x, ld
    return x.clone(memory_format=torch.contiguous_format), width


def _param(x, name, shape):
    """A float32 parameter or state of that shape, dense (None stays None)."""
    if x is None:
        return None
    x = _prep(x, name)
    if tuple(x.shape) != shape:
        raise ValueError(f"{name} must be {shape}")
    return x


def _ptr(x):
    return x.data_ptr() if x is not None and x.numel() else None


def _silu(act):
    if act not in ("silu", None):
        raise ValueError('act must be "silu" or None')
    return int(act == "silu")


def _sequences(cu_seqlens, x, B):
    """(cu, number of sequences) of a batch of B rows of sequences."""
    if cu_seqlens is None:
        return None, B
    if B != 1:
        raise ValueError("with cu_seqlens the batch must be one packed sequence")
    cu = _cu(cu_seqlens, x)
    if cu.numel() < 2:
        raise ValueError("cu_seqlens must name at least one sequence")
    return cu, cu.numel() - 1


def _slots(slots, state, B):
    if slots is None:
        if state.shape[0] < B:
            raise ValueError("state must have an entry for every row of the batch")
        return None
    if not isinstance(slots, torch.Tensor) or not slots.is_cuda or slots.dtype != torch.int64 \
            or slots.dim() != 1 or slots.numel() != B:
        raise ValueError("slots must be a CUDA int64 tensor with one entry for each row")
    slots = slots.contiguous()
    return slots.clone() if slots.data_ptr() % 16 else slots


def _state(state, name, dtype, inner):
    """A pool of states that a call updates in place: never copied."""
    if not isinstance(state, torch.Tensor) or not state.is_cuda or state.dtype != dtype \
            or state.dim() != 1 + len(inner) or tuple(state.shape[1:]) != inner \
            or not state.is_contiguous() or state.data_ptr() % 16:
        raise ValueError(f"{name} must be a dense, 16-byte aligned {dtype} CUDA tensor "
                         f"(states, {', '.join(map(str, inner))})")
    return state


# -------------------------------------------------------------- convolution

def _conv_args(x, w, bias, x0, cu_seqlens):
    x, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != 3:
        raise ValueError("x must be (B, T, D)")
    B, T, D = x.shape
    w = _prep(w, "w")
    if w.dim() != 2 or w.shape[0] != D or not 1 <= w.shape[1] <= MAX_TAPS:
        raise ValueError(f"w must be (D, W) with W at most {MAX_TAPS}")
    W = w.shape[1]
    cu, nseq = _sequences(cu_seqlens, x, B)
    bias = _param(bias, "bias", (D,))
    edge = (nseq, W - 1, D)
    if x0 is not None:
        x0 = _prep(x0, "x0", (x.dtype,))
        if tuple(x0.shape) != edge:
            raise ValueError(f"x0 must be {edge}")
    return x, ldx, w, bias, x0, cu, nseq, edge


@_on_stream
def mg_causal_conv_fwd(x, w, bias=None, x0=None, *, act="silu", cu_seqlens=None, out=None, ws=None):
    """(y (B,T,D), x_last (sequences, W-1, D)): y = act(bias + sum_k w[:, k]
    x_{t-W+1+k}), from the W-1 rows x0 before each sequence (zero without
    them); x_last holds each sequence's last W-1 inputs, the x0 of what
    follows.  w (D, W), 1 <= W <= 8; act "silu" or None."""
    x, ldx, w, bias, x0, cu, nseq, edge = _conv_args(x, w, bias, x0, cu_seqlens)
    B, T, D = x.shape
    y = _out(out, 0, x.shape, x, x.dtype)
    x_last = _out(out, 1, edge, x, x.dtype)
    sh = _stream_handle(None, x.device)
    wk = _workspace(_CONTROL_BYTES, x.device, sh, ws)
    _check(load().mg_causal_conv_fwd(_ptr(x), ldx, _DT[x.dtype], _ptr(w), _ptr(bias), _ptr(x0),
                                     _ptr(cu), nseq, _silu(act), _ptr(y), _ptr(x_last), B, T, D,
                                     w.shape[1], wk.data_ptr(), wk.numel(), sh),
           "mg_causal_conv_fwd")
    return y, x_last


@_on_stream
def mg_causal_conv_bwd(dy, x, w, bias=None, x0=None, dx_last=None, *, act="silu", cu_seqlens=None,
                       out=None, ws=None):
    """(dx, dw, dbias, dx0): gradients of sum(dy*y) + sum(dx_last*x_last) for
    mg_causal_conv_fwd on the same inputs; dbias and dx0 are None without bias
    and x0."""
    x, ldx, w, bias, x0, cu, nseq, edge = _conv_args(x, w, bias, x0, cu_seqlens)
    dy, lddy = _rows(dy, "dy", (x.dtype,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    if dx_last is not None:
        dx_last = _prep(dx_last, "dx_last", (x.dtype,))
        if tuple(dx_last.shape) != edge:
            raise ValueError(f"dx_last must be {edge}")
    B, T, D = x.shape
    dx = _out(out, 0, x.shape, x, x.dtype)
    dw = _out(out, 1, w.shape, x)
    dbias = _out(out, 2, (D,), x) if bias is not None else None
    dx0 = _out(out, 3, edge, x, x.dtype) if x0 is not None else None
    sh = _stream_handle(None, x.device)
    lib = load()
    wk = _workspace(lib.mg_causal_conv_workspace_size(B, T, D, w.shape[1]), x.device, sh, ws)
    _check(lib.mg_causal_conv_bwd(_ptr(dy), lddy, _ptr(x), ldx, _DT[x.dtype], _ptr(w), _ptr(bias),
                                  _ptr(x0), _ptr(dx_last), _ptr(cu), nseq, _silu(act), _ptr(dx),
                                  _ptr(dw), _ptr(dbias), _ptr(dx0), B, T, D, w.shape[1],
                                  wk.data_ptr(), wk.numel(), sh),
           "mg_causal_conv_bwd")
    return dx, dw, dbias, dx0


@_on_stream
def mg_causal_conv_step(x, w, state, bias=None, *, slots=None, act="silu", out=None):
    """y (B, D): one token x (B, D) a row through the convolution.  Row i's
    last W-1 inputs are state[slots[i]] (state[i] without slots), of x's type,
    (states, W-1, D), moved on in place; a row whose slot is not in the pool
    is idle: y 0, no state written."""
    x, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != 2:
        raise ValueError("x must be (B, D)")
    B, D = x.shape
    w = _prep(w, "w")
    if w.dim() != 2 or w.shape[0] != D or not 1 <= w.shape[1] <= MAX_TAPS:
        raise ValueError(f"w must be (D, W) with W at most {MAX_TAPS}")
    W = w.shape[1]
    state = _state(state, "state", x.dtype, (W - 1, D))
    slots = _slots(slots, state, B)
    bias = _param(bias, "bias", (D,))
    y = _out(None if out is None else (out,), 0, x.shape, x, x.dtype)
    _check(load().mg_causal_conv_step(_ptr(x), ldx, _DT[x.dtype], _ptr(w), _ptr(bias), _ptr(state),
                                      state.shape[0], _ptr(slots), _silu(act), _ptr(y), B, D, W,
                                      _stream_handle(None, x.device)),
           "mg_causal_conv_step")
    return y


# ------------------------------------------------------------ selective scan

def _scan_args(x, dt, A, B, C, D, dt_bias, lead):
    """The arguments that the scan's three calls share; x has `lead` leading
    dimensions.  B and C may leave out the group dimension."""
    x, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != lead + 1:
        raise ValueError("x must be (B, T, D)" if lead == 2 else "x must be (B, D)")
    dt, ldt = _rows(dt, "dt", (x.dtype,))
    if dt.shape != x.shape:
        raise ValueError("dt must have x's shape")
    Dx = x.shape[-1]
    A = _prep(A, "A")
    if A.dim() != 2 or A.shape[0] != Dx or not 1 <= A.shape[1] <= MAX_STATES:
        raise ValueError(f"A must be (D, N) with N at most {MAX_STATES}")
    N = A.shape[1]
    bc = []
    for m, name in ((B, "B"), (C, "C")):
        if not isinstance(m, torch.Tensor) or m.dim() not in (lead + 1, lead + 2) \
                or m.shape[:lead] != x.shape[:lead] or m.shape[-1] != N:
            raise ValueError(f"{name} must be x's leading dimensions and (G, N), or (N)")
        bc.append(_rows(m, name, (x.dtype,), m.dim() - lead))
    (B, ldb), (C, ldc) = bc
    if B.shape != C.shape:
        raise ValueError("B and C must have the same shape")
    G = B.shape[-2] if B.dim() == lead + 2 else 1
    if G < 1 or Dx % G:
        raise ValueError("D must be a multiple of the number of groups of B and C")
    return (x, ldx, dt, ldt, A, B, ldb, C, ldc, _param(D, "D", (Dx,)),
            _param(dt_bias, "dt_bias", (Dx,)), N, G)


@_on_stream
def mg_selective_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, h0=None, *, softplus=True,
                          cu_seqlens=None, save=False, out=None, ws=None):
    """(y (B,T,D), h_last (sequences, D, N), saved): the selective scan
      h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = C_t h_t + D x_t,
    delta = softplus(dt + dt_bias) (without softplus: dt + dt_bias), from h0.
    x, dt (B,T,D); A (D,N), N <= 64; B, C (B,T,G,N), or (B,T,N) for one group;
    channel d reads group d // (D/G).  saved, with save=True, is what
    mg_selective_scan_bwd needs of this call; else None."""
    x, ldx, dt, ldt, A, Bm, ldb, Cm, ldc, D, dt_bias, N, G = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    Bx, T, Dx = x.shape
    cu, nseq = _sequences(cu_seqlens, x, Bx)
    h0 = _param(h0, "h0", (nseq, Dx, N))
    y = _out(out, 0, x.shape, x, x.dtype)
    h_last = _out(out, 1, (nseq, Dx, N), x)
    lib = load()
    saved = _out(out[2:] if out is not None and len(out) > 2 else None, 0,
                 (lib.mg_selective_scan_saved_size(Bx, T, Dx, N) // 4,), x) if save else None
    sh = _stream_handle(None, x.device)
    wk = _workspace(lib.mg_selective_scan_fwd_workspace_size(Bx, T, Dx, N, G, nseq), x.device, sh, ws)
    _check(lib.mg_selective_scan_fwd(_ptr(x), ldx, _ptr(dt), ldt, _ptr(A), _ptr(Bm), ldb, _ptr(Cm),
                                     ldc, _DT[x.dtype], _ptr(D), _ptr(dt_bias), int(bool(softplus)),
                                     _ptr(h0), _ptr(cu), nseq, _ptr(y), _ptr(h_last), _ptr(saved),
                                     Bx, T, Dx, N, G, wk.data_ptr(), wk.numel(), sh),
           "mg_selective_scan_fwd")
    return y, h_last, saved


@_on_stream
def mg_selective_scan_bwd(dy, saved, x, dt, A, B, C, D=None, dt_bias=None, h0=None, dh_last=None, *,
                          softplus=True, cu_seqlens=None, out=None, ws=None):
    """(dx, ddt, dA, dB, dC, dD, ddt_bias, dh0): gradients of sum(dy*y) +
    sum(dh_last*h_last) for mg_selective_scan_fwd on the same inputs, with the
    `saved` that it returned.  dD, ddt_bias and dh0 are None where their input
    is."""
    x, ldx, dt, ldt, A, Bm, ldb, Cm, ldc, D, dt_bias, N, G = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    dy, lddy = _rows(dy, "dy", (x.dtype,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    Bx, T, Dx = x.shape
    cu, nseq = _sequences(cu_seqlens, x, Bx)
    h0 = _param(h0, "h0", (nseq, Dx, N))
    dh_last = _param(dh_last, "dh_last", (nseq, Dx, N))
    lib = load()
    saved = _param(saved, "saved", (lib.mg_selective_scan_saved_size(Bx, T, Dx, N) // 4,))
    if saved is None:
        raise ValueError("saved must be what mg_selective_scan_fwd returned with save=True")
    dx, ddt = _out(out, 0, x.shape, x, x.dtype), _out(out, 1, x.shape, x, x.dtype)
    dA = _out(out, 2, A.shape, x)
    dB, dC = _out(out, 3, Bm.shape, x, x.dtype), _out(out, 4, Cm.shape, x, x.dtype)
    dD = _out(out, 5, (Dx,), x) if D is not None else None
    ddt_bias = _out(out, 6, (Dx,), x) if dt_bias is not None else None
    dh0 = _out(out, 7, (nseq, Dx, N), x) if h0 is not None else None
    sh = _stream_handle(None, x.device)
    wk = _workspace(lib.mg_selective_scan_bwd_workspace_size(Bx, T, Dx, N, G, nseq), x.device, sh, ws)
    _check(lib.mg_selective_scan_bwd(_ptr(dy), lddy, _ptr(saved), _ptr(x), ldx, _ptr(dt), ldt,
                                     _ptr(A), _ptr(Bm), ldb, _ptr(Cm), ldc, _DT[x.dtype], _ptr(D),
                                     _ptr(dt_bias), int(bool(softplus)), _ptr(h0), _ptr(dh_last),
                                     _ptr(cu), nseq, _ptr(dx), _ptr(ddt), _ptr(dA), _ptr(dB),
                                     _ptr(dC), _ptr(dD), _ptr(ddt_bias), _ptr(dh0), Bx, T, Dx, N, G,
                                     wk.data_ptr(), wk.numel(), sh),
           "mg_selective_scan_bwd")
    return dx, ddt, dA, dB, dC, dD, ddt_bias, dh0


@_on_stream
def mg_selective_scan_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, slots=None,
                           softplus=True, out=None):
    """y (B, D): one token a row through mg_selective_scan_fwd's recurrence.
    x, dt (B, D); B, C (B, G, N) or (B, N).  Row i's state is state[slots[i]]
    (state[i] without slots) of (states, D, N) float32, updated in place; a
    row whose slot is not in the pool is idle: y 0, no state written."""
    x, ldx, dt, ldt, A, Bm, ldb, Cm, ldc, D, dt_bias, N, G = _scan_args(x, dt, A, B, C, D, dt_bias, 1)
    Bx, Dx = x.shape
    state = _state(state, "state", torch.float32, (Dx, N))
    slots = _slots(slots, state, Bx)
    y = _out(None if out is None else (out,), 0, x.shape, x, x.dtype)
    _check(load().mg_selective_scan_step(_ptr(x), ldx, _ptr(dt), ldt, _ptr(A), _ptr(Bm), ldb,
                                         _ptr(Cm), ldc, _DT[x.dtype], _ptr(D), _ptr(dt_bias),
                                         int(bool(softplus)), _ptr(state), state.shape[0],
                                         _ptr(slots), _ptr(y), Bx, Dx, N, G,
                                         _stream_handle(None, x.device)),
           "mg_selective_scan_step")
    return y


# -------------------------------------------------------------- group norm

MG_GATE_NONE, MG_GATE_AFTER, MG_GATE_FIRST = range(3)


def _norm_args(x, w, bias, z, groups, gate_first):
    x, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() < 1:
        raise ValueError("x must be (..., D)")
    D = x.shape[-1]
    if groups < 1 or D % groups:
        raise ValueError("the channels must be a multiple of groups")
    ldz, gate = D, MG_GATE_NONE
    if z is not None:
        z, ldz = _rows(z, "z", (x.dtype,))
        if z.shape != x.shape:
            raise ValueError("z must have x's shape")
        gate = MG_GATE_FIRST if gate_first else MG_GATE_AFTER
    elif gate_first:
        raise ValueError("gate_first needs z")
    w = _param(w, "w", (D,))
    if w is None:
        raise ValueError("w must be (D,)")
    M = x.numel() // D if D else 0
    return x, ldx, z, ldz, w, _param(bias, "bias", (D,)), gate, M, D


@_on_stream
def mg_group_norm_fwd(x, w, bias=None, z=None, *, groups=1, eps=1e-5, rms=False, gate_first=False,
                      act="silu", out=None):
    """(y, stats): each row of x (..., D) in `groups` groups of neighbouring
    channels, each normalised by itself (rms: without taking the mean out),
    o = n w + bias; y = o act(z), or with gate_first the norm is of x act(z)
    and y = o, or without z y = act(o).  act "silu" or None; groups of at most
    16384 channels.  stats (rows, groups, 2) is for mg_group_norm_bwd."""
    x, ldx, z, ldz, w, bias, gate, M, D = _norm_args(x, w, bias, z, groups, gate_first)
    y = _out(out, 0, x.shape, x, x.dtype)
    stats = _out(out, 1, (M, groups, 2), x)
    _check(load().mg_group_norm_fwd(_ptr(x), ldx, _ptr(z), ldz, _DT[x.dtype], _ptr(w), _ptr(bias),
                                    float(eps), int(bool(rms)), gate, _silu(act), _ptr(y),
                                    _ptr(stats), M, D, groups, _stream_handle(None, x.device)),
           "mg_group_norm_fwd")
    return y, stats


@_on_stream
def mg_group_norm_bwd(dy, stats, x, w, bias=None, z=None, *, groups=1, eps=1e-5, rms=False,
                      gate_first=False, act="silu", out=None, ws=None):
    """(dx, dw, dbias, dz): gradients of sum(dy*y) for mg_group_norm_fwd on the
    same inputs, with the stats that it returned (eps is in them already);
    dbias and dz are None without bias and z."""
    x, ldx, z, ldz, w, bias, gate, M, D = _norm_args(x, w, bias, z, groups, gate_first)
    dy, lddy = _rows(dy, "dy", (x.dtype,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    stats = _param(stats, "stats", (M, groups, 2))
    if stats is None:
        raise ValueError("stats must be what mg_group_norm_fwd returned")
    dx = _out(out, 0, x.shape, x, x.dtype)
    dw = _out(out, 1, (D,), x)
    dbias = _out(out, 2, (D,), x) if bias is not None else None
    dz = _out(out, 3, x.shape, x, x.dtype) if z is not None else None
    sh = _stream_handle(None, x.device)
    lib = load()
    wk = _workspace(lib.mg_group_norm_workspace_size(M, D, groups), x.device, sh, ws)
    _check(lib.mg_group_norm_bwd(_ptr(dy), lddy, _ptr(stats), _ptr(x), ldx, _ptr(z), ldz,
                                 _DT[x.dtype], _ptr(w), _ptr(bias), int(bool(rms)), gate, _silu(act),
                                 _ptr(dx), _ptr(dz), _ptr(dw), _ptr(dbias), M, D, groups,
                                 wk.data_ptr(), wk.numel(), sh),
           "mg_group_norm_bwd")
    return dx, dw, dbias, dz


causal_conv_fwd = mg_causal_conv_fwd
causal_conv_bwd = mg_causal_conv_bwd
causal_conv_step = mg_causal_conv_step
selective_scan_fwd = mg_selective_scan_fwd
selective_scan_bwd = mg_selective_scan_bwd
selective_scan_step = mg_selective_scan_step
group_norm_fwd = mg_group_norm_fwd
group_norm_bwd = mg_group_norm_bwd
