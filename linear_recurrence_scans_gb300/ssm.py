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
import struct

import torch
from torch import Tensor

from . import (_DT, MG_ERR_INVALID_ARG, MG_OK, _check, _cu, _out, _prep, _stream_handle, _workspace,
               load)

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
    "mg_group_norm_bwd", "mg_ssm_call",
)

MAX_STATES, MAX_TAPS = 64, 8
_ACTIVATIONS = (torch.float32, torch.bfloat16)
_F32 = torch.float32
_CONTROL_BYTES = 256

# The calls' argument blocks (mg_ssm_call): one packed argument costs a third
# of what ctypes takes for twenty.
_OPS = {name: (op, struct.Struct(words).pack, len(words)) for op, (name, words) in enumerate({
    "mg_causal_conv_fwd": "q" * 18, "mg_causal_conv_bwd": "q" * 23, "mg_causal_conv_step": "q" * 14,
    "mg_selective_scan_fwd": "q" * 27, "mg_selective_scan_bwd": "q" * 36,
    "mg_selective_scan_step": "q" * 22,
    "mg_group_norm_fwd": "q" * 7 + "d" + "q" * 9, "mg_group_norm_bwd": "q" * 23,
}.items())}
_call = None


def declare(lib):
    """Argument types of the entry points of mg_ssm.h that are called."""
    global _call
    i64, i32, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sizes = {"mg_causal_conv_workspace_size": [i64, i64, i64, i32],
             "mg_selective_scan_fwd_workspace_size": [i64] * 6,
             "mg_selective_scan_bwd_workspace_size": [i64] * 6,
             "mg_selective_scan_saved_size": [i64] * 4,
             "mg_group_norm_workspace_size": [i64] * 3}
    for name, args in sizes.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, sz
    lib.mg_selective_scan_saved_rows.argtypes, lib.mg_selective_scan_saved_rows.restype = [], i32
    vp, f64 = ctypes.c_void_p, ctypes.c_double
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
    lib.mg_ssm_call.argtypes, lib.mg_ssm_call.restype = [i32, ctypes.c_char_p, i32], i32
    _call = lib.mg_ssm_call


def _run(name, *words):
    """The C call `name`; `words` are its arguments."""
    op, pack, n = _OPS[name]
    st = (_call or load().mg_ssm_call)(op, pack(*words), n)
    if st != MG_OK:
        _check(st, name)


def _run_ws(name, need, device, ws, words, sh):
    """The C call `name` with a workspace: arguments `words`, then workspace,
    its size and the stream.  The stream's cached workspace is tried as it is;
    need() is asked only when the call says that it does not do."""
    op, pack, n = _OPS[name]
    buf = _workspace(_CONTROL_BYTES, device, sh, ws)
    st = (_call or load().mg_ssm_call)(op, pack(*words, buf.data_ptr(), buf.numel(), sh), n)
    if st == MG_ERR_INVALID_ARG and ws is None:
        size = need()
        if size > buf.numel():
            buf = _workspace(size, device, sh, None)
            st = _call(op, pack(*words, buf.data_ptr(), buf.numel(), sh), n)
    if st != MG_OK:
        _check(st, name)


# ---------------------------------------------------------------- arguments

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(x) -> int:
    return _raw_stream(x.get_device()) if _raw_stream is not None else _stream_handle(None, x.device)


def _rows(x, name, dtypes, inner=1):
    """(x, pointer, row stride) of an activation whose rows are its last
    ``inner`` dimensions: x itself where the kernels can read its rows in
    place, else a dense copy."""
    if not isinstance(x, Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {x.dtype} not in {dtypes}")
    shape = x.shape
    width = shape[-1] if inner == 1 else shape[-1] * shape[-2]
    ptr = x.data_ptr()
    if not ptr & 15:
        if x.is_contiguous():
            return x, ptr, width
        stride, ok, step = x.stride(), True, 1
        for i in range(1, inner + 1):
            ok = ok and (shape[-i] == 1 or stride[-i] == step)
            step *= shape[-i]
        ld, rows = 0, 1
        for i in range(len(shape) - inner - 1, -1, -1):
            n = shape[i]
            if n != 1:
                if rows == 1:
                    ld = stride[i]
                elif stride[i] != ld * rows:
                    ok = False
                rows *= n
        if rows == 1:
            ld = width
        if ok and ld >= width:
            return x, ptr, ld
    x = x.clone(memory_format=torch.contiguous_format)
    return x, x.data_ptr(), width


def _param(x, name, shape, dtype=_F32):
    """(x, pointer) of a dense parameter or state of that shape (None and NULL
    stay what they are)."""
    if x is None:
        return None, 0
    if not isinstance(x, Tensor) or x.dtype != dtype or not x.is_cuda or not x.is_contiguous() \
            or x.data_ptr() & 15:
        x = _prep(x, name, (dtype,))
    if x.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}")
    return x, x.data_ptr()


def _new(out, i, shape, like, dtype):
    """(output i, its pointer): the caller's, or a new one."""
    if out is None or i >= len(out) or out[i] is None:
        o = torch.empty(shape, dtype=dtype, device=like.device)
    else:
        o = _out(out, i, shape, like, dtype)
    return o, o.data_ptr()


def _silu(act):
    if act == "silu":
        return 1
    if act is not None:
        raise ValueError('act must be "silu" or None')
    return 0


def _sequences(cu_seqlens, x, B):
    """(cu, its pointer, number of sequences) of a batch of B rows of sequences."""
    if cu_seqlens is None:
        return None, 0, B
    if B != 1:
        raise ValueError("with cu_seqlens the batch must be one packed sequence")
    cu = _cu(cu_seqlens, x)
    if cu.numel() < 2:
        raise ValueError("cu_seqlens must name at least one sequence")
    if cu.data_ptr() & 7:
        cu = cu.clone()
    return cu, cu.data_ptr(), cu.numel() - 1


def _slots(slots, state, B):
    if slots is None:
        if state.shape[0] < B:
            raise ValueError("state must have an entry for every row of the batch")
        return None, 0
    if not isinstance(slots, Tensor) or slots.dtype != torch.int64 or not slots.is_cuda or slots.shape != (B,):
        raise ValueError("slots must be a CUDA int64 tensor with one entry for each row")
    if not slots.is_contiguous():
        slots = slots.clone(memory_format=torch.contiguous_format)
    return slots, slots.data_ptr()


def _state(state, name, dtype, inner):
    """A pool of states that a call updates in place: never copied."""
    if not isinstance(state, Tensor) or state.dtype != dtype or not state.is_cuda \
            or state.shape[1:] != inner or state.dim() != 1 + len(inner) \
            or not state.is_contiguous() or state.data_ptr() & 15:
        raise ValueError(f"{name} must be a dense, 16-byte aligned {dtype} CUDA tensor "
                         f"(states, {', '.join(map(str, inner))})")
    return state.data_ptr()


# -------------------------------------------------------------- convolution

def _taps(w, D):
    if not isinstance(w, Tensor) or w.dim() != 2 or w.shape[0] != D or not 1 <= w.shape[1] <= MAX_TAPS:
        raise ValueError(f"w must be (D, W) with W at most {MAX_TAPS}")
    return _param(w, "w", w.shape)


def mg_causal_conv_fwd(x, w, bias=None, x0=None, *, act="silu", cu_seqlens=None, out=None, ws=None,
                       stream=None):
    """(y (B,T,D), x_last (sequences, W-1, D)): y = act(bias + sum_k w[:, k]
    x_{t-W+1+k}), from the W-1 rows x0 before each sequence (zero without
    them); x_last holds each sequence's last W-1 inputs, the x0 of what
    follows.  w (D, W), 1 <= W <= 8; act "silu" or None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_causal_conv_fwd(x, w, bias, x0, act=act, cu_seqlens=cu_seqlens, out=out, ws=ws)
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != 3:
        raise ValueError("x must be (B, T, D)")
    (B, T, D), ty = x.shape, x.dtype
    w, pw = _taps(w, D)
    W = w.shape[1]
    cu, pcu, nseq = _sequences(cu_seqlens, x, B)
    edge = (nseq, W - 1, D)
    bias, pb = _param(bias, "bias", (D,))
    x0, px0 = _param(x0, "x0", edge, ty)
    y, py = _new(out, 0, (B, T, D), x, ty)
    x_last, pl = _new(out, 1, edge, x, ty)
    sh = _stream(x)
    _run_ws("mg_causal_conv_fwd", lambda: _CONTROL_BYTES, x.device, ws,
            (px, ldx, _DT[ty], pw, pb, px0, pcu, nseq, _silu(act), py, pl, B, T, D, W), sh)
    return y, x_last


def mg_causal_conv_bwd(dy, x, w, bias=None, x0=None, dx_last=None, *, act="silu", cu_seqlens=None,
                       out=None, ws=None, stream=None):
    """(dx, dw, dbias, dx0): gradients of sum(dy*y) + sum(dx_last*x_last) for
    mg_causal_conv_fwd on the same inputs; dbias and dx0 are None without bias
    and x0."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_causal_conv_bwd(dy, x, w, bias, x0, dx_last, act=act, cu_seqlens=cu_seqlens,
                                      out=out, ws=ws)
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != 3:
        raise ValueError("x must be (B, T, D)")
    (B, T, D), ty = x.shape, x.dtype
    dy, pdy, lddy = _rows(dy, "dy", (ty,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    w, pw = _taps(w, D)
    W = w.shape[1]
    cu, pcu, nseq = _sequences(cu_seqlens, x, B)
    edge = (nseq, W - 1, D)
    bias, pb = _param(bias, "bias", (D,))
    x0, px0 = _param(x0, "x0", edge, ty)
    dx_last, pdl = _param(dx_last, "dx_last", edge, ty)
    dx, pdx = _new(out, 0, (B, T, D), x, ty)
    dw, pdw = _new(out, 1, (D, W), x, _F32)
    dbias, pdb = _new(out, 2, (D,), x, _F32) if bias is not None else (None, 0)
    dx0, pdx0 = _new(out, 3, edge, x, ty) if x0 is not None else (None, 0)
    sh = _stream(x)
    _run_ws("mg_causal_conv_bwd", lambda: load().mg_causal_conv_workspace_size(B, T, D, W), x.device, ws,
            (pdy, lddy, px, ldx, _DT[ty], pw, pb, px0, pdl, pcu, nseq, _silu(act), pdx, pdw, pdb, pdx0,
             B, T, D, W), sh)
    return dx, dw, dbias, dx0


def mg_causal_conv_step(x, w, state, bias=None, *, slots=None, act="silu", out=None, stream=None):
    """y (B, D): one token x (B, D) a row through the convolution.  Row i's
    last W-1 inputs are state[slots[i]] (state[i] without slots), of x's type,
    (states, W-1, D), moved on in place; a row whose slot is not in the pool
    is idle: y 0, no state written."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_causal_conv_step(x, w, state, bias, slots=slots, act=act, out=out)
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    if x.dim() != 2:
        raise ValueError("x must be (B, D)")
    (B, D), ty = x.shape, x.dtype
    w, pw = _taps(w, D)
    W = w.shape[1]
    ps = _state(state, "state", ty, (W - 1, D))
    slots, psl = _slots(slots, state, B)
    bias, pb = _param(bias, "bias", (D,))
    y, py = _new(None if out is None else (out,), 0, (B, D), x, ty)
    _run("mg_causal_conv_step", px, ldx, _DT[ty], pw, pb, ps, state.shape[0], psl, _silu(act), py, B, D, W,
         _stream(x))
    return y


# ------------------------------------------------------------ selective scan

def _scan_args(x, dt, A, B, C, D, dt_bias, lead):
    """The arguments that the scan's three calls share; x has `lead` leading
    dimensions.  B and C may leave out the group dimension.  The tensors (kept
    alive until the call is made), the words of the C calls from x to the
    softplus flag, N, G and the shape of B and C."""
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    shape, ty = x.shape, x.dtype
    if len(shape) != lead + 1:
        raise ValueError("x must be (B, T, D)" if lead == 2 else "x must be (B, D)")
    like = (ty,)
    dt, pdt, ldt = _rows(dt, "dt", like)
    if dt.shape != shape:
        raise ValueError("dt must have x's shape")
    Dx = shape[-1]
    if not isinstance(A, Tensor) or A.dim() != 2 or A.shape[0] != Dx or not 1 <= A.shape[1] <= MAX_STATES:
        raise ValueError(f"A must be (D, N) with N at most {MAX_STATES}")
    A, pA = _param(A, "A", A.shape)
    N = A.shape[1]
    bshape = B.shape if isinstance(B, Tensor) else ()
    dims = len(bshape) - lead
    if dims not in (1, 2) or bshape[-1] != N or bshape[:lead] != shape[:lead] \
            or not isinstance(C, Tensor) or C.shape != bshape:
        raise ValueError("B and C must both be x's leading dimensions and (G, N), or (N)")
    B, pB, ldb = _rows(B, "B", like, dims)
    C, pC, ldc = _rows(C, "C", like, dims)
    G = bshape[-2] if dims == 2 else 1
    if G < 1 or Dx % G:
        raise ValueError("D must be a multiple of the number of groups of B and C")
    D, pD = _param(D, "D", (Dx,))
    dt_bias, pbias = _param(dt_bias, "dt_bias", (Dx,))
    return ((x, dt, A, B, C, D, dt_bias), (px, ldx, pdt, ldt, pA, pB, ldb, pC, ldc, _DT[ty], pD, pbias),
            N, G, bshape)


_seg = 0   # rows between two saved states


def _saved_numel(B, T, D, N):
    global _seg
    if _seg == 0:
        _seg = load().mg_selective_scan_saved_rows()
    return B * -(-T // _seg) * D * N


def mg_selective_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, h0=None, *, softplus=True,
                          cu_seqlens=None, save=False, out=None, ws=None, stream=None):
    """(y (B,T,D), h_last (sequences, D, N), saved): the selective scan
      h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,  y_t = C_t h_t + D x_t,
    delta = softplus(dt + dt_bias) (without softplus: dt + dt_bias), from h0.
    x, dt (B,T,D); A (D,N), N <= 64; B, C (B,T,G,N), or (B,T,N) for one group;
    channel d reads group d // (D/G).  saved, with save=True, is what
    mg_selective_scan_bwd needs of this call; else None."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_selective_scan_fwd(x, dt, A, B, C, D, dt_bias, h0, softplus=softplus,
                                         cu_seqlens=cu_seqlens, save=save, out=out, ws=ws)
    keep, words, N, G, _ = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    x = keep[0]
    Bx, T, Dx = x.shape
    cu, pcu, nseq = _sequences(cu_seqlens, x, Bx)
    states = (nseq, Dx, N)
    h0, ph0 = _param(h0, "h0", states)
    y, py = _new(out, 0, x.shape, x, x.dtype)
    h_last, pl = _new(out, 1, states, x, _F32)
    saved, psv = _new(out, 2, (_saved_numel(Bx, T, Dx, N),), x, _F32) if save else (None, 0)
    sh = _stream(x)
    _run_ws("mg_selective_scan_fwd",
            lambda: load().mg_selective_scan_fwd_workspace_size(Bx, T, Dx, N, G, nseq), x.device, ws,
            (*words, 1 if softplus else 0, ph0, pcu, nseq, py, pl, psv, Bx, T, Dx, N, G), sh)
    return y, h_last, saved


def mg_selective_scan_bwd(dy, saved, x, dt, A, B, C, D=None, dt_bias=None, h0=None, dh_last=None, *,
                          softplus=True, cu_seqlens=None, out=None, ws=None, stream=None):
    """(dx, ddt, dA, dB, dC, dD, ddt_bias, dh0): gradients of sum(dy*y) +
    sum(dh_last*h_last) for mg_selective_scan_fwd on the same inputs, with the
    `saved` that it returned.  dD, ddt_bias and dh0 are None where their input
    is."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_selective_scan_bwd(dy, saved, x, dt, A, B, C, D, dt_bias, h0, dh_last,
                                         softplus=softplus, cu_seqlens=cu_seqlens, out=out, ws=ws)
    keep, words, N, G, bshape = _scan_args(x, dt, A, B, C, D, dt_bias, 2)
    x, ty = keep[0], keep[0].dtype
    dy, pdy, lddy = _rows(dy, "dy", (ty,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    Bx, T, Dx = x.shape
    cu, pcu, nseq = _sequences(cu_seqlens, x, Bx)
    states = (nseq, Dx, N)
    h0, ph0 = _param(h0, "h0", states)
    dh_last, pdl = _param(dh_last, "dh_last", states)
    if saved is None:
        raise ValueError("saved must be what mg_selective_scan_fwd returned with save=True")
    saved, psv = _param(saved, "saved", (_saved_numel(Bx, T, Dx, N),))
    dx, pdx = _new(out, 0, x.shape, x, ty)
    ddt, pddt = _new(out, 1, x.shape, x, ty)
    dA, pdA = _new(out, 2, (Dx, N), x, _F32)
    dB, pdB = _new(out, 3, bshape, x, ty)
    dC, pdC = _new(out, 4, bshape, x, ty)
    dD, pdD = _new(out, 5, (Dx,), x, _F32) if D is not None else (None, 0)
    ddt_bias, pdbias = _new(out, 6, (Dx,), x, _F32) if dt_bias is not None else (None, 0)
    dh0, pdh0 = _new(out, 7, states, x, _F32) if h0 is not None else (None, 0)
    sh = _stream(x)
    _run_ws("mg_selective_scan_bwd",
            lambda: load().mg_selective_scan_bwd_workspace_size(Bx, T, Dx, N, G, nseq), x.device, ws,
            (pdy, lddy, psv, *words, 1 if softplus else 0, ph0, pdl, pcu, nseq, pdx, pddt, pdA, pdB, pdC,
             pdD, pdbias, pdh0, Bx, T, Dx, N, G), sh)
    return dx, ddt, dA, dB, dC, dD, ddt_bias, dh0


def mg_selective_scan_step(x, dt, A, B, C, state, D=None, dt_bias=None, *, slots=None, softplus=True,
                           out=None, stream=None):
    """y (B, D): one token a row through mg_selective_scan_fwd's recurrence.
    x, dt (B, D); B, C (B, G, N) or (B, N).  Row i's state is state[slots[i]]
    (state[i] without slots) of (states, D, N) float32, updated in place; a
    row whose slot is not in the pool is idle: y 0, no state written."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_selective_scan_step(x, dt, A, B, C, state, D, dt_bias, slots=slots,
                                          softplus=softplus, out=out)
    keep, words, N, G, _ = _scan_args(x, dt, A, B, C, D, dt_bias, 1)
    x = keep[0]
    Bx, Dx = x.shape
    ps = _state(state, "state", _F32, (Dx, N))
    slots, psl = _slots(slots, state, Bx)
    y, py = _new(None if out is None else (out,), 0, (Bx, Dx), x, x.dtype)
    _run("mg_selective_scan_step", *words, 1 if softplus else 0, ps, state.shape[0], psl, py, Bx, Dx, N, G,
         _stream(x))
    return y


# -------------------------------------------------------------- group norm

MG_GATE_NONE, MG_GATE_AFTER, MG_GATE_FIRST = range(3)


def _norm_args(x, w, bias, z, groups, gate_first):
    x, px, ldx = _rows(x, "x", _ACTIVATIONS)
    shape = x.shape
    if len(shape) < 1:
        raise ValueError("x must be (..., D)")
    D = shape[-1]
    if groups < 1 or D % groups:
        raise ValueError("the channels must be a multiple of groups")
    pz, ldz, gate = 0, D, MG_GATE_NONE
    if z is not None:
        z, pz, ldz = _rows(z, "z", (x.dtype,))
        if z.shape != shape:
            raise ValueError("z must have x's shape")
        gate = MG_GATE_FIRST if gate_first else MG_GATE_AFTER
    elif gate_first:
        raise ValueError("gate_first needs z")
    w, pw = _param(w, "w", (D,))
    if w is None:
        raise ValueError("w must be (D,)")
    bias, pb = _param(bias, "bias", (D,))
    return (x, z, w, bias), (px, ldx, pz, ldz, _DT[x.dtype], pw, pb), gate, x.numel() // D if D else 0, D


def mg_group_norm_fwd(x, w, bias=None, z=None, *, groups=1, eps=1e-5, rms=False, gate_first=False,
                      act="silu", out=None, stream=None):
    """(y, stats): each row of x (..., D) in `groups` groups of neighbouring
    channels, each normalised by itself (rms: without taking the mean out),
    o = n w + bias; y = o act(z), or with gate_first the norm is of x act(z)
    and y = o, or without z y = act(o).  act "silu" or None; groups of at most
    16384 channels.  stats (rows, groups, 2) is for mg_group_norm_bwd."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_group_norm_fwd(x, w, bias, z, groups=groups, eps=eps, rms=rms,
                                     gate_first=gate_first, act=act, out=out)
    keep, words, gate, M, D = _norm_args(x, w, bias, z, groups, gate_first)
    x = keep[0]
    y, py = _new(out, 0, x.shape, x, x.dtype)
    stats, pst = _new(out, 1, (M, groups, 2), x, _F32)
    _run("mg_group_norm_fwd", *words, float(eps), 1 if rms else 0, gate, _silu(act), py, pst, M, D, groups,
         _stream(x))
    return y, stats


def mg_group_norm_bwd(dy, stats, x, w, bias=None, z=None, *, groups=1, eps=1e-5, rms=False,
                      gate_first=False, act="silu", out=None, ws=None, stream=None):
    """(dx, dw, dbias, dz): gradients of sum(dy*y) for mg_group_norm_fwd on the
    same inputs, with the stats that it returned (eps is in them already);
    dbias and dz are None without bias and z."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return mg_group_norm_bwd(dy, stats, x, w, bias, z, groups=groups, eps=eps, rms=rms,
                                     gate_first=gate_first, act=act, out=out, ws=ws)
    keep, words, gate, M, D = _norm_args(x, w, bias, z, groups, gate_first)
    x, ty = keep[0], keep[0].dtype
    dy, pdy, lddy = _rows(dy, "dy", (ty,))
    if dy.shape != x.shape:
        raise ValueError("dy must have x's shape")
    if stats is None:
        raise ValueError("stats must be what mg_group_norm_fwd returned")
    stats, pst = _param(stats, "stats", (M, groups, 2))
    dx, pdx = _new(out, 0, x.shape, x, ty)
    dw, pdw = _new(out, 1, (D,), x, _F32)
    dbias, pdb = _new(out, 2, (D,), x, _F32) if bias is not None else (None, 0)
    dz, pdz = _new(out, 3, x.shape, x, ty) if z is not None else (None, 0)
    sh = _stream(x)
    _run_ws("mg_group_norm_bwd", lambda: load().mg_group_norm_workspace_size(M, D, groups), x.device, ws,
            (pdy, lddy, pst, *words, 1 if rms else 0, gate, _silu(act), pdx, pdz, pdw, pdb, M, D, groups), sh)
    return dx, dw, dbias, dz


causal_conv_fwd = mg_causal_conv_fwd
causal_conv_bwd = mg_causal_conv_bwd
causal_conv_step = mg_causal_conv_step
selective_scan_fwd = mg_selective_scan_fwd
selective_scan_bwd = mg_selective_scan_bwd
selective_scan_step = mg_selective_scan_step
group_norm_fwd = mg_group_norm_fwd
group_norm_bwd = mg_group_norm_bwd
