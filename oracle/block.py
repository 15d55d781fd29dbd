"""Float64 oracle of the gated block's operators (numpy, one row at a time).

Written from the formulas, without any code of the CUDA path; batches come as
``spans`` (see oracle/ssm.py).  With ``absolute=True`` every product enters by
its magnitude (the decays stay what they are): the scale that an output's
rounding errors are proportional to.
"""
from __future__ import annotations

import numpy as np


def _mag(absolute):
    return np.abs if absolute else (lambda v: v)


def _each(x, H):
    """(..., G, N) to (..., H, N): a group's row for each of its heads."""
    return np.repeat(x, H // x.shape[-2], -2)


def _shared(x, G):
    """(..., H, N) to (..., G, N): sums over the heads of a group."""
    return x.reshape(*x.shape[:-2], G, x.shape[-2] // G, x.shape[-1]).sum(-2)


# -------------------------------------------------------- gated recurrence

def scan_fwd(q, k, v, g, scale, S0, sp, absolute=False):
    """(o, S_last, the state before each row): q, k (B,T,G,N), v (B,T,H,P), g
    (B,T,H), S0 (nseq,H,N,P) or None."""
    m = _mag(absolute)
    H, N, P = v.shape[2], q.shape[3], v.shape[3]
    q, k, v = m(_each(q, H)), m(_each(k, H)), m(v)
    o, last = np.zeros_like(v), np.zeros((len(sp), H, N, P))
    kept = np.zeros((*v.shape[:3], N, P))
    for i, (b, lo, hi) in enumerate(sp):
        S = np.zeros((H, N, P)) if S0 is None else m(S0[i]).copy()
        for t in range(lo, hi):
            kept[b, t] = S
            S = np.exp(g[b, t])[:, None, None] * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = abs(scale) * np.einsum("hn,hnp->hp", q[b, t], S) if absolute else scale * np.einsum("hn,hnp->hp", q[b, t], S)
        last[i] = S
    return o, last, kept


def scan_bwd(do, q, k, v, g, scale, S0, dS_last, sp, absolute=False):
    """(dq, dk, dv, dg, dS0) of sum(do*o) + sum(dS_last*S_last)."""
    m = _mag(absolute)
    G, H = q.shape[2], v.shape[2]
    kept = scan_fwd(q, k, v, g, scale, S0, sp, absolute)[2]
    q, k, v, up = m(_each(q, H)), m(_each(k, H)), m(v), m(scale * do)
    dq, dk, dv, dg = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), np.zeros_like(g)
    dS0 = np.zeros((len(sp), H, q.shape[3], v.shape[3]))
    for i, (b, lo, hi) in enumerate(sp):
        D = np.zeros(dS0.shape[1:]) if dS_last is None else m(dS_last[i]).copy()
        for t in reversed(range(lo, hi)):
            a = np.exp(g[b, t])[:, None, None]
            S = a * kept[b, t] + k[b, t][:, :, None] * v[b, t][:, None, :]
            D = D + q[b, t][:, :, None] * up[b, t][:, None, :]
            dq[b, t] = np.einsum("hnp,hp->hn", S, up[b, t])
            dk[b, t] = np.einsum("hnp,hp->hn", D, v[b, t])
            dv[b, t] = np.einsum("hnp,hn->hp", D, k[b, t])
            dg[b, t] = (D * a * kept[b, t]).sum((1, 2))
            D = a * D
        dS0[i] = D
    if absolute:
        # the gate's gradient is a difference of sums over the rows near it: its
        # errors go by what those rows' q . dq and k . dk are made of
        rows = (q * dq).sum(-1) + (k * dk).sum(-1)
        for i, (b, lo, hi) in enumerate(sp):
            for t in range(lo, hi):
                dg[b, t] += rows[b, max(lo, t - 127):min(hi, t + 128)].sum(0)
    return _shared(dq, G), _shared(dk, G), dv, dg, dS0


def scan_step(q, k, v, g, scale, state, slots, absolute=False):
    """(o, new state): q, k (B,G,N), v (B,H,P), g (B,H), slots (B) or None."""
    m = _mag(absolute)
    H = v.shape[1]
    q, k, v, state, o = m(_each(q, H)), m(_each(k, H)), m(v), m(state).copy(), np.zeros_like(v)
    for i in range(len(v)):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < len(state):
            continue
        state[s] = np.exp(g[i])[:, None, None] * state[s] + k[i][:, :, None] * v[i][:, None, :]
        o[i] = (abs(scale) if absolute else scale) * np.einsum("hn,hnp->hp", q[i], state[s])
    return o, state


# ---------------------------------------------------------------- rms norm

def norm_fwd(r, w, eps):
    """(y, rstd) of rows r (M,D), the residual already added."""
    rstd = 1.0 / np.sqrt((r * r).mean(-1) + eps)
    return r * rstd[:, None] * w, rstd


def norm_quant(y, block):
    """(y / scale, scale (M, D/block)) before the rounding to 8 bits."""
    blocks = y.reshape(len(y), -1, block)
    scale = np.maximum(np.abs(blocks).max(-1), 1e-30) / 448.0
    return (blocks / scale[..., None]).reshape(y.shape), scale


def norm_bwd(dy, r, w, eps, dr=None, absolute=False):
    """(dx, dw) of sum(dy*y) + sum(dr*r)."""
    m = _mag(absolute)
    _, rstd = norm_fwd(r, w, eps)
    n = m(r * rstd[:, None])
    dn = m(dy * w)
    mean = (dn * n).mean(-1, keepdims=True)
    dx = rstd[:, None] * (dn + n * mean if absolute else dn - n * mean)
    return dx + (0.0 if dr is None else m(dr)), (m(dy) * n).sum(0)
