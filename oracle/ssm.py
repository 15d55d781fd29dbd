"""Float64 oracle of the selective mixer's operators (numpy, one row at a time).

Written from the formulas, without any code of the CUDA path.  Batches come as
lists of sequences' bounds (``spans``: (batch index, first row, end row) for
each sequence), so a dense and a packed batch are the same loop.

With ``absolute=True`` every product enters by its magnitude (the decays stay
what they are): the result is the sum of the magnitudes of the terms of each
output, the scale that its rounding errors are proportional to.
"""
from __future__ import annotations

import numpy as np


def spans(B, T, cu=None):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(cu[i]), int(cu[i + 1])) for i in range(len(cu) - 1)]


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def _mag(absolute):
    return np.abs if absolute else (lambda v: v)


# -------------------------------------------------------------- convolution

def conv_fwd(x, w, bias, x0, sp, silu=True, absolute=False):
    """(y, x_last): x (B,T,D), w (D,W), bias (D) or None, x0 (nseq,W-1,D) or None."""
    m = _mag(absolute)
    B, T, D = x.shape
    W = w.shape[1]
    y = np.zeros_like(x)
    last = np.zeros((len(sp), W - 1, D))
    for i, (b, lo, hi) in enumerate(sp):
        rows = np.concatenate([np.zeros((W - 1, D)) if x0 is None else x0[i], x[b, lo:hi]])
        last[i] = rows[len(rows) - (W - 1):]
        for t in range(hi - lo):
            v = np.zeros(D) if bias is None else bias.copy()
            mv = m(v)
            for k in range(W):
                v = v + w[:, k] * rows[t + k]
                mv = mv + m(w[:, k] * rows[t + k])
            y[b, lo + t] = mv if absolute else (v * sigmoid(v) if silu else v)
    return y, last


def conv_bwd(dy, x, w, bias, x0, dx_last, sp, silu=True, absolute=False):
    """(dx, dw, dbias, dx0)."""
    m = _mag(absolute)
    B, T, D = x.shape
    W = w.shape[1]
    dx, dw, db = np.zeros_like(x), np.zeros_like(w), np.zeros(D)
    dx0 = np.zeros((len(sp), W - 1, D))
    for i, (b, lo, hi) in enumerate(sp):
        rows = np.concatenate([np.zeros((W - 1, D)) if x0 is None else x0[i], x[b, lo:hi]])
        d = np.zeros_like(rows)
        if dx_last is not None:
            d[len(rows) - (W - 1):] += m(dx_last[i])
        for t in range(hi - lo):
            v = np.zeros(D) if bias is None else bias.copy()
            for k in range(W):
                v = v + w[:, k] * rows[t + k]
            s = sigmoid(v)
            # |v| where the derivative's own terms may cancel
            slope = (s * (1 + m(v) * (1 - s)) if absolute else s * (1 + v * (1 - s))) if silu else 1.0
            dv = m(dy[b, lo + t]) * slope
            db += dv
            for k in range(W):
                dw[:, k] += dv * m(rows[t + k])
                d[t + k] += dv * m(w[:, k])
        dx0[i], dx[b, lo:hi] = d[:W - 1], d[W - 1:]
    return dx, dw, db, dx0


def conv_step(x, w, bias, state, slots, silu=True):
    """(y, new state): x (B,D), state (S,W-1,D), slots (B) or None."""
    state, y = state.copy(), np.zeros_like(x)
    for i in range(len(x)):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < len(state):
            continue
        rows = np.concatenate([state[s], x[i:i + 1]])
        v = np.zeros(x.shape[1]) if bias is None else bias.copy()
        for k in range(w.shape[1]):
            v = v + w[:, k] * rows[k]
        y[i] = v * sigmoid(v) if silu else v
        state[s] = rows[1:]
    return y, state


# ------------------------------------------------------------ selective scan

def _delta(raw, dt_bias, use_softplus):
    v = raw if dt_bias is None else raw + dt_bias
    return (softplus(v), sigmoid(v)) if use_softplus else (v, np.ones_like(v))


def scan_fwd(x, raw, A, Bm, Cm, D, dt_bias, h0, sp, use_softplus=True, absolute=False):
    """(y, h_last, all states): Bm, Cm (B,T,G,N); the states before each row, (B,T,D,N)."""
    m = _mag(absolute)
    Bx, T, Dx = x.shape
    G, N = Bm.shape[2:]
    group = np.arange(Dx) // (Dx // G)
    delta, _ = _delta(raw, dt_bias, use_softplus)
    y, before = np.zeros_like(x), np.zeros((Bx, T, Dx, N))
    last = np.zeros((len(sp), Dx, N))
    for i, (b, lo, hi) in enumerate(sp):
        h = np.zeros((Dx, N)) if h0 is None else m(h0[i])
        for t in range(lo, hi):
            before[b, t] = h
            h = np.exp(delta[b, t][:, None] * A) * h + m((delta[b, t] * x[b, t])[:, None] * Bm[b, t][group])
            y[b, t] = np.sum(m(Cm[b, t][group]) * h, axis=1) + (0 if D is None else m(D * x[b, t]))
        last[i] = h
    return y, last, before


def scan_bwd(dy, x, raw, A, Bm, Cm, D, dt_bias, h0, dh_last, sp, use_softplus=True, absolute=False):
    """(dx, ddt, dA, dB, dC, dD, ddt_bias, dh0)."""
    m = _mag(absolute)
    Bx, T, Dx = x.shape
    G, N = Bm.shape[2:]
    group = np.arange(Dx) // (Dx // G)
    delta, slope = _delta(raw, dt_bias, use_softplus)
    _, _, before = scan_fwd(x, raw, A, Bm, Cm, D, dt_bias, h0, sp, use_softplus, absolute)
    dx, draw, dA = np.zeros_like(x), np.zeros_like(x), np.zeros_like(A)
    dB, dC = np.zeros_like(Bm), np.zeros_like(Cm)
    dh0 = np.zeros((len(sp), Dx, N))
    per_group = lambda v: np.add.reduceat(v, np.arange(0, Dx, Dx // G), axis=0)  # noqa: E731
    for i, (b, lo, hi) in enumerate(sp):
        g = np.zeros((Dx, N)) if dh_last is None else m(dh_last[i])
        for t in reversed(range(lo, hi)):
            dl = delta[b, t][:, None]
            a, Br, Cr = np.exp(dl * A), m(Bm[b, t][group]), m(Cm[b, t][group])
            u = m(delta[b, t] * x[b, t])[:, None]
            dyr = m(dy[b, t])[:, None]
            dC[b, t] = per_group(dyr * (a * before[b, t] + u * Br))
            g = g + Cr * dyr
            dB[b, t] = per_group(g * u)
            gB = np.sum(g * Br, axis=1)
            gah = g * a * before[b, t]
            dx[b, t] = m(delta[b, t]) * gB + (0 if D is None else m(D * dy[b, t]))
            draw[b, t] = (m(x[b, t]) * gB + np.sum(m(A) * gah, axis=1)) * slope[b, t]
            dA += m(dl) * gah
            g = a * g
        dh0[i] = g
    return dx, draw, dA, dB, dC, m(dy * x).sum((0, 1)), draw.sum((0, 1)), dh0


def scan_step(x, raw, A, Bm, Cm, D, dt_bias, state, slots, use_softplus=True, absolute=False):
    """(y, new state): x, raw (B,D), Bm, Cm (B,G,N), state (S,D,N)."""
    m = _mag(absolute)
    Dx, G = x.shape[1], Bm.shape[1]
    group = np.arange(Dx) // (Dx // G)
    delta, _ = _delta(raw, dt_bias, use_softplus)
    state, y = state.copy(), np.zeros_like(x)
    for i in range(len(x)):
        s = i if slots is None else int(slots[i])
        if not 0 <= s < len(state):
            continue
        h = np.exp(delta[i][:, None] * A) * m(state[s]) + m((delta[i] * x[i])[:, None] * Bm[i][group])
        y[i] = np.sum(m(Cm[i][group]) * h, axis=1) + (0 if D is None else m(D * x[i]))
        state[s] = h
    return y, state


# --------------------------------------------------------------- group norm

def _silu(v, on):
    return v * sigmoid(v) if on else v


def _silu_grad(v, on, absolute=False):
    s = sigmoid(v)
    return s * (1 + _mag(absolute)(v) * (1 - s)) if on else np.ones_like(v)


def norm_fwd(x, w, bias, z, G, eps, rms, gate_first, silu=True, absolute=False):
    """(y, mean, rstd): x (M,D)."""
    M, D = x.shape
    p = x * _silu(z, silu) if z is not None and gate_first else x
    q = p.reshape(M, G, D // G)
    mean = np.zeros((M, G, 1)) if rms else q.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((q - mean) ** 2).mean(-1, keepdims=True) + eps)
    if absolute:
        o = ((np.abs(q) + np.abs(mean)) * rstd).reshape(M, D) * np.abs(w) + (0 if bias is None else np.abs(bias))
        return o * (np.abs(_silu(z, silu)) if z is not None and not gate_first else 1), mean, rstd
    o = ((q - mean) * rstd).reshape(M, D) * w + (0 if bias is None else bias)
    if not gate_first:
        o = o * _silu(z, silu) if z is not None else _silu(o, silu)
    return o, mean[..., 0], rstd[..., 0]


def norm_bwd(dy, x, w, bias, z, G, eps, rms, gate_first, silu=True, absolute=False):
    """(dx, dw, dbias, dz)."""
    m = _mag(absolute)
    M, D = x.shape
    shape = (M, G, D // G)
    first = z is not None and gate_first
    p = x * _silu(z, silu) if first else x
    q = p.reshape(shape)
    mean = np.zeros((M, G, 1)) if rms else q.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((q - mean) ** 2).mean(-1, keepdims=True) + eps)
    n = ((np.abs(q) + np.abs(mean) if absolute else q - mean) * rstd).reshape(M, D)
    o = n * m(w) + (0 if bias is None else m(bias))
    true_o = ((q - mean) * rstd).reshape(M, D) * w + (0 if bias is None else bias)
    do, dz = m(dy), None
    if z is not None and not first:
        dz = m(dy) * o * _silu_grad(z, silu, absolute)
        do = m(dy * _silu(z, silu))
    elif z is None:
        # errors of o move the derivative too: at most by |o| there
        do = m(dy) * (_silu_grad(true_o, silu, True) + o if absolute else _silu_grad(true_o, silu))
    dn = (do * m(w)).reshape(shape)
    nr = n.reshape(shape)
    sub = 0 if rms else dn.mean(-1, keepdims=True)
    if absolute:
        dp = rstd * (dn + sub + nr * (dn * nr).mean(-1, keepdims=True))
    else:
        dp = rstd * (dn - sub - nr * (dn * nr).mean(-1, keepdims=True))
    dx = dp.reshape(M, D)
    if first:
        dz = dx * m(x) * _silu_grad(z, silu, absolute)
        dx = dx * m(_silu(z, silu))
    return dx, (do * n).sum(0), do.sum(0), dz
