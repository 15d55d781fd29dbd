"""CPU pins of the mixer operators' float64 oracle (oracle/ssm.py): closed
forms, and every gradient against central differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import ssm as o

EPS = 1e-5


def _rng(seed):
    return np.random.default_rng(seed)


def _central(f, x, h=1e-5):
    """df/dx of a scalar function by central differences, element by element."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f()
        x[i] = keep - h
        g[i] = (up - f()) / (2 * h)
        x[i] = keep
    return g


def _close(a, b):
    if not b.size:
        return
    # the differences' own error: h^2 f''' / 6 and eps f / h, with values of order 1..10
    assert np.max(np.abs(a - b)) <= 1e-7 * (1 + np.max(np.abs(b))), np.max(np.abs(a - b))


def _scan_case(seed, G=2, cu=None):
    r = _rng(seed)
    B, T, D, N = (2, 5, 4, 3) if cu is None else (1, cu[-1], 4, 3)
    sp = o.spans(B, T, cu)
    return dict(x=r.normal(size=(B, T, D)), raw=r.normal(size=(B, T, D)), A=-np.exp(r.normal(size=(D, N))),
                Bm=r.normal(size=(B, T, G, N)), Cm=r.normal(size=(B, T, G, N)), D=r.normal(size=D),
                dt_bias=r.normal(size=D), h0=r.normal(size=(len(sp), D, N)), sp=sp)


def test_scan_is_the_sum_over_earlier_rows():
    c = _scan_case(0)
    y, last, _ = o.scan_fwd(**c)
    delta = np.log1p(np.exp(c["raw"] + c["dt_bias"]))
    B, T, D = c["x"].shape
    for b in range(B):
        for d in range(D):
            g = d // 2
            h = c["h0"][b, d] * np.exp(c["A"][d] * delta[b, :, d].sum())
            for s in range(T):
                h = h + delta[b, s, d] * c["x"][b, s, d] * c["Bm"][b, s, g] * np.exp(c["A"][d] * delta[b, s + 1:, d].sum())
            assert np.allclose(h, last[b, d], rtol=1e-12)
            assert np.allclose(c["Cm"][b, -1, g] @ h + c["D"][d] * c["x"][b, -1, d], y[b, -1, d], rtol=1e-11)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 8]])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_against_differences(cu, softplus):
    c = _scan_case(1, cu=cu)
    if not softplus:
        c["raw"] = np.abs(c["raw"])
    r = _rng(2)
    dy, dl = r.normal(size=c["x"].shape), r.normal(size=c["h0"].shape)

    def loss():
        y, last, _ = o.scan_fwd(**c, use_softplus=softplus)
        return (y * dy).sum() + (last * dl).sum()

    got = o.scan_bwd(dy, **{k: v for k, v in c.items() if k not in ("sp",)}, dh_last=dl, sp=c["sp"], use_softplus=softplus)
    for name, g in zip(("x", "raw", "A", "Bm", "Cm", "D", "dt_bias", "h0"), got):
        _close(g, _central(loss, c[name]))


def test_scan_of_two_packed_sequences_is_the_two_scans():
    c = _scan_case(3, cu=[0, 3, 8])
    y, last, _ = o.scan_fwd(**c)
    for i, (lo, hi) in enumerate(((0, 3), (3, 8))):
        part = {k: (c[k][:, lo:hi] if k in ("x", "raw", "Bm", "Cm") else c[k]) for k in c}
        part["h0"], part["sp"] = c["h0"][i:i + 1], [(0, 0, hi - lo)]
        yp, lp, _ = o.scan_fwd(**part)
        assert np.array_equal(yp, y[:, lo:hi]) and np.array_equal(lp[0], last[i])


def test_scan_steps_are_the_scan():
    c = _scan_case(4)
    y, last, _ = o.scan_fwd(**c)
    state = c["h0"]
    for t in range(c["x"].shape[1]):
        yt, state = o.scan_step(c["x"][:, t], c["raw"][:, t], c["A"], c["Bm"][:, t], c["Cm"][:, t], c["D"], c["dt_bias"], state, None)
        assert np.allclose(yt, y[:, t], rtol=1e-12)
    assert np.allclose(state, last, rtol=1e-12)


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("cu", [None, [0, 1, 1, 3, 8]])
def test_conv_gradients_against_differences(W, cu):
    r = _rng(5)
    B, T, D = (2, 5, 3) if cu is None else (1, 8, 3)
    sp = o.spans(B, T, cu)
    x, w, bias = r.normal(size=(B, T, D)), r.normal(size=(D, W)), r.normal(size=D)
    x0 = r.normal(size=(len(sp), W - 1, D))
    dy, dl = r.normal(size=x.shape), r.normal(size=x0.shape)

    def loss():
        y, last = o.conv_fwd(x, w, bias, x0, sp)
        return (y * dy).sum() + (last * dl).sum()

    for g, v in zip(o.conv_bwd(dy, x, w, bias, x0, dl, sp), (x, w, bias, x0)):
        _close(g, _central(loss, v))


def test_conv_steps_are_the_convolution():
    r = _rng(6)
    x, w, x0 = r.normal(size=(2, 6, 3)), r.normal(size=(3, 4)), r.normal(size=(2, 3, 3))
    y, last = o.conv_fwd(x, w, None, x0, o.spans(2, 6))
    state = x0
    for t in range(6):
        yt, state = o.conv_step(x[:, t], w, None, state, None)
        assert np.allclose(yt, y[:, t], rtol=1e-13)
    assert np.array_equal(state, last)


@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("silu", [True, False])
def test_norm_gradients_against_differences(rms, gate, silu):
    r = _rng(7)
    M, D, G = 3, 8, 2
    x, w, bias = r.normal(size=(M, D)), r.normal(size=D), r.normal(size=D)
    z = None if gate == "none" else r.normal(size=(M, D))
    dy = r.normal(size=(M, D))
    kw = dict(G=G, eps=EPS, rms=rms, gate_first=gate == "first", silu=silu)

    def loss():
        return (o.norm_fwd(x, w, bias, z, **kw)[0] * dy).sum()

    got = o.norm_bwd(dy, x, w, bias, z, **kw)
    for g, v in zip(got, (x, w, bias, z)):
        if v is not None:
            _close(g, _central(loss, v))


def test_magnitudes_bound_the_values():
    c = _scan_case(8)
    y, last, _ = o.scan_fwd(**c)
    ya, la, _ = o.scan_fwd(**c, absolute=True)
    assert np.all(np.abs(y) <= ya + 1e-12) and np.all(np.abs(last) <= la + 1e-12)
    r = _rng(9)
    dy, dl = r.normal(size=c["x"].shape), r.normal(size=c["h0"].shape)
    more = {k: v for k, v in c.items() if k != "sp"}
    for g, s in zip(o.scan_bwd(dy, **more, dh_last=dl, sp=c["sp"]), o.scan_bwd(dy, **more, dh_last=dl, sp=c["sp"], absolute=True)):
        assert np.all(np.abs(g) <= s + 1e-12)
