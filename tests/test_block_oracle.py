"""CPU pins of the gated block's float64 oracle (oracle/block.py): closed
forms, and every gradient against central differences."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import block as o
from oracle.ssm import spans

EPS = 1e-5


def _central(f, x, h=1e-5):
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
    # the differences' own error: h^2 f''' / 6 and eps f / h, with values of order 1..10
    if b.size:
        assert np.max(np.abs(a - b)) <= 1e-7 * (1 + np.max(np.abs(b))), np.max(np.abs(a - b))


def _case(seed, cu=None, G=2, H=4, N=3, P=2):
    r = np.random.default_rng(seed)
    B, T = (2, 5) if cu is None else (1, cu[-1])
    sp = spans(B, T, cu)
    n = lambda *s: r.normal(size=s)  # noqa: E731
    return dict(q=n(B, T, G, N), k=n(B, T, G, N), v=n(B, T, H, P), g=-np.abs(n(B, T, H)), scale=0.7,
                S0=n(len(sp), H, N, P), sp=sp), n(B, T, H, P), n(len(sp), H, N, P)


def test_scan_is_the_sum_over_earlier_rows():
    c, _, _ = _case(0)
    oo, last, _ = o.scan_fwd(**c)
    B, T, H, P = c["v"].shape
    for b in range(B):
        for h in range(H):
            G = np.cumsum(c["g"][b, :, h])
            q, k = c["q"][b, :, h // 2], c["k"][b, :, h // 2]
            for t in range(T):
                S = np.exp(G[t]) * c["S0"][b, h]
                for s in range(t + 1):
                    S = S + np.exp(G[t] - G[s]) * np.outer(k[s], c["v"][b, s, h])
                assert np.allclose(oo[b, t, h], 0.7 * q[t] @ S, rtol=1e-12, atol=1e-12)
            assert np.allclose(last[b, h], S, rtol=1e-12, atol=1e-12)


def test_packed_is_each_sequence_alone():
    cu = [0, 3, 3, 4, 9]
    c, _, _ = _case(1, cu)
    oo, last, _ = o.scan_fwd(**c)
    for i in range(4):
        part = {n: c[n][:, cu[i]:cu[i + 1]] for n in "qkvg"}
        alone, end, _ = o.scan_fwd(**part, scale=0.7, S0=c["S0"][i:i + 1], sp=[(0, 0, cu[i + 1] - cu[i])])
        assert np.array_equal(alone, oo[:, cu[i]:cu[i + 1]]) and np.array_equal(end[0], last[i])


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 7]])
def test_scan_gradients(cu):
    c, do, dl = _case(2, cu)

    def loss():
        oo, last, _ = o.scan_fwd(**c)
        return (oo * do).sum() + (last * dl).sum()

    got = dict(zip(("q", "k", "v", "g", "S0"), o.scan_bwd(do, c["q"], c["k"], c["v"], c["g"], 0.7, c["S0"], dl, c["sp"])))
    for name, grad in got.items():
        _close(grad, _central(loss, c[name]))


def test_steps_are_the_scan():
    c, _, _ = _case(3)
    oo, last, _ = o.scan_fwd(**c)
    state = np.concatenate([np.zeros((1, *c["S0"].shape[1:])), c["S0"][::-1]])
    for t in range(5):
        y, state = o.scan_step(c["q"][:, t], c["k"][:, t], c["v"][:, t], c["g"][:, t], 0.7, state, [2, 1])
        assert np.allclose(y, oo[:, t], rtol=1e-12, atol=1e-12)
    assert np.allclose(state[[2, 1]], last, rtol=1e-12, atol=1e-12) and not state[0].any()
    y, same = o.scan_step(c["q"][:, 0], c["k"][:, 0], c["v"][:, 0], c["g"][:, 0], 0.7, state, [-1, 3])
    assert not y.any() and np.array_equal(same, state)


def test_norm_and_its_gradients():
    r = np.random.default_rng(4)
    x, w, dy, dr = r.normal(size=(3, 6)), r.normal(size=6), r.normal(size=(3, 6)), r.normal(size=(3, 6))
    y, rstd = o.norm_fwd(x, w, EPS)
    assert np.allclose((y / w) ** 2 @ np.ones(6) / 6, 1 - EPS * rstd ** 2, rtol=1e-12)

    def loss():
        return (o.norm_fwd(x, w, EPS)[0] * dy).sum() + (x * dr).sum()

    dx, dw = o.norm_bwd(dy, x, w, EPS, dr)
    _close(dx, _central(loss, x))
    _close(dw, _central(loss, w))
    q, scale = o.norm_quant(y, 3)
    assert np.allclose(np.abs(q).reshape(3, 2, 3).max(-1), 448.0) and np.allclose(q * np.repeat(scale, 3, 1), y)
    assert np.allclose(o.norm_quant(np.zeros((1, 4)), 2)[1], 1e-30 / 448)
