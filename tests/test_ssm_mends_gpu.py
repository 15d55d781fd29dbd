"""Calls of the selective mixer's operators that once came out wrong or were
refused, against the float64 oracle (tolerances as in test_ssm_gpu.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ssm as o
from test_ssm_gpu import BF16, DEV, F32, Scan, _conv, _dev, _nan, _near, _norm, _np, _rng

pytestmark = pytest.mark.gpu


def test_slots_on_any_8_byte_boundary(cuda_lib):
    """The C calls take slots aligned as int64 is; the binding passes a slice of
    a longer array in place."""
    mg = cuda_lib
    lib = mg.load()
    x, A, bc = torch.randn(3, 24, device=DEV), -torch.rand(24, 16, device=DEV), torch.randn(3, 16, device=DEV)
    w, all_slots = torch.randn(24, 4, device=DEV), torch.tensor([9, 2, 0, 3], device=DEV)
    slots = all_slots[1:]
    assert slots.data_ptr() % 16 == 8
    pools = [torch.randn(4, 24, 16, device=DEV), torch.randn(4, 3, 24, device=DEV)]
    want = [p.clone() for p in pools]
    aligned = slots.clone()
    wy = [mg.selective_scan_step(x, x, A, bc, bc, want[0], slots=aligned), mg.causal_conv_step(x, w, want[1], slots=aligned)]
    y = torch.empty(2, 3, 24, device=DEV)
    assert lib.mg_selective_scan_step(x.data_ptr(), 24, x.data_ptr(), 24, A.data_ptr(), bc.data_ptr(), 16, bc.data_ptr(),
                                      16, 0, None, None, 1, pools[0].data_ptr(), 4, slots.data_ptr(), y[0].data_ptr(),
                                      3, 24, 16, 1, torch.cuda.current_stream().cuda_stream) == mg.MG_OK
    assert torch.equal(y[0], wy[0]) and torch.equal(pools[0], want[0])
    assert torch.equal(mg.causal_conv_step(x, w, pools[1], slots=slots), wy[1]) and torch.equal(pools[1], want[1])


def _same_finite(name, got, want, scale, count):
    """Finite where the oracle is, and near it there."""
    fin = np.isfinite(want)
    assert np.array_equal(np.isfinite(_np(got)), fin), name
    got = torch.where(torch.from_numpy(fin).to(DEV), got, torch.zeros_like(got))
    _near(name, got, np.where(fin, want, 0.0), np.where(np.isfinite(scale), scale, 0.0), count)


@pytest.mark.parametrize("N", [1, 3, 5, 12, 16, 24, 33, 48])
@pytest.mark.parametrize("T,at", [(1, 0), (37, 20), (700, 3)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_inputs_with_any_number_of_states(cuda_lib, N, T, at, dtype):
    """An infinite x or step reaches its own channel from that row on, whatever
    the padding of the states."""
    for which in ("x", "raw"):
        c = Scan(cuda_lib, 1, T, 21, N, dtype=dtype, seed=N + T)
        getattr(c, which)[0, at, 7] = float("inf")
        getattr(c, "n" + which)[0, at, 7] = float("inf")
        with np.errstate(invalid="ignore"):
            wy, wl, _ = o.scan_fwd(*c.oracle_inputs(), c.sp)
            sy, sl, _ = o.scan_fwd(*c.oracle_inputs(), c.sp, absolute=True)
        assert not np.isfinite(wy[0, at:, 7]).any()
        y, last, _ = c.forward()
        _same_finite("y", y, wy, sy, T + N)
        _same_finite("h_last", last, wl, sl, T + N)
        if T == 1:
            pool = c.h0.clone()
            y = cuda_lib.selective_scan_step(c.x[:, 0], c.raw[:, 0], c.A, c.Bm[:, 0], c.Cm[:, 0], pool, c.Ds, c.bias)
            _same_finite("token", y, wy[:, 0], sy[:, 0], 1 + N)
            _same_finite("state", pool, wl, sl, 1 + N)


@pytest.mark.parametrize("N", [1, 5, 12, 16, 24, 33])
@pytest.mark.parametrize("T,at", [(37, 20), (700, 650)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_before_an_infinite_step(cuda_lib, N, T, at, dtype):
    """An infinite step cuts the rows before it off: their gradients are finite
    by the formulas, whatever the padding of the states."""
    c = Scan(cuda_lib, 1, T, 21, N, dtype=dtype, seed=N + T)
    c.raw[0, at, 7] = float("inf")
    c.nraw[0, at, 7] = float("inf")
    _, _, saved = c.forward()
    got = c.backward(saved)
    with np.errstate(invalid="ignore"):
        more = (c.ndl, c.sp, c.softplus)
        want = o.scan_bwd(c.ndy, *c.oracle_inputs(), *more)
        scale = o.scan_bwd(c.ndy, *c.oracle_inputs(), *more, absolute=True)
    counts = (T, T, 2 * T, T + 21, T + 21, T, 2 * T, T)
    for name, g, w, s, n in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), got, want, scale, counts):
        if name in ("dx", "ddt", "dB", "dC"):
            assert np.isfinite(w[0, :at]).all()
        _same_finite(name, g, w, s, n + N)


@pytest.mark.parametrize("N,G,cu", [(16, 1, None), (12, 3, None), (5, 1, [0, 3, 20, 37]), (16, 1, [0, 37, 37])], ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gradients_of_an_infinite_last_row(cuda_lib, N, G, cu, dtype):
    """An infinite x in the batch's last row leaves dA finite by the formulas
    (no row follows), also where that row is not the last of a tile."""
    c = Scan(cuda_lib, 1 if cu else 2, 37, 21, N, G=G, cu=cu, dtype=dtype, seed=N)
    c.x[-1, 36, 7] = float("inf")
    c.nx[-1, 36, 7] = float("inf")
    _, _, saved = c.forward()
    got = c.backward(saved)
    with np.errstate(invalid="ignore"):
        more = (c.ndl, c.sp, c.softplus)
        want = o.scan_bwd(c.ndy, *c.oracle_inputs(), *more)
        scale = o.scan_bwd(c.ndy, *c.oracle_inputs(), *more, absolute=True)
    assert np.isfinite(want[2]).all()
    counts = (37, 37, 111, 58, 58, 74, 111, 37)
    for name, g, w, s, n in zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0"), got, want, scale, counts):
        _same_finite(name, g, w, s, n + N)


def test_prompts_outside_the_pool_leave_it_alone(cuda_lib):
    """The layer's prompts with idle slots: their outputs are those of fresh
    sequences, and no entry of the pool changes for them."""
    from linear_recurrence_scans_gb300.mixer import SelectiveMixer, States
    m = SelectiveMixer(width=32, channels=48, states=16, dtype=F32, seed=2)
    u = torch.randn(3, 9, 32, device=DEV)
    fresh = m.prompt(u)
    states = States(m, 3)
    for t in (states.conv, states.scan):
        t.normal_()
    before = states.conv.clone(), states.scan.clone()
    for _ in range(2):
        out = m.prompt(u, states, torch.tensor([-1, 7, 1 << 40], device=DEV))
        assert torch.equal(out, fresh)
        assert torch.equal(states.conv, before[0]) and torch.equal(states.scan, before[1])
    m.prompt(u, states, torch.tensor([-1, 2, 3], device=DEV))
    assert torch.equal(states.scan[:2], before[1][:2]) and not torch.equal(states.scan[2], before[1][2])
    y = m.token(u[:, 0], states, torch.tensor([2, -1, 0], device=DEV))
    assert (y[1] == 0).all()
