"""The mixer layer's handling of its pool of states, with stand-ins for the
operators (host tensors): which entries a prompt reads and writes."""
from __future__ import annotations

import pytest
import torch

import linear_recurrence_scans_gb300 as mg
from linear_recurrence_scans_gb300.mixer import SelectiveMixer, States


@pytest.fixture
def mixer(monkeypatch):
    """A layer whose operators add 1 to the states that they are given."""
    seen = {}

    def conv(x, w, b, x0, cu_seqlens=None):
        seen["x0"] = x0.clone()
        return x, x0 + 1

    def scan(x, dt, A, B, C, D, bias, h0, cu_seqlens=None, save=False):
        seen["h0"] = h0.clone()
        return x, h0 + 1, None

    monkeypatch.setattr(mg, "causal_conv_fwd", conv)
    monkeypatch.setattr(mg, "selective_scan_fwd", scan)
    monkeypatch.setattr(mg, "group_norm_fwd", lambda y, w, z=None, **kw: (y, None))
    m = SelectiveMixer(width=8, channels=12, states=4, dtype=torch.float32, device="cpu")
    m.seen = seen
    return m


def _pool(m, count):
    states = States(m, count)
    for i in range(count):
        states.conv[i], states.scan[i] = 10.0 * (i + 1), 100.0 * (i + 1)
    return states


@pytest.mark.parametrize("slots", [[2, 0, 3], [-1, 2, 4], [9, -(1 << 40), 1 << 40], [3, -1, -1]])
def test_prompt_slots_outside_the_pool(mixer, slots):
    """As for single tokens, a slot outside the pool is no entry of it: its
    sequence begins from zero, and no entry changes."""
    states = _pool(mixer, 4)
    want = [10.0 * (i + 1) for i in range(4)]
    for _ in range(2):
        begin = [want[s] if 0 <= s < 4 else 0.0 for s in slots]
        mixer.prompt(torch.randn(3, 5, 8), states, torch.tensor(slots))
        assert mixer.seen["x0"][:, 0, 0].tolist() == begin
        for s in slots:
            if 0 <= s < 4:
                want[s] += 1
        assert states.conv[:, 0, 0].tolist() == want
        assert (states.conv == states.conv[:, :1, :1]).all() and states.conv.shape[0] == 4
        assert torch.equal(states.scan[:, 0, 0] % 10, states.conv[:, 0, 0] % 10)


@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
def test_prompt_without_slots(mixer, cu):
    """Sequence i's entry is i, as for single tokens."""
    states = _pool(mixer, 4)
    u = torch.randn(3 if cu is None else 1, 5, 8)
    mixer.prompt(u, states, cu_seqlens=None if cu is None else torch.tensor(cu))
    assert mixer.seen["h0"][:, 0, 0].tolist() == [100.0, 200.0, 300.0]
    assert states.scan[:, 0, 0].tolist() == [101.0, 201.0, 301.0, 400.0]
