"""The gated block's handling of its pool of states, with stand-ins for the
operators (host tensors): which entries a prompt reads and writes, and what of
the convolution's output goes where."""
from __future__ import annotations

import pytest
import torch

import linear_recurrence_scans_gb300 as mg
from linear_recurrence_scans_gb300.mixer import GatedMixer, States


@pytest.fixture
def mixer(monkeypatch):
    """A block whose operators add 1 to the states that they are given."""
    seen = {}

    def conv(x, w, b, x0, cu_seqlens=None):
        seen["x0"] = None if x0 is None else x0.clone()
        seen["conv"] = x.clone()
        return x.clone(), None if x0 is None else x0 + 1

    def scan(q, k, v, g, S0, scale, cu_seqlens=None, save=False):
        seen.update(q=q, k=k, v=v, g=g, S0=None if S0 is None else S0.clone(), scale=scale)
        return v.clone(), None if S0 is None else S0 + 1, None

    monkeypatch.setattr(mg, "rms_norm_fwd", lambda x, w, r=None: (x, x if r is None else x + r, None))
    monkeypatch.setattr(mg, "causal_conv_fwd", conv)
    monkeypatch.setattr(mg, "gated_scan_fwd", scan)
    monkeypatch.setattr(mg, "group_norm_fwd", lambda y, w, z=None, **kw: (y, None))
    m = GatedMixer(width=8, heads=4, keys=3, values=5, groups=2, dtype=torch.float32, device="cpu")
    m.seen = seen
    return m


@pytest.mark.parametrize("slots", [[2, 0, 3], [-1, 2, 4], [9, -(1 << 40), 1 << 40], [3, -1, -1]])
def test_a_prompt_reads_and_writes_its_slots_only(mixer, slots):
    states = States(mixer, 4)
    for i in range(4):
        states.conv[i], states.scan[i] = 10.0 * (i + 1), 100.0 * (i + 1)
    before = states.conv.clone(), states.scan.clone()
    mixer.prompt(torch.zeros(3, 6, 8), None, states, torch.tensor(slots))
    for i, s in enumerate(slots):
        inside = 0 <= s < 4
        assert (mixer.seen["x0"][i] == (10.0 * (s + 1) if inside else 0)).all()
        assert (mixer.seen["S0"][i] == (100.0 * (s + 1) if inside else 0)).all()
    for s in range(4):
        more = 1 if s in slots else 0
        assert torch.equal(states.conv[s], before[0][s] + more) and torch.equal(states.scan[s], before[1][s] + more)


def test_shapes_and_where_the_convolution_goes(mixer):
    states = States(mixer, 2)
    assert states.conv.shape == (2, 3, 2 * 2 * 3 + 4 * 5) and states.scan.shape == (2, 4, 3, 5)
    out, r = mixer.prompt(torch.randn(2, 6, 8), torch.randn(2, 6, 8))
    s = mixer.seen
    assert out.shape == r.shape == (2, 6, 8) and s["x0"] is None and s["S0"] is None and s["scale"] == 3 ** -0.5
    assert torch.equal(torch.cat([s[n].flatten(-2) for n in ("q", "k", "v")], -1), s["conv"])
    assert s["q"].shape == s["k"].shape == (2, 6, 2, 3) and s["v"].shape == (2, 6, 4, 5)
    assert s["g"].shape == (2, 6, 4) and s["g"].dtype == torch.float32 and (s["g"] <= 0).all()
