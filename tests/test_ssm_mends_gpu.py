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
