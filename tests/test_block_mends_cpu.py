"""Host-side checks of the gated block's operators beside test_block_abi_cpu.py's:
sizes of nothing, copies' ranges, calls by name (no GPU needed)."""
from __future__ import annotations

import pytest

import linear_recurrence_scans_gb300 as mg


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


@pytest.mark.parametrize("dt", [mg.MG_F32, mg.MG_BF16])
@pytest.mark.parametrize("B,T,H", [(1, 8, 0), (0, 8, 2), (1, 0, 2), (0, 0, 0)])
def test_sizes_of_nothing(lib, B, T, H, dt):
    """A batch without rows or heads has nothing to save."""
    for packed in (0, 1):
        assert lib.mg_gated_scan_saved_size(B, T, H, 16, 16, B, packed, dt) == 0
        for bwd in (0, 1):
            assert lib.mg_gated_scan_workspace_size(B, T, H, 1, 16, 16, B, packed, dt, bwd) == 256
