"""GPU checks of the gated block's operators beside test_block_gpu.py's."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [F32, BF16]
IDS = ["fp32", "bf16"]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_no_heads(cuda_lib, dtype):
    """Values without heads: nothing is saved, and q and k have gradients of zero."""
    mg = cuda_lib
    q, v, g = torch.randn(2, 5, 1, 4, device=DEV).to(dtype), torch.empty(2, 5, 0, 8, device=DEV, dtype=dtype), torch.empty(2, 5, 0, device=DEV)
    o, last, saved = mg.gated_scan_fwd(q, q, v, g, save=True)
    assert o.shape == v.shape and last.shape == (2, 0, 4, 8) and saved.numel() == 0
    nan = lambda: torch.full_like(q, float("nan"))  # noqa: E731
    dq, dk, dv, dg, _ = mg.gated_scan_bwd(v, saved, q, q, v, g, out=(nan(), nan(), None, None, None))
    assert not dq.any() and not dk.any() and dv.shape == v.shape and dg.shape == g.shape
