"""GPU checks of the gated block's operators beside test_block_gpu.py's, whose
tolerances they take where they name none."""
from __future__ import annotations

import pytest
import torch

from oracle import block as o
from test_block_gpu import _near, _np

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


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("D", range(1, 10))
def test_gradients_of_narrow_rows(cuda_lib, D, dtype):
    """Rows narrower than a 16-byte piece, several of them in the array's last
    one; behind each array lie NaNs."""
    mg = cuda_lib
    for M in (1, 2, 3, 5, 10, 11, 37, 64, 701):
        def rows():
            wide = torch.full((M * D + 64,), float("nan"), device=DEV, dtype=dtype)
            wide[:M * D].copy_(torch.randn(M * D, device=DEV))
            return wide[:M * D].view(M, D)
        torch.manual_seed(100 * D + M)
        dy, r, dr, w = rows(), rows(), rows(), 1 + 0.1 * torch.randn(D, device=DEV)
        rstd = mg.rms_norm_fwd(r, w)[2]
        dx, dw = mg.rms_norm_bwd(dy, rstd, r, w, dr)
        args = (*(_np(t) for t in (dy, r, w)), 1e-5, _np(dr))
        for name, a, b, s in zip(("dx", "dw"), (dx, dw), o.norm_bwd(*args), o.norm_bwd(*args, absolute=True)):
            _near(name, a, b, s, D if name == "dx" else M)


def test_calls_by_name(cuda_lib):
    """Every argument by its name gives the bits of the same call by position."""
    mg = cuda_lib
    q, k, do, v = (torch.randn(1, 9, 2, 8, device=DEV) for _ in range(4))
    g, S0, side = -torch.rand(1, 9, 2, device=DEV), torch.randn(1, 2, 8, 8, device=DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    want, got = mg.gated_scan_fwd(q, k, v, g, S0, save=True), mg.gated_scan_fwd(q=q, k=k, v=v, g=g, S0=S0, save=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want, got = mg.gated_scan_bwd(do, want[2], q, k, v, g, S0), mg.gated_scan_bwd(do=do, saved=want[2], q=q, k=k, v=v, g=g, S0=S0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pools = S0.clone(), S0.clone()
    row = dict(q=q[:, 0], k=k[:, 0], v=v[:, 0], g=g[:, 0])
    assert torch.equal(mg.gated_scan_step(*row.values(), pools[0]), mg.gated_scan_step(**row, state=pools[1])) and torch.equal(*pools)
    x, w, residual = torch.randn(4, 64, device=DEV), torch.rand(64, device=DEV), torch.randn(4, 64, device=DEV)
    want, got = mg.rms_norm_fwd(x, w, residual), mg.rms_norm_fwd(x=x, w=w, residual=residual)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    _, r, rstd = want
    want, got = mg.rms_norm_bwd(x, rstd, r, w), mg.rms_norm_bwd(dy=x, rstd=rstd, r=r, w=w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want, got = mg.rms_norm_quant(x, w, residual), mg.rms_norm_quant(x=x, w=w, residual=residual)
    assert all(torch.equal(a.float(), b.float()) for a, b in zip(got, want))


def test_a_stream_of_another_device_is_refused(cuda_lib):
    """The call would run on its tensors' device, behind none of that stream's work."""
    class Other:
        device, cuda_stream = torch.device("cuda", torch.cuda.device_count()), 0
    x, w = torch.randn(4, 64, device=DEV), torch.rand(64, device=DEV)
    with pytest.raises(ValueError, match="stream must be on"):
        cuda_lib.rms_norm_fwd(x, w, stream=Other())
    with pytest.raises(ValueError, match="stream must be on"):
        cuda_lib.rms_norm_fwd(x=x, w=w, stream=Other())


def test_rows_without_channels(cuda_lib):
    mg = cuda_lib
    x, w = torch.empty(3, 0, device=DEV), torch.empty(0, device=DEV)
    with pytest.raises(mg.MgScanError, match="channels"):
        mg.rms_norm_fwd(x, w)
    with pytest.raises(mg.MgScanError, match="channels"):
        mg.rms_norm_quant(x, w, x)
    assert mg.rms_norm_fwd(torch.empty(2, 0, 8, device=DEV), torch.rand(8, device=DEV))[2].shape == (2, 0)
