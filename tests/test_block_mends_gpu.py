"""GPU checks of the gated block's operators beside test_block_gpu.py's, whose
tolerances they take where they name none."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import block as o
from test_block_gpu import SIZES, Scan, _near, _np

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


# ------------------------------------------------------- the gates' gradients

def _near_dg(c, dg, heads=slice(None)):
    """Each head's dg as a whole.  dg_t is a sum over the rows of t's chunk of the
    products q_n dq_n and k_n dk_n, each of which carries errors of its own, of no
    common sign: together 2^-24 sqrt(count) of the products' norm; 4 times that.
    The bound is far below dg itself, or the check would say nothing."""
    H = c.nv.shape[2]
    q, k = (np.repeat(x, H // x.shape[2], 2) for x in (c.nq, c.nk))
    dq, dk, _, want, _ = o.scan_bwd(c.ndo, q, k, c.nv, c.ng, c.scale, c.nS0, c.ndl, c.sp)
    squares, near = ((q * dq) ** 2 + (k * dk) ** 2).sum(-1), np.zeros_like(want)
    chunk = 128 if c.dtype == BF16 else 64
    for b, lo, hi in c.sp:
        for at in range(lo, hi, chunk):
            end = min(hi, at + chunk)
            near[b, at:end] = squares[b, at:end].sum(0)
    norm = lambda x: np.sqrt((x ** 2).sum((0, 1)))  # noqa: E731
    bound, size = 2.0 ** -22 * np.sqrt(c.count) * norm(np.sqrt(near)), norm(want)
    assert (bound < 1e-3 * size).all(), (bound / size).max()
    off = norm(_np(dg) - want)
    assert (off <= bound).all(), (off / bound).max()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_gates_gradients_as_a_whole(cuda_lib, sizes, dtype):
    for gates in ("mixed", "none"):
        c = Scan(cuda_lib, *sizes, dtype=dtype, seed=sum(sizes), gates=gates)
        _near_dg(c, c.backward(c.forward()[2])[3])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gates_gradients_as_a_whole_elsewhere(cuda_lib, dtype):
    """Packed sequences, no states, many rows, heads in parts."""
    for c in (Scan(cuda_lib, 1, 300, 4, 2, 72, 80, dtype=dtype, cu=[0, 0, 5, 5, 6, 134, 134, 263, 300], seed=40),
              Scan(cuda_lib, 2, 150, 2, 1, 48, 64, dtype=dtype, state=False, dl=False, seed=41),
              Scan(cuda_lib, 1, 1500, 2, 1, 80, 96, dtype=dtype, gates="mild", seed=42),
              Scan(cuda_lib, 20, 129, 9, 1, 40, 24, dtype=dtype, seed=43)):
        _near_dg(c, c.backward(c.forward()[2])[3])


# --------------------------------------------- segments of many chunks (bf16)

def _segments(mg, B, T, H, N, P, nseq, packed):
    """How many segments the bf16 kernels cut a batch into, from what they save:
    states of every chunk and segment, a float and two times 128 sums a chunk."""
    state = -(-P // 4) * 4 * N
    chunks = T // 128 + min(nseq, T) if packed else B * -(-T // 128)
    rest = mg.load().mg_gated_scan_saved_size(B, T, H, N, P, nseq, packed, mg.MG_BF16) - chunks * H * (state * 4 + 1024) - -(-chunks * H * 4 // 16) * 16
    assert rest % (H * state * 4) == 0
    return rest // (H * state * 4)


# heads' sizes: both above 64, with rows on 16-byte boundaries and without; one of them; none
LONG = [(52, 1100, 2, 1, 128, 128), (52, 1100, 2, 2, 72, 72), (52, 1100, 2, 1, 71, 65), (104, 700, 2, 1, 128, 64), (52, 700, 2, 2, 40, 128),
        (104, 700, 2, 1, 64, 64), (104, 700, 2, 2, 33, 17)]


def _repeated(c, times, cu=None):
    """The case's batch `times` times over: what every copy must give is the same."""
    def more(x):
        return None if x is None else torch.cat([x] * times, 1 if cu is not None and x.shape[0] == 1 and x is not c.S0 and x is not c.dl else 0)
    args = [more(x) for x in (c.q, c.k, c.v, c.g, c.S0)]
    kw = dict(scale=c.scale, cu_seqlens=cu)
    oo, last, saved = c.mg.gated_scan_fwd(*args, **kw, save=True)
    out = [oo, last, *c.mg.gated_scan_bwd(more(c.do), saved, *args, more(c.dl), **kw)]
    plain = c.mg.gated_scan_fwd(*args, **kw)
    assert torch.equal(plain[0], oo) and torch.equal(plain[1], last)
    ones = []
    for i, x in enumerate(out):
        if x is None:
            ones.append(None)
            continue
        parts = x.chunk(times, 1 if cu is not None and i not in (1, 6) else 0)
        assert all(torch.equal(p, parts[0]) for p in parts[1:]), i
        ones.append(parts[0])
    return ones


def _check_all(c, got):
    want = [*o.scan_fwd(*c.args(), c.sp)[:2], *o.scan_bwd(c.ndo, *c.args(), c.ndl, c.sp)]
    size = [*o.scan_fwd(*c.args(), c.sp, absolute=True)[:2], *o.scan_bwd(c.ndo, *c.args(), c.ndl, c.sp, absolute=True)]
    for name, a, b, s in zip(("o", "S_last", "dq", "dk", "dv", "dg", "dS0"), got, want, size):
        if a is not None:
            _near(name, a, b, s, c.count + 128, name in ("o", "dq", "dk", "dv"))
    _near_dg(c, got[5])


@pytest.mark.parametrize("state", [True, False], ids=["states", "zeros"])
@pytest.mark.parametrize("sizes", LONG, ids=lambda s: "x".join(map(str, s)))
def test_segments_of_many_chunks(cuda_lib, sizes, state):
    """Walks of six to nine chunks, the last one ragged, in one segment a sequence."""
    B, T, H, G, N, P = sizes
    assert _segments(cuda_lib, B, T, H, N, P, B, 0) == B
    c = Scan(cuda_lib, 2, T, H, G, N, P, dtype=BF16, seed=sum(sizes), gates="mild", state=state, dl=state)
    _check_all(c, _repeated(c, B // 2))


@pytest.mark.parametrize("sizes", [(2, 1, 128, 128), (2, 2, 72, 72), (2, 1, 71, 65), (4, 2, 128, 64), (4, 1, 24, 40)], ids=lambda s: "x".join(map(str, s)))
def test_segments_of_many_chunks_packed(cuda_lib, sizes):
    """Sequences of one row to eleven chunks, most of them in a segment or two."""
    H, G, N, P = sizes
    lens, times = [1100, 1, 700, 0, 1400, 129], 12
    cu = [0, *np.cumsum(lens)]
    c = Scan(cuda_lib, 1, int(cu[-1]), H, G, N, P, dtype=BF16, cu=[int(x) for x in cu], seed=sum(sizes), gates="mild")
    whole = torch.tensor([0, *np.cumsum(lens * times)], dtype=torch.int64, device=DEV)
    T, n = int(whole[-1]), len(lens) * times
    assert _segments(cuda_lib, 1, T, H, N, P, n, 1) - n <= T // (5 * 128)   # segments of five chunks or more
    _check_all(c, _repeated(c, times, whole))


# ------------------------------------------------------- one rounding (bf16)

@pytest.mark.parametrize("sizes", [(2, 300, 2, 1, 128, 128), (2, 300, 2, 2, 71, 65), (2, 300, 4, 2, 128, 64), (2, 300, 2, 1, 40, 128), (2, 300, 4, 1, 64, 64),
                                   (2, 300, 4, 2, 23, 41), (20, 129, 9, 1, 40, 24)], ids=lambda s: "x".join(map(str, s)))
def test_activations_are_rounded_once(cuda_lib, sizes):
    """o, dq, dk and dv have the error of the exact values rounded at their store.
    What their sums lose besides is 2^-16 of a term at a time, of no common sign:
    2^-8 of the rounding's error, in quadrature 2^-17; some values near a border go
    to the other side.  1% is ample; a rounding of operands of its own adds 41%."""
    for state in (True, False):
        c = Scan(cuda_lib, *sizes, dtype=BF16, seed=50 + sum(sizes), gates="mild", state=state, dl=state)
        oo, _, saved = c.forward()
        want = [o.scan_fwd(*c.args(), c.sp)[0], *o.scan_bwd(c.ndo, *c.args(), c.ndl, c.sp)[:3]]
        for name, got, exact in zip(("o", "dq", "dk", "dv"), [oo, *c.backward(saved)[:3]], want):
            once = np.linalg.norm(_np(torch.from_numpy(exact).bfloat16()) - exact)
            assert np.linalg.norm(_np(got) - exact) <= 1.01 * once, (name, np.linalg.norm(_np(got) - exact) / once)


# -------------------------------------------------- launches of the norm

@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_norm_on_both_sides_of_each_launch(cuda_lib, dtype, pad):
    """Widths around those where the kernels' shape changes: vectors a thread,
    threads a block, rows copied ahead; and some between."""
    mg = cuda_lib
    edges = [32, 64, 128, 256, 498, 512, 1024, 2768, 4096, 5544, 8192, 8520, 16376]
    widths = sorted({d + i for d in edges for i in (-8, -1, 0, 1, 2, 8) if 0 < d + i <= 16384} | {9, 700, 1111, 3001, 6000, 7001, 10000, 12345, 16378, 16383, 16384})
    torch.manual_seed(60 + pad)
    for D in widths:
        x, res, dy, dr = (torch.randn(3, D + pad, device=DEV).to(dtype)[:, :D] for _ in range(4))
        w = 1 + 0.1 * torch.randn(D, device=DEV)
        y, r, rstd = mg.rms_norm_fwd(x, w, res)
        dx, dw = mg.rms_norm_bwd(dy, rstd, r, w, dr)
        args = (*(_np(t) for t in (dy, r, w)), 1e-5, _np(dr))
        want = o.norm_fwd(_np(r), _np(w), 1e-5)[0]
        _near(("y", D), y, want, np.abs(want), 8)
        for name, a, b, s in zip(("dx", "dw"), (dx, dw), o.norm_bwd(*args), o.norm_bwd(*args, absolute=True)):
            _near((name, D), a, b, s, D if name == "dx" else 3)
