"""The kernels that widths and row strides choose between, each against the
float64 oracle (tolerances as in test_ssm_gpu.py): convolutions of four, two
and one channel a thread, norms of groups and rows that 16-byte vectors do not
fit."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ssm as o
from test_ssm_gpu import BF16, DEV, F32, PACKS, _dev, _framed, _nan, _near, _np, _rng

pytestmark = pytest.mark.gpu


def _strided(r, B, T, D, pad, dtype):
    """(B, T, D) inside rows of D + pad values, the others NaN."""
    t, n = _dev(r.normal(size=(B, T, D)), dtype)
    return (_framed(t, 0, pad) if pad else t), n


def _conv(mg, B, T, D, W, dtype, pads=(0, 0), cu=None, seed=0, act="silu", x0=True):
    r = _rng(seed)
    sp = o.spans(B, T, cu)
    cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)
    (x, nx), (dy, ndy) = (_strided(r, B, T, D, p, dtype) for p in pads)
    w, nw = _dev(r.normal(size=(D, W)))
    b, nb = _dev(r.normal(size=D))
    e = (len(sp), W - 1, D)
    e0, ne0 = _dev(r.normal(size=e) if x0 else None, dtype)
    dl, ndl = _dev(r.normal(size=e) if x0 else None, dtype)
    kw = dict(silu=act is not None)
    y, last = mg.causal_conv_fwd(x, w, b, e0, act=act, cu_seqlens=cu_dev, out=(_nan((B, T, D), dtype), _nan(e, dtype)))
    wy, wl = o.conv_fwd(nx, nw, nb, ne0, sp, **kw)
    sy, _ = o.conv_fwd(nx, nw, nb, ne0, sp, **kw, absolute=True)
    _near("y", y, wy, sy, W)
    assert np.array_equal(_np(last), wl)
    out = (_nan((B, T, D), dtype), _nan(w.shape), _nan((D,)), _nan(e, dtype))
    got = mg.causal_conv_bwd(dy, x, w, b, e0, dl, act=act, cu_seqlens=cu_dev, out=out)
    want = o.conv_bwd(ndy, nx, nw, nb, ne0, ndl, sp, **kw)
    scale = o.conv_bwd(ndy * (1 + sy), nx, nw, nb, ne0, ndl, sp, **kw, absolute=True)
    for n, g, v, s, c in zip(("dx", "dw", "dbias", "dx0"), got, want, scale, (W, B * T, B * T, W)):
        if g is not None:
            _near(n, g, v, s, c)
    again = mg.causal_conv_bwd(dy, x, w, b, e0, dl, act=act, cu_seqlens=cu_dev)
    assert all(a is None or torch.equal(a, g) for a, g in zip(again, got))
    mg.workspace_status()


@pytest.mark.parametrize("W", range(1, 9))
@pytest.mark.parametrize("D,pads", [(40, (0, 0)), (42, (0, 0)), (40, (2, 0)), (40, (4, 6)), (41, (0, 0)), (40, (1, 0)),
                                    (42, (0, 3))], ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_taps_at_every_vector_width(cuda_lib, W, D, pads, dtype):
    _conv(cuda_lib, 2, 37, D, W, dtype, pads, seed=W + D)


@pytest.mark.parametrize("shape", [(1, 1, 2), (3, 2, 2), (2, 129, 130), (1, 200, 1002), (2, 5, 258), (1, 700, 66)], ids=str)
@pytest.mark.parametrize("pads", [(0, 0), (2, 6), (8, 4)], ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_of_two_channels_a_thread(cuda_lib, shape, pads, dtype):
    _conv(cuda_lib, *shape, 4, dtype, pads, seed=sum(shape), act="silu" if shape[1] != 5 else None)


@pytest.mark.parametrize("cu", PACKS + [[0, 2, 3, 5, 5, 6, 7, 60]], ids=lambda c: f"{len(c) - 1}seq{c[-1]}")
@pytest.mark.parametrize("D,pads", [(70, (0, 0)), (72, (2, 2)), (71, (0, 1))], ids=str)
@pytest.mark.parametrize("W", [2, 4, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_packed_at_every_vector_width(cuda_lib, cu, D, pads, W, dtype):
    _conv(cuda_lib, 1, cu[-1], D, W, dtype, pads, cu=cu, seed=len(cu) + W, x0=W != 4)


@pytest.mark.parametrize("M,D,G,pad", [(3, 8193, 1, 0), (2, 8204, 1, 0), (2, 12002, 1, 0), (2, 16383, 1, 0), (1, 16380, 1, 0),
                                       (9, 64, 1, 1), (300, 128, 2, 3), (5, 1024, 1, 7), (3, 4096, 1, 1), (33, 40, 5, 2),
                                       (2, 16384, 1, 1), (4, 2048, 16, 5)], ids=str)
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_of_wide_groups_and_odd_strides(cuda_lib, M, D, G, pad, gate, dtype):
    mg, r = cuda_lib, _rng(M + D)
    (x, nx), (z, nz), (dy, ndy) = (_strided(r, 1, M, D, p, dtype) for p in (pad, pad and pad + 1, pad))
    x, z, dy, nx, nz, ndy = x[0], z[0], dy[0], nx[0], nz[0], ndy[0]
    if gate == "none":
        z = nz = None
    w, nw = _dev(1 + 0.1 * r.normal(size=D))
    b, nb = _dev(r.normal(size=D))
    rms = gate == "first"
    kw = dict(groups=G, rms=rms, gate_first=gate == "first")
    okw = dict(G=G, eps=1e-5, rms=rms, gate_first=gate == "first")
    y, stats = mg.group_norm_fwd(x, w, b, z, **kw, out=(_nan((M, D), dtype), _nan((M, G, 2))))
    _near("y", y, o.norm_fwd(nx, nw, nb, nz, **okw)[0], o.norm_fwd(nx, nw, nb, nz, **okw, absolute=True)[0], D // G)
    out = (_nan((M, D), dtype), _nan((D,)), _nan((D,)), _nan((M, D), dtype))
    got = mg.group_norm_bwd(dy, stats, x, w, b, z, **kw, out=out)
    want, scale = (o.norm_bwd(ndy, nx, nw, nb, nz, **okw, absolute=a) for a in (False, True))
    for n, g, v, s, c in zip(("dx", "dw", "dbias", "dz"), got, want, scale, (D // G, M + D // G, M, D // G)):
        if g is not None:
            _near(n, g, v, s, c)
