"""GPU parity of the selective mixer's operators (short causal convolution,
selective scan, gated group norm) against the float64 oracle in oracle/ssm.py,
through the public entry points.

Tolerances.  Every output is a sum of products, and its rounding error is at
most a multiple of the sum S of the magnitudes of its terms, which the oracle
gives (absolute=True).  A term passes one row's arithmetic for each row it
lives through (the decay's 2^x, within 2^-22, and two roundings of 2^-24) and
one addition for each row or channel summed: (rows + summed channels + 64)
2^-22 S covers a term that lives through the whole sequence.  A bf16 output
adds its own rounding, 2^-8 |value|.  Outputs start as NaN, so that an
unwritten element fails.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import ssm as o

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def _rng(seed):
    return np.random.default_rng(seed)


def _np(x):
    return x.detach().double().cpu().numpy()


def _dev(a, dtype=F32):
    """The array on the device, and the values that it has there in float64."""
    if a is None:
        return None, None
    t = torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)
    return t, _np(t)


def _nan(shape, dtype=F32):
    return torch.full(tuple(shape), float("nan"), dtype=dtype, device=DEV)


def _near(name, got, want, scale, count):
    got_np = _np(got)
    assert got_np.shape == want.shape, (name, got_np.shape, want.shape)
    tol = (count + 64) * 2.0 ** -22 * scale + 1e-30
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    bad = ~(np.abs(got_np - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.max(np.abs(got_np - want)[bad] / tol[bad]))


# ------------------------------------------------------------ selective scan

class Scan:
    """One case's inputs on the device (rows optionally inside wider rows) and
    in float64."""

    def __init__(self, mg, B, T, D, N, G=1, dtype=F32, cu=None, seed=0, skip=True, bias=True, h0=True,
                 softplus=True, wide=True, scale_a=1.0):
        r = _rng(seed)
        self.mg, self.dtype, self.softplus, self.cu = mg, dtype, softplus, cu
        self.B, self.T, self.D, self.N, self.G = B, T, D, N, G
        self.sp = o.spans(B, T, cu)
        S = len(self.sp)
        self.cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)
        pad = 24 if wide else 0

        def rows(width, scale=1.0):
            t = torch.from_numpy(r.normal(size=(B, T, width + pad)) * scale).to(dtype).to(DEV)
            t = t[..., :width]
            return t, _np(t)

        self.x, self.nx = rows(D)
        raw = r.normal(size=(B, T, D)) * 0.5 if softplus else np.exp(r.normal(size=(B, T, D)) - 2)
        self.raw, self.nraw = _dev(raw, dtype)
        bc, nbc = rows(2 * G * N)
        self.Bm, self.Cm = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
        self.nB, self.nC = (nbc[..., i * G * N:(i + 1) * G * N].reshape(B, T, G, N) for i in (0, 1))
        self.A, self.nA = _dev(-np.arange(1, N + 1) * np.exp(0.1 * r.normal(size=(D, N))) * scale_a)
        self.Ds, self.nD = _dev(r.normal(size=D) if skip else None)
        step = np.exp(r.uniform(np.log(1e-3), np.log(0.1), size=D))
        self.bias, self.nbias = _dev(step + np.log(-np.expm1(-step)) if bias and softplus else None)
        self.h0, self.nh0 = _dev(r.normal(size=(S, D, N)) if h0 else None)
        self.dy, self.ndy = rows(D)
        self.dl, self.ndl = _dev(r.normal(size=(S, D, N)) if h0 else None)

    def inputs(self):
        return (self.x, self.raw, self.A, self.Bm, self.Cm, self.Ds, self.bias, self.h0)

    def oracle_inputs(self):
        return (self.nx, self.nraw, self.nA, self.nB, self.nC, self.nD, self.nbias, self.nh0)

    def forward(self, save=True, **kw):
        S = len(self.sp)
        y, last, saved = self.mg.selective_scan_fwd(
            *self.inputs(), softplus=self.softplus, cu_seqlens=self.cu_dev, save=save,
            out=(_nan((self.B, self.T, self.D), self.dtype), _nan((S, self.D, self.N))), **kw)
        return y, last, saved

    def check_forward(self):
        y, last, saved = self.forward()
        want_y, want_last, _ = o.scan_fwd(*self.oracle_inputs(), self.sp, self.softplus)
        sy, sl, _ = o.scan_fwd(*self.oracle_inputs(), self.sp, self.softplus, absolute=True)
        count = max((hi - lo for _, lo, hi in self.sp), default=0) + self.N
        _near("y", y, want_y, sy, count)
        _near("h_last", last, want_last, sl, count)
        y2, last2, none = self.forward(save=False)
        assert none is None and torch.equal(y2, y) and torch.equal(last2, last)
        return saved

    def backward(self, saved, **kw):
        S, shp = len(self.sp), (self.B, self.T, self.D)
        gn = (self.B, self.T, self.G, self.N)
        out = (_nan(shp, self.dtype), _nan(shp, self.dtype), _nan((self.D, self.N)), _nan(gn, self.dtype),
               _nan(gn, self.dtype), _nan((self.D,)), _nan((self.D,)), _nan((S, self.D, self.N)))
        return self.mg.selective_scan_bwd(self.dy, saved, *self.inputs(), self.dl, softplus=self.softplus,
                                          cu_seqlens=self.cu_dev, out=out, **kw)

    def check(self):
        saved = self.check_forward()
        got = self.backward(saved)
        more = (self.ndl, self.sp, self.softplus)
        want = o.scan_bwd(self.ndy, *self.oracle_inputs(), *more)
        scale = o.scan_bwd(self.ndy, *self.oracle_inputs(), *more, absolute=True)
        rows = max((hi - lo for _, lo, hi in self.sp), default=0)
        total = self.B * self.T
        names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dh0")
        counts = (rows, rows, rows + total, rows + self.D // self.G, rows + self.D // self.G, total,
                  rows + total, rows)
        present = (True, True, True, True, True, self.Ds is not None, self.bias is not None, self.h0 is not None)
        for n, g, w, s, c, p in zip(names, got, want, scale, counts, present):
            if p:
                _near(n, g, w, s, c + self.N)
            else:
                assert g is None
        again = self.backward(saved)
        for n, a, b in zip(names, got, again):
            assert a is None or torch.equal(a, b), n
        self.mg.workspace_status()


SHAPES = [
    dict(B=1, T=1, D=1, N=1),
    dict(B=2, T=1, D=8, N=16),
    dict(B=1, T=2, D=33, N=5),
    dict(B=3, T=17, D=40, N=4),
    dict(B=2, T=33, D=64, N=8),
    dict(B=1, T=130, D=160, N=16),
    dict(B=2, T=65, D=37, N=16),
    dict(B=1, T=64, D=130, N=24),
    dict(B=1, T=50, D=48, N=33),
    dict(B=1, T=40, D=24, N=64),
    dict(B=2, T=70, D=96, N=16, G=2),
    dict(B=1, T=45, D=60, N=12, G=5),
    dict(B=1, T=31, D=12, N=7, G=12),
    dict(B=1, T=600, D=16, N=16),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s.values())))
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_shapes(cuda_lib, shape, dtype):
    Scan(cuda_lib, **shape, dtype=dtype, seed=sum(shape.values())).check()


PACKS = [
    [0, 1],
    [0, 5, 5, 6, 23],
    [0, 0, 0, 40, 40],
    [0, 16, 32, 64, 80],
    [0, 31, 32, 33, 100, 164, 164, 300],
    list(range(0, 41)),
]


@pytest.mark.parametrize("cu", PACKS, ids=lambda c: f"{len(c) - 1}seq{c[-1]}")
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_packed(cuda_lib, cu, dtype):
    Scan(cuda_lib, 1, cu[-1], 72, 16, cu=cu, dtype=dtype, seed=len(cu)).check()
    Scan(cuda_lib, 1, cu[-1], 20, 6, G=2, cu=cu, dtype=dtype, seed=len(cu), h0=False, wide=False).check()


@pytest.mark.parametrize("T", [255, 256, 257, 1023, 2050])
def test_scan_long(cuda_lib, T):
    """Lengths around the multiples at which time may be cut, few channels."""
    Scan(cuda_lib, 1, T, 24, 16, seed=T).check()


@pytest.mark.parametrize("kw", [dict(skip=False), dict(bias=False), dict(h0=False), dict(softplus=False),
                                dict(skip=False, bias=False, h0=False, wide=False)],
                         ids=lambda k: ",".join(k))
def test_scan_optional_inputs(cuda_lib, kw):
    Scan(cuda_lib, 2, 75, 48, 16, seed=5, **kw).check()


def test_scan_one_group_without_its_dimension(cuda_lib):
    c = Scan(cuda_lib, 2, 20, 16, 8, seed=6)
    y, last, saved = c.forward()
    args = (c.x, c.raw, c.A, c.Bm[:, :, 0], c.Cm[:, :, 0], c.Ds, c.bias, c.h0)
    y2, last2, saved2 = cuda_lib.selective_scan_fwd(*args, save=True)
    assert torch.equal(y, y2) and torch.equal(last, last2)
    got = cuda_lib.selective_scan_bwd(c.dy, saved2, *args, c.dl)
    want = c.backward(saved)
    assert got[3].shape == (2, 20, 8) and torch.equal(got[3], want[3][:, :, 0])


def test_scan_strong_decay_and_extreme_steps(cuda_lib):
    """Decays from e^-1000 to 1, raw steps to +-60 (softplus saturates on both
    sides): nothing overflows."""
    c = Scan(cuda_lib, 1, 60, 32, 16, seed=7)
    c.raw = torch.linspace(-60, 60, 60 * 32, device=DEV).reshape(1, 60, 32)[:, torch.randperm(60)]
    c.nraw = _np(c.raw)
    c.check()


def test_scan_steps_are_the_scan(cuda_lib):
    """Tokens one at a time, from and into a pool of states, against the prompt."""
    mg = cuda_lib
    c = Scan(mg, 3, 9, 40, 16, dtype=BF16, seed=8)
    _, want, _ = c.forward()
    pool = torch.randn(7, 40, 16, device=DEV)
    keep = pool.clone()
    slots = torch.tensor([5, 0, 3], device=DEV)
    pool[slots] = c.h0
    wy, _, _ = o.scan_fwd(*c.oracle_inputs(), c.sp)
    sy, sl, _ = o.scan_fwd(*c.oracle_inputs(), c.sp, absolute=True)
    for t in range(9):
        y = mg.selective_scan_step(c.x[:, t], c.raw[:, t], c.A, c.Bm[:, t], c.Cm[:, t], pool, c.Ds, c.bias,
                                   slots=slots, out=_nan((3, 40), BF16))
        _near("y", y, wy[:, t], sy[:, t], 9 + 16)
    _near("state", pool[slots], _np(want), sl, 9 + 16)
    rest = [1, 2, 4, 6]
    assert torch.equal(pool[rest], keep[rest])


@pytest.mark.parametrize("N,G,D", [(1, 1, 5), (4, 2, 8), (16, 1, 33), (16, 4, 64), (24, 1, 40), (64, 2, 12)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_step_shapes(cuda_lib, N, G, D, dtype):
    c = Scan(cuda_lib, 5, 1, D, N, G=G, dtype=dtype, seed=N + D)
    ny, ns = o.scan_step(c.nx[:, 0], c.nraw[:, 0], c.nA, c.nB[:, 0], c.nC[:, 0], c.nD, c.nbias, c.nh0, None)
    sy, ss = o.scan_step(c.nx[:, 0], c.nraw[:, 0], c.nA, c.nB[:, 0], c.nC[:, 0], c.nD, c.nbias, c.nh0, None,
                         absolute=True)
    y = cuda_lib.selective_scan_step(c.x[:, 0], c.raw[:, 0], c.A, c.Bm[:, 0], c.Cm[:, 0], c.h0, c.Ds, c.bias,
                                     out=_nan((5, D), dtype))
    _near("y", y, ny, sy, N)
    _near("state", c.h0, ns, ss, 1)


def test_idle_rows_touch_nothing(cuda_lib):
    """Rows whose slot is outside the pool: output 0, every state as it was,
    even where the row's inputs are NaN."""
    mg = cuda_lib
    c = Scan(mg, 6, 1, 24, 16, seed=9, wide=False)
    pool = torch.randn(4, 24, 16, device=DEV)
    before = pool.clone()
    slots = torch.tensor([-1, 2, 4, 1 << 40, 0, -(1 << 40)], device=DEV)
    x = c.x[:, 0].clone()
    x[[0, 2, 3, 5]] = float("nan")
    y = mg.selective_scan_step(x, c.raw[:, 0], c.A, c.Bm[:, 0], c.Cm[:, 0], pool, c.Ds, c.bias, slots=slots)
    assert (y[[0, 2, 3, 5]] == 0).all() and torch.isfinite(y).all() and (y[[1, 4]] != 0).any()
    assert torch.equal(pool[[1, 3]], before[[1, 3]]) and not torch.equal(pool[[0, 2]], before[[0, 2]])
    w = torch.randn(24, 4, device=DEV)
    cpool = torch.randn(4, 3, 24, device=DEV)
    cbefore = cpool.clone()
    y = mg.causal_conv_step(x, w, cpool, slots=slots)
    assert (y[[0, 2, 3, 5]] == 0).all() and torch.isfinite(y).all() and (y[[1, 4]] != 0).any()
    assert torch.equal(cpool[[1, 3]], cbefore[[1, 3]]) and torch.equal(cpool[2, 2], x[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_sequence_keeps_its_nans(cuda_lib, bad):
    """NaN or infinite inputs and states of one packed sequence reach no other,
    forward or backward."""
    cu = [0, 20, 50, 50, 90]
    ref = Scan(cuda_lib, 1, 90, 40, 16, cu=cu, seed=10)
    hit = Scan(cuda_lib, 1, 90, 40, 16, cu=cu, seed=10)
    for t in (hit.x, hit.raw, hit.dy):
        t[:, 20:50] = bad
    hit.h0[1], hit.dl[1] = bad, bad
    (y0, l0, s0), (y1, l1, s1) = ref.forward(), hit.forward()
    rows = [i for i in range(90) if not 20 <= i < 50]
    assert torch.equal(y0[:, rows], y1[:, rows]) and torch.equal(l0[[0, 2, 3]], l1[[0, 2, 3]])
    g0, g1 = ref.backward(s0), hit.backward(s1)
    for i in (0, 1, 3, 4):
        assert torch.equal(g0[i][:, rows], g1[i][:, rows]), i
    assert torch.equal(g0[7][[0, 2, 3]], g1[7][[0, 2, 3]])
    conv = [cuda_lib.causal_conv_fwd(c.x, torch.ones(40, 4, device=DEV), cu_seqlens=c.cu_dev) for c in (ref, hit)]
    assert torch.equal(conv[0][0][:, rows], conv[1][0][:, rows])


def test_scan_large_offsets(cuda_lib):
    """A batch entry whose values lie past 2^31: the same as that entry alone."""
    B, T, D, N = 3, 131072, 8192, 4
    mg = cuda_lib
    x = torch.empty(B, T, D, dtype=BF16, device=DEV).normal_()
    raw = torch.full((B, T, 1), -2.0, dtype=BF16, device=DEV).expand(B, T, D)
    A = -torch.ones(D, N, device=DEV)
    bc = torch.randn(B, T, 2 * N, dtype=BF16, device=DEV)
    Bm, Cm = bc[..., :N], bc[..., N:]
    y, last, _ = mg.selective_scan_fwd(x, raw, A, Bm, Cm)
    tail = slice(T - 1024, T)   # decays of e^-0.127 a row: earlier rows are gone
    y1, last1, _ = mg.selective_scan_fwd(x[2:, tail].contiguous(), raw[2:, tail].contiguous(), A,
                                         Bm[2:, tail].contiguous(), Cm[2:, tail].contiguous())
    torch.testing.assert_close(y[2, -512:], y1[0, -512:], rtol=2 ** -7, atol=1e-3)
    torch.testing.assert_close(last[2], last1[0], rtol=1e-4, atol=1e-4)
    w = torch.randn(D, 4, device=DEV)
    y, x_last = mg.causal_conv_fwd(x, w)
    y1, _ = mg.causal_conv_fwd(x[2:, tail].contiguous(), w)
    assert torch.equal(y[2, -1000:], y1[0, -1000:]) and torch.equal(x_last[2], x[2, -3:])
    n, _ = mg.group_norm_fwd(x, torch.ones(D, device=DEV), groups=64)
    n1, _ = mg.group_norm_fwd(x[2:, tail].contiguous(), torch.ones(D, device=DEV), groups=64)
    assert torch.equal(n[2, tail], n1[0])


# -------------------------------------------------------------- convolution

def _conv(mg, B, T, D, W, dtype, cu=None, seed=0, bias=True, x0=True, act="silu", wide=True):
    r = _rng(seed)
    sp = o.spans(B, T, cu)
    cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)
    pad = 16 if wide else 0
    xw = torch.from_numpy(r.normal(size=(B, T, D + pad))).to(dtype).to(DEV)
    x = xw[..., :D]
    nx = _np(x)
    w, nw = _dev(r.normal(size=(D, W)))
    b, nb = _dev(r.normal(size=D) if bias else None)
    e = (len(sp), W - 1, D)
    e0, ne0 = _dev(r.normal(size=e) if x0 else None, dtype)
    dy, ndy = _dev(r.normal(size=(B, T, D)), dtype)
    dl, ndl = _dev(r.normal(size=e) if x0 else None, dtype)
    y, last = mg.causal_conv_fwd(x, w, b, e0, act=act, cu_seqlens=cu_dev, out=(_nan(x.shape, dtype), _nan(e, dtype)))
    kw = dict(silu=act is not None)
    wy, wl = o.conv_fwd(nx, nw, nb, ne0, sp, **kw)
    sy, _ = o.conv_fwd(nx, nw, nb, ne0, sp, **kw, absolute=True)
    _near("y", y, wy, sy, W)
    assert np.array_equal(_np(last), wl)
    out = (_nan(x.shape, dtype), _nan(w.shape), _nan((D,)), _nan(e, dtype))
    got = mg.causal_conv_bwd(dy, x, w, b, e0, dl, act=act, cu_seqlens=cu_dev, out=out)
    want = o.conv_bwd(ndy, nx, nw, nb, ne0, ndl, sp, **kw)
    # silu' is at most 1.1 and its slope at most 1/2: a rounding of v moves dv by less than |dy| S_v
    scale = o.conv_bwd(ndy * (1 + sy), nx, nw, nb, ne0, ndl, sp, **kw, absolute=True)
    for n, g, v, s, c, p in zip(("dx", "dw", "dbias", "dx0"), got, want, scale, (W, B * T, B * T, W),
                                (True, True, bias, x0)):
        if p:
            _near(n, g, v, s, c)
        else:
            assert g is None
    again = mg.causal_conv_bwd(dy, x, w, b, e0, dl, act=act, cu_seqlens=cu_dev)
    assert all(a is None or torch.equal(a, g) for a, g in zip(again, got))
    mg.workspace_status()


@pytest.mark.parametrize("W", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_widths(cuda_lib, W, dtype):
    _conv(cuda_lib, 2, 37, 40, W, dtype, seed=W)


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 8), (3, 2, 33), (2, 3, 516), (1, 200, 128), (2, 129, 37), (4, 66, 1032)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_shapes(cuda_lib, shape, dtype):
    _conv(cuda_lib, *shape, 4, dtype, seed=sum(shape), wide=shape[2] % 2 == 0)


@pytest.mark.parametrize("cu", PACKS + [[0, 2, 3, 5, 5, 6, 7, 60]], ids=lambda c: f"{len(c) - 1}seq{c[-1]}")
@pytest.mark.parametrize("W", [2, 4])
def test_conv_packed(cuda_lib, cu, W):
    _conv(cuda_lib, 1, cu[-1], 72, W, F32, cu=cu, seed=len(cu))
    _conv(cuda_lib, 1, cu[-1], 21, W, BF16, cu=cu, seed=len(cu), x0=False)


@pytest.mark.parametrize("kw", [dict(bias=False), dict(x0=False), dict(act=None)], ids=lambda k: ",".join(k))
def test_conv_optional_inputs(cuda_lib, kw):
    _conv(cuda_lib, 2, 50, 64, 4, F32, seed=3, **kw)


@pytest.mark.parametrize("W", [1, 2, 4])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_steps_are_the_convolution(cuda_lib, W, dtype):
    mg = cuda_lib
    x = torch.randn(3, 7, 44, device=DEV).to(dtype)
    w, b = torch.randn(44, W, device=DEV), torch.randn(44, device=DEV)
    y, last = mg.causal_conv_fwd(x, w, b)
    pool = torch.zeros(5, W - 1, 44, device=DEV, dtype=dtype)
    slots = torch.tensor([4, 0, 2], device=DEV)
    for t in range(7):
        assert torch.equal(mg.causal_conv_step(x[:, t], w, pool, b, slots=slots), y[:, t])
    assert torch.equal(pool[slots], last)


# --------------------------------------------------------------- group norm

def _norm(mg, M, D, G, dtype, gate="after", rms=False, bias=True, act="silu", seed=0, shift=0.0, wide=True):
    r = _rng(seed)
    pad = 16 if wide else 0
    x = torch.from_numpy(r.normal(size=(M, D + pad)) + shift).to(dtype).to(DEV)[:, :D]
    z = torch.from_numpy(r.normal(size=(M, D + pad))).to(dtype).to(DEV)[:, pad:] if gate != "none" else None
    nx, nz = _np(x), None if z is None else _np(z)
    w, nw = _dev(1 + 0.1 * r.normal(size=D))
    b, nb = _dev(r.normal(size=D) if bias else None)
    dy, ndy = _dev(r.normal(size=(M, D)), dtype)
    first = gate == "first"
    kw = dict(groups=G, rms=rms, gate_first=first, act=act)
    okw = dict(G=G, eps=1e-5, rms=rms, gate_first=first, silu=act is not None)
    y, stats = mg.group_norm_fwd(x, w, b, z, **kw, out=(_nan((M, D), dtype), _nan((M, G, 2))))
    wy, mean, rstd = o.norm_fwd(nx, nw, nb, nz, **okw)
    sy = o.norm_fwd(nx, nw, nb, nz, **okw, absolute=True)[0]
    _near("y", y, wy, sy, D // G)
    _near("rstd", stats[..., 1], rstd, rstd, D // G)
    out = (_nan((M, D), dtype), _nan((D,)), _nan((D,)), _nan((M, D), dtype))
    got = mg.group_norm_bwd(dy, stats, x, w, b, z, **kw, out=out)
    want = o.norm_bwd(ndy, nx, nw, nb, nz, **okw)
    scale = o.norm_bwd(ndy, nx, nw, nb, nz, **okw, absolute=True)
    for n, g, v, s, c in zip(("dx", "dw", "dbias", "dz"), got, want, scale, (D // G, M + D // G, M, D // G)):
        if (n == "dbias" and not bias) or (n == "dz" and z is None):
            assert g is None
        else:
            _near(n, g, v, s, c)
    again = mg.group_norm_bwd(dy, stats, x, w, b, z, **kw)
    assert all(a is None or torch.equal(a, g) for a, g in zip(again, got))


@pytest.mark.parametrize("shape", [(1, 1, 1), (3, 8, 1), (5, 40, 8), (2, 33, 3), (7, 1000, 5), (4, 512, 4), (3, 4096, 1),
                                   (2, 4104, 1), (2, 16384, 1), (1, 9000, 1), (1, 8191, 1), (300, 64, 64),
                                   (2000, 96, 3)],
                         ids=str)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_shapes(cuda_lib, shape, dtype):
    _norm(cuda_lib, *shape, dtype, seed=sum(shape))


@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("act", ["silu", None])
def test_norm_forms(cuda_lib, gate, rms, act):
    for dtype in (F32, BF16):
        _norm(cuda_lib, 21, 192, 3, dtype, gate, rms, not rms, act, seed=4)


def test_norm_far_from_zero(cuda_lib):
    """Rows around 1000 with a spread of 1: the variance comes from the
    differences, not from E[x^2] - E[x]^2."""
    _norm(cuda_lib, 9, 256, 2, F32, seed=5, shift=1000.0)


def test_norm_leading_dimensions(cuda_lib):
    mg = cuda_lib
    x = torch.randn(2, 3, 5, 64, device=DEV)
    w = torch.randn(64, device=DEV)
    y, stats = mg.group_norm_fwd(x, w, groups=4)
    y2, _ = mg.group_norm_fwd(x.reshape(30, 64), w, groups=4)
    assert torch.equal(y.reshape(30, 64), y2) and stats.shape == (30, 4, 2)
    assert mg.group_norm_fwd(x[:0], w, groups=4)[0].shape == (0, 3, 5, 64)
    dx, dw, _, _ = mg.group_norm_bwd(x[:0], stats[:0], x[:0], w, groups=4)
    assert dx.numel() == 0 and (dw == 0).all()


# ----------------------------------------------------- streams, empty calls

def test_calls_without_rows(cuda_lib):
    mg = cuda_lib
    z = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    h0 = torch.randn(2, 8, 4, device=DEV)
    y, last, saved = mg.selective_scan_fwd(z(2, 0, 8), z(2, 0, 8), z(8, 4), z(2, 0, 4), z(2, 0, 4), h0=h0, save=True)
    assert y.shape == (2, 0, 8) and torch.equal(last, h0)
    got = mg.selective_scan_bwd(z(2, 0, 8), saved, z(2, 0, 8), z(2, 0, 8), z(8, 4), z(2, 0, 4), z(2, 0, 4), D=z(8), h0=h0, dh_last=2 * h0)
    assert (got[2] == 0).all() and (got[5] == 0).all() and torch.equal(got[7], 2 * h0)
    x0 = torch.randn(2, 3, 8, device=DEV)
    y, last = mg.causal_conv_fwd(z(2, 0, 8), z(8, 4), x0=x0)
    assert y.shape == (2, 0, 8) and torch.equal(last, x0)
    cu = torch.zeros(3, dtype=torch.int64, device=DEV)
    _, last, _ = mg.selective_scan_fwd(z(1, 0, 8), z(1, 0, 8), z(8, 4), z(1, 0, 4), z(1, 0, 4), h0=h0, cu_seqlens=cu)
    assert torch.equal(last, h0)
    assert mg.selective_scan_step(z(0, 8), z(0, 8), z(8, 4), z(0, 4), z(0, 4), z(3, 8, 4)).shape == (0, 8)


def test_on_another_stream(cuda_lib):
    """stream=: arguments that need a copy, outputs and kernels all on it."""
    mg = cuda_lib
    c = Scan(mg, 2, 300, 256, 16, seed=11, wide=False)
    want = c.forward()
    side = torch.cuda.Stream()
    xt = c.x.transpose(1, 2).contiguous().transpose(1, 2)   # not readable row by row
    torch.cuda.synchronize()
    for _ in range(3):
        y, last, saved = mg.selective_scan_fwd(xt, *c.inputs()[1:], save=True, stream=side)
        got = mg.selective_scan_bwd(c.dy, saved, xt, *c.inputs()[1:], c.dl, stream=side)
        cy, _ = mg.causal_conv_fwd(xt, c.A[:, :4].contiguous(), stream=side)
    side.synchronize()
    assert torch.equal(y, want[0]) and torch.equal(last, want[1])
    for a, b in zip(got, c.backward(want[2])):
        assert torch.equal(a, b)
    assert torch.equal(cy, mg.causal_conv_fwd(c.x, c.A[:, :4].contiguous())[0])


def test_workspace_is_shared_with_the_scans(cuda_lib):
    """The ops take turns on one workspace with the look-back scans."""
    mg = cuda_lib
    ws = mg.new_workspace(64 << 20, DEV)
    c = Scan(mg, 2, 200, 64, 16, seed=12)
    a, b = torch.rand(2, 500, 64, device=DEV), torch.randn(2, 500, 64, device=DEV)
    want_lin, want = mg.linear_scan_fwd(a, b), c.forward()
    want_b = c.backward(want[2])
    for _ in range(3):
        got = c.forward(ws=ws)
        lin = mg.linear_scan_fwd(a, b, ws=ws)
        gb = c.backward(got[2], ws=ws)
        lin2 = mg.linear_scan_fwd(a, b, ws=ws)
        assert torch.equal(got[0], want[0]) and all(torch.equal(p, q) for p, q in zip(gb, want_b))
        assert all(torch.equal(p, q) for p, q in zip(lin + lin2, want_lin + want_lin))
    mg.workspace_status(ws)


def test_graph_capture(cuda_lib):
    """The token calls in a CUDA graph, replayed on new inputs."""
    mg = cuda_lib
    c = Scan(mg, 4, 1, 64, 16, seed=13, wide=False)
    w = torch.randn(64, 4, device=DEV)
    x, pool, cpool = c.x[:, 0].clone(), c.h0.clone(), torch.randn(4, 3, 64, device=DEV)
    pool0, cpool0 = pool.clone(), cpool.clone()

    def token():
        v = mg.causal_conv_step(x, w, cpool)
        y = mg.selective_scan_step(v, c.raw[:, 0], c.A, c.Bm[:, 0], c.Cm[:, 0], pool, c.Ds, c.bias)
        return mg.group_norm_fwd(y, torch.ones(64, device=DEV))[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
    torch.cuda.current_stream().wait_stream(side)
    pool.copy_(pool0), cpool.copy_(cpool0)
    want = [token().clone() for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    ones = torch.ones(64, device=DEV)
    with torch.cuda.graph(graph):
        v = mg.causal_conv_step(x, w, cpool)
        y = mg.selective_scan_step(v, c.raw[:, 0], c.A, c.Bm[:, 0], c.Cm[:, 0], pool, c.Ds, c.bias)
        n, _ = mg.group_norm_fwd(y, ones)
    pool.copy_(pool0), cpool.copy_(cpool0)
    for i in range(3):
        graph.replay()
        assert torch.equal(n, want[i])


# ------------------------------------------------------------------ refusals

def test_bad_cu_seqlens_are_reported(cuda_lib):
    """Offsets that are not non-decreasing from 0 to T: no fault, and the next
    status query says so."""
    mg = cuda_lib
    for cu in ([0, 50, 20, 64], [3, 30, 64], [0, 30, 60], [0, 30, 90], [-5, 64], [0, 1 << 50, 64]):
        c = Scan(mg, 1, 64, 40, 16, cu=[0] + [64] * (len(cu) - 1), seed=14)
        c.cu_dev = torch.tensor(cu, dtype=torch.int64, device=DEV)
        w = torch.randn(40, 4, device=DEV)
        x0 = torch.zeros(len(cu) - 1, 3, 40, device=DEV)
        for call in (lambda: c.forward(), lambda: c.backward(torch.zeros(
                mg.load().mg_selective_scan_saved_size(1, 64, 40, 16) // 4, device=DEV)),
                lambda: mg.causal_conv_fwd(c.x, w, cu_seqlens=c.cu_dev),
                lambda: mg.causal_conv_bwd(c.dy, c.x, w, x0=x0, cu_seqlens=c.cu_dev)):
            call()
            with pytest.raises(mg.MgScanError) as e:
                mg.workspace_status()
            assert e.value.status == mg.MG_ERR_INVALID_ARG
    mg.workspace_status()


def test_refusals(cuda_lib):
    mg = cuda_lib
    x, z = torch.zeros(2, 6, 8, device=DEV), lambda *s: torch.zeros(*s, device=DEV)
    A, bc = z(8, 4), z(2, 6, 4)
    scan = lambda **k: mg.selective_scan_fwd(**{**dict(x=x, dt=x, A=A, B=bc, C=bc), **k})  # noqa: E731
    for bad in (dict(x=x.cpu()), dict(x=x.double()), dict(x=z(6, 8)), dict(dt=x.bfloat16()), dict(dt=z(2, 5, 8)),
                dict(A=z(8, 65)), dict(A=z(7, 4)), dict(A=A.bfloat16()), dict(B=z(2, 6, 5)), dict(B=z(2, 6, 3, 4)),
                dict(B=z(2, 6, 2, 4)), dict(D=z(7)), dict(dt_bias=z(8, 1)), dict(h0=z(1, 8, 4)),
                dict(cu_seqlens=torch.tensor([0, 6], device=DEV)), dict(out=(z(2, 6, 7), None))):
        with pytest.raises(ValueError):
            scan(**bad)
    y, last, saved = scan(save=True)
    with pytest.raises(ValueError):
        mg.selective_scan_bwd(y, None, x, x, A, bc, bc)
    with pytest.raises(ValueError):
        mg.selective_scan_bwd(y, saved[:-1], x, x, A, bc, bc)
    step = lambda **k: mg.selective_scan_step(**{**dict(x=x[:, 0], dt=x[:, 0], A=A, B=bc[:, 0], C=bc[:, 0], state=z(2, 8, 4)), **k})  # noqa: E731
    for bad in (dict(state=z(1, 8, 4)), dict(state=z(2, 4, 8)), dict(state=z(2, 4, 8).transpose(1, 2)),
                dict(state=z(2, 8, 4).bfloat16()), dict(slots=torch.zeros(2, dtype=torch.int32, device=DEV)),
                dict(slots=torch.zeros(3, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            step(**bad)
    w = z(8, 4)
    for f in (lambda: mg.causal_conv_fwd(x, z(8, 9)), lambda: mg.causal_conv_fwd(x, z(7, 4)),
              lambda: mg.causal_conv_fwd(x, w, act="tanh"), lambda: mg.causal_conv_fwd(x, w, x0=z(2, 4, 8)),
              lambda: mg.causal_conv_bwd(z(2, 5, 8), x, w), lambda: mg.causal_conv_bwd(x, x, w, dx_last=z(2, 3, 7)),
              lambda: mg.causal_conv_step(x[:, 0], w, z(2, 4, 8)), lambda: mg.group_norm_fwd(x, z(8), groups=3),
              lambda: mg.group_norm_fwd(x, z(7)), lambda: mg.group_norm_fwd(x, z(8), gate_first=True),
              lambda: mg.group_norm_fwd(x, z(8), z=z(2, 6, 7)), lambda: mg.group_norm_bwd(x, z(1, 1, 2), x, z(8))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(mg.MgScanError) as e:
        mg.group_norm_fwd(z(1, 16385), z(16385))
    assert e.value.status == mg.MG_ERR_UNSUPPORTED
    with pytest.raises(mg.MgScanError):
        mg.group_norm_fwd(x, z(8), eps=-1.0)


# ------------------------------------------- rows that 16-byte vectors do not fit

def _framed(t, before, after):
    """The tensor inside wider rows whose other values are NaN (`before` keeps
    the data's 16-byte alignment)."""
    wide = torch.full((*t.shape[:-1], before + t.shape[-1] + after), float("nan"), dtype=t.dtype, device=DEV)
    inner = wide[..., before:before + t.shape[-1]]
    inner.copy_(t)
    return inner


@pytest.mark.parametrize("D,N,G", [(33, 16, 1), (129, 12, 1), (66, 6, 2), (45, 24, 3), (21, 33, 1), (70, 3, 1), (257, 8, 1)])
@pytest.mark.parametrize("after", [1, 2, 7])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_rows_of_any_alignment(cuda_lib, D, N, G, after, dtype):
    """Odd widths and row strides: the values between the rows, NaN here, reach
    no result."""
    c = Scan(cuda_lib, 2, 41, D, N, G=G, dtype=dtype, seed=D + after)
    c.x, c.raw, c.dy = _framed(c.x, 8, after), _framed(c.raw, 0, after + 1), _framed(c.dy, 16, 2 * after)
    c.check()


@pytest.mark.parametrize("shape", [(9, 1001, 1), (5, 4097, 1), (300, 126, 2), (70, 250, 1), (33, 515, 5), (3, 2050, 1),
                                   (40, 1024, 1), (40, 2048, 1), (90, 512, 1), (6, 1536, 1), (700, 128, 2)], ids=str)
@pytest.mark.parametrize("gate", ["none", "after", "first"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_group_widths(cuda_lib, shape, gate, dtype):
    """Groups of every way to hold them: pairs of any alignment, one or two
    vectors a thread, a part of a warp, a warp, a block."""
    _norm(cuda_lib, *shape, dtype, gate, rms=gate == "first", seed=sum(shape), wide=shape[1] % 8 == 0)


@pytest.mark.parametrize("D,G", [(1001, 7), (250, 1), (40, 8), (77, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norm_rows_among_nans(cuda_lib, D, G, dtype):
    mg = cuda_lib
    x, z, dy = (torch.randn(21, D, device=DEV).to(dtype) for _ in range(3))
    w = torch.randn(D, device=DEV)
    fx, fz, fdy = _framed(x, 8, 3), _framed(z, 16, 1), _framed(dy, 0, 5)
    y, st = mg.group_norm_fwd(x, w, w, z, groups=G)
    fy, fst = mg.group_norm_fwd(fx, w, w, fz, groups=G)
    assert torch.equal(y, fy) and torch.equal(st, fst)
    for a, b in zip(mg.group_norm_bwd(dy, st, x, w, w, z, groups=G), mg.group_norm_bwd(fdy, st, fx, w, w, fz, groups=G)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("B,D,W", [(1, 1, 4), (5, 44, 4), (9, 1025, 3), (13, 514, 8), (4, 8, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_step_batches(cuda_lib, B, D, W, dtype):
    """Batches that end inside a thread's rows, with idle rows among them."""
    mg = cuda_lib
    r = _rng(B + D)
    x, nx = _dev(r.normal(size=(B, D)), dtype)
    w, nw = _dev(r.normal(size=(D, W)))
    b, nb = _dev(r.normal(size=D))
    pool, npool = _dev(r.normal(size=(2 * B, W - 1, D)), dtype)
    slots = r.permutation(2 * B)[:B]
    slots[B // 2] = -1 if B > 1 else slots[0]
    y = mg.causal_conv_step(x, w, pool, b, slots=torch.from_numpy(slots).to(DEV), out=_nan((B, D), dtype))
    want, state = o.conv_step(nx, nw, nb, npool, slots)
    scale = np.abs(nx * nw[:, -1]) + np.abs(nb)
    for j in range(W - 1):
        scale = scale + np.abs(nw[:, j]) * np.abs(npool[np.maximum(slots, 0), j])
    _near("y", y, want, scale, W)
    assert np.array_equal(_np(pool), state)


@pytest.mark.parametrize("cu", [None, [0, 5, 5, 300, 700]])
def test_graph_capture_of_a_training_step(cuda_lib, cu):
    """Forward and gradients in a CUDA graph (several dependent kernels a call),
    replayed on new inputs, equal the calls' own results."""
    mg = cuda_lib
    B, T, D, N = (1, 700, 200, 16) if cu else (3, 333, 200, 16)
    x, dy = (torch.randn(B, T, D, device=DEV).bfloat16() for _ in range(2))
    bc = torch.randn(B, T, 2 * N, device=DEV).bfloat16()
    A, b, w = -torch.rand(D, N, device=DEV) - 0.1, torch.full((D,), -3.0, device=DEV), torch.randn(D, 4, device=DEV)
    seqs = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)

    def step():
        args = (x, x, A, bc[..., :N], bc[..., N:], b, b)
        y, last, saved = mg.selective_scan_fwd(*args, save=True, cu_seqlens=seqs)
        n, stats = mg.group_norm_fwd(y, b, b, x, groups=2)
        return (y, last, n, *mg.selective_scan_bwd(dy, saved, *args, cu_seqlens=seqs),
                *mg.group_norm_bwd(dy, stats, y, b, b, x, groups=2), *mg.causal_conv_bwd(dy, x, w, b, cu_seqlens=seqs))

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()   # the stream's workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = step()
    for _ in range(5):
        x.normal_()
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(a is None or torch.equal(a, v) for a, v in zip(got, want))
    mg.workspace_status()
