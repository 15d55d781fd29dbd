"""GPU parity of the gated block's operators against the float64 oracle in
oracle/block.py, through the public entry points.

Tolerances, from the arithmetic.  Every output is a sum of products whose
magnitudes add up to S, which the oracle gives (absolute=True).
* float32 sums: a term passes at most (rows + summed values + 64) operations of
  2^-24, with exponentials within a few units; (rows + values + 64) 2^-22 S
  covers it.
* bf16 calls round, besides the output (2^-8 of its value), the weights of a
  chunk's products and the state as an operand of the rows' products, each to
  2^-8 of the term: 2^-8 S for o, dq, dk and dv, of which each term has one of
  the two.  States, their gradients and dg have no such rounding: where a state
  or weight meets them it is carried in three bf16 pieces, 2^-24 in all.
Outputs start as NaN, so that an unwritten element fails.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import block as o
from oracle.ssm import spans

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
TYPES = [F32, BF16]
IDS = ["fp32", "bf16"]


def _np(x):
    return x.detach().double().cpu().numpy()


def _nan(shape, dtype=F32):
    return torch.full(tuple(shape), float("nan"), dtype=dtype, device=DEV)


def _near(name, got, want, scale, count, rounded=False):
    """rounded: a bf16 output of products whose operands were rounded."""
    g = _np(got)
    assert g.shape == want.shape, (name, g.shape, want.shape)
    tol = (count + 64) * 2.0 ** -22 * scale + 1e-30
    if got.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(want) + (2.0 ** -8 * scale * (1 + 2.0 ** -8) if rounded else 0.0)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (name, int(bad.sum()), np.argwhere(bad)[:4].tolist(), float(np.max(np.abs(g - want)[bad] / tol[bad])))


class Scan:
    """One case's inputs on the device (q, k and v slices of wider rows) and in
    float64."""

    def __init__(self, mg, B, T, H, G, N, P, dtype=F32, cu=None, seed=0, state=True, pad=8, gates="mixed", dl=True):
        r = np.random.default_rng(seed)
        self.mg, self.dtype, self.cu, self.scale = mg, dtype, cu, float(np.float32(N ** -0.5))
        self.sp = spans(B, T, cu)
        S = len(self.sp)
        self.sizes = (B, T, H, G, N, P)
        self.cu_dev = None if cu is None else torch.tensor(cu, dtype=torch.int64, device=DEV)

        def rows(heads, width):
            t = torch.from_numpy(r.normal(size=(B, T, heads * width + pad))).to(dtype).to(DEV)
            t = t[..., :heads * width].unflatten(-1, (heads, width))
            return t, _np(t)

        def dev(a):
            if a is None:
                return None, None
            t = torch.from_numpy(np.ascontiguousarray(a)).float().to(DEV)
            return t, _np(t)

        self.q, self.nq = rows(G, N)
        self.k, self.nk = rows(G, N)
        self.v, self.nv = rows(H, P)
        self.do, self.ndo = rows(H, P)
        g = -np.exp(r.uniform(np.log(1e-3), 0, size=H)) * np.log1p(np.exp(r.normal(size=(B, T, H))))
        if gates == "mixed":
            g = np.where(r.random(g.shape) < 0.03, g - 40.0, g)
        elif gates == "none":
            g = np.zeros_like(g)
        self.g, self.ng = dev(g)
        self.S0, self.nS0 = dev(r.normal(size=(S, H, N, P)) if state else None)
        self.dl, self.ndl = dev(r.normal(size=(S, H, N, P)) if dl else None)
        self.count = max((hi - lo for _, lo, hi in self.sp), default=0) + N + P

    def forward(self, save=True, **kw):
        B, T, H, G, N, P = self.sizes
        return self.mg.gated_scan_fwd(self.q, self.k, self.v, self.g, self.S0, scale=self.scale, cu_seqlens=self.cu_dev,
                                      save=save, out=(_nan((B, T, H, P), self.dtype), _nan((len(self.sp), H, N, P))), **kw)

    def backward(self, saved, **kw):
        B, T, H, G, N, P = self.sizes
        out = (_nan((B, T, G, N), self.dtype), _nan((B, T, G, N), self.dtype), _nan((B, T, H, P), self.dtype), _nan((B, T, H)),
               _nan((len(self.sp), H, N, P)))
        return self.mg.gated_scan_bwd(self.do, saved, self.q, self.k, self.v, self.g, self.S0, self.dl, scale=self.scale,
                                      cu_seqlens=self.cu_dev, out=out, **kw)

    def args(self):
        return self.nq, self.nk, self.nv, self.ng, self.scale, self.nS0

    def check(self, backward=True):
        oo, last, saved = self.forward()
        want, wl, _ = o.scan_fwd(*self.args(), self.sp)
        S, Sl, _ = o.scan_fwd(*self.args(), self.sp, absolute=True)
        _near("o", oo, want, S, self.count, True)
        _near("S_last", last, wl, Sl, self.count)
        o2, last2, none = self.forward(save=False)
        assert none is None and torch.equal(o2, oo) and torch.equal(last2, last)
        if not backward:
            return
        got = self.backward(saved)
        want = o.scan_bwd(self.ndo, *self.args(), self.ndl, self.sp)
        S = o.scan_bwd(self.ndo, *self.args(), self.ndl, self.sp, absolute=True)
        for name, a, b, s in zip(("dq", "dk", "dv", "dg", "dS0"), got, want, S):
            if a is not None:
                _near(name, a, b, s, self.count + 128, name in ("dq", "dk", "dv"))
        again = self.backward(saved)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


SIZES = [  # B, T, H, G, N, P
    (1, 1, 1, 1, 1, 1), (2, 2, 2, 1, 3, 5), (1, 63, 2, 2, 16, 16), (1, 64, 1, 1, 32, 64), (2, 65, 4, 2, 24, 40),
    (1, 127, 2, 1, 64, 64), (1, 128, 3, 3, 128, 128), (1, 129, 2, 2, 127, 97), (1, 257, 6, 2, 80, 48), (3, 200, 4, 1, 17, 128),
    (1, 300, 8, 1, 128, 64), (1, 400, 2, 2, 64, 33),
]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_scan(cuda_lib, sizes, dtype):
    Scan(cuda_lib, *sizes, dtype=dtype, seed=sum(sizes)).check()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("cu", [[0, 1], [0, 0, 5, 5, 6, 134, 134, 263, 300], [0, 64, 128, 256, 257], [0, 0, 0, 40, 40]],
                         ids=["one", "ragged", "whole", "empty"])
def test_packed(cuda_lib, cu, dtype):
    Scan(cuda_lib, 1, cu[-1], 4, 2, 32, 48, dtype=dtype, cu=cu, seed=cu[-1]).check()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("gates", ["none", "mixed"])
def test_without_states(cuda_lib, dtype, gates):
    Scan(cuda_lib, 2, 150, 2, 1, 48, 64, dtype=dtype, state=False, dl=False, gates=gates, seed=3).check()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_of_any_stride(cuda_lib, dtype):
    """Row strides that leave rows off every alignment, and tensors that are
    no rows at all (these are copied)."""
    Scan(cuda_lib, 1, 140, 3, 3, 33, 31, dtype=dtype, pad=1, seed=4).check()
    c = Scan(cuda_lib, 2, 40, 4, 2, 16, 32, dtype=dtype, seed=5)
    want = c.forward(save=False)[:2]
    for n in "qkv":
        x = getattr(c, n)
        setattr(c, n, x.transpose(1, 2).contiguous().transpose(1, 2))
    c.g = c.g.transpose(0, 2).contiguous().transpose(0, 2)
    got = c.forward(save=False)[:2]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gates_that_forget_everything(cuda_lib, dtype):
    """-inf and gates far below float32's exponents: what is before such a row
    has no part in what follows, and the sums behind it keep their precision."""
    c = Scan(cuda_lib, 1, 200, 2, 1, 32, 32, dtype=dtype, gates="mild", seed=6)
    for t, value in ((0, -np.inf), (70, -1e30), (71, -np.inf), (130, -500.0), (199, -128.0)):
        c.g[0, t, 0] = value
    c.ng = np.maximum(_np(c.g), -128.0)
    c.check()
    oo, last, _ = c.forward()
    c.v[0, :71], c.S0[:] = 1e30, 1e30
    o2, last2, _ = c.forward()
    assert torch.equal(o2[0, 71:, 0], oo[0, 71:, 0]) and torch.equal(last2[0, 0], last[0, 0])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_nothing_passes_from_one_sequence_to_another(cuda_lib, dtype):
    cu = [0, 50, 51, 51, 180, 200]
    c = Scan(cuda_lib, 1, 200, 2, 1, 32, 32, dtype=dtype, cu=cu, seed=7)
    oo, last, saved = c.forward()
    grads = c.backward(saved)
    for x in (c.q, c.k, c.v, c.do):
        x[0, 51:180] = float("nan")
    c.g[0, 51:180], c.S0[3], c.dl[3] = float("nan"), float("nan"), float("inf")
    o2, last2, saved2 = c.forward()
    grads2 = c.backward(saved2)
    rows, seqs = [t for t in range(200) if not 51 <= t < 180], [0, 1, 2, 4]
    assert torch.equal(o2[:, rows], oo[:, rows]) and torch.equal(last2[seqs], last[seqs])
    assert all(torch.equal(a[:, rows], b[:, rows]) for a, b in zip(grads[:4], grads2[:4]))
    assert torch.equal(grads[4][seqs], grads2[4][seqs])
    assert torch.isnan(o2[0, 51:180]).all()


def test_long_sequence_of_small_gates(cuda_lib):
    """Thousands of rows whose decays are near 1, over many chunks."""
    Scan(cuda_lib, 1, 3000, 1, 1, 16, 16, dtype=BF16, gates="none", seed=8).check()
    Scan(cuda_lib, 1, 3000, 1, 1, 16, 16, dtype=F32, gates="mild", seed=9).check()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_bad_cu_seqlens_is_reported(cuda_lib, dtype):
    mg = cuda_lib
    for cu in ([0, 50, 20, 100], [0, 300, 100], [5, 60, 100], [0, -7, 100], [0, 1 << 40, 100]):
        c = Scan(mg, 1, 100, 2, 1, 16, 16, dtype=dtype, cu=[0] + [1] * (len(cu) - 2) + [100], seed=10)
        ws = mg.new_workspace(1 << 24, DEV)
        _, _, saved = c.forward(ws=ws)
        c.cu_dev = torch.tensor(cu, dtype=torch.int64, device=DEV)
        c.forward(ws=ws)
        with pytest.raises(mg.MgScanError, match="cu_seqlens"):
            mg.workspace_status(ws)
        c.backward(saved, ws=ws)
        with pytest.raises(mg.MgScanError, match="cu_seqlens"):
            mg.workspace_status(ws)
        mg.workspace_status(ws)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_empty_calls(cuda_lib, dtype):
    mg = cuda_lib
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t, device=DEV)  # noqa: E731
    S0, dl = torch.randn(2, 2, 4, 8, device=DEV), torch.randn(2, 2, 4, 8, device=DEV)
    q, v, g = z(2, 0, 1, 4), z(2, 0, 2, 8), z(2, 0, 2, t=F32)
    oo, last, saved = mg.gated_scan_fwd(q, q, v, g, S0, save=True)
    assert oo.shape == v.shape and torch.equal(last, S0) and saved.numel() == 0
    dq, dk, dv, dg, dS0 = mg.gated_scan_bwd(v, saved, q, q, v, g, S0, dl)
    assert dq.shape == q.shape and dv.shape == v.shape and torch.equal(dS0, dl)
    assert not mg.gated_scan_fwd(q, q, v, g)[1].any()
    cu = torch.zeros(3, dtype=torch.int64, device=DEV)
    assert torch.equal(mg.gated_scan_fwd(q[:1], q[:1], v[:1], g[:1], S0, cu_seqlens=cu)[1], S0)
    assert mg.gated_scan_step(z(0, 1, 4), z(0, 1, 4), z(0, 2, 8), z(0, 2, t=F32), S0).shape == (0, 2, 8)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("B,H,G,N,P", [(1, 1, 1, 1, 1), (5, 4, 2, 24, 40), (3, 2, 2, 128, 128), (4, 6, 1, 127, 33), (2, 8, 1, 128, 64), (2, 2, 1, 7, 127)])
def test_step(cuda_lib, B, H, G, N, P, dtype):
    mg = cuda_lib
    r = np.random.default_rng(B * H + N)
    new = lambda *s, t=dtype: torch.from_numpy(r.normal(size=s)).to(t).to(DEV)  # noqa: E731
    qk = new(B, 2 * G * N + 5)
    q, k = (qk[:, i * G * N:(i + 1) * G * N].unflatten(-1, (G, N)) for i in (0, 1))
    v, g, state = new(B, H, P), -new(B, H, t=F32).abs(), new(B + 2, H, N, P, t=F32)
    for slots in (None, torch.randperm(B + 2, device=DEV)[:B]):
        if slots is not None and B > 1:
            slots[0], slots[-1] = -1, 1 << 40
        before = state.clone()
        out = mg.gated_scan_step(q, k, v, g, state, slots=slots, scale=0.5, out=_nan((B, H, P), dtype))
        args = (_np(q), _np(k), _np(v), _np(g), 0.5, _np(before), None if slots is None else _np(slots))
        want, ws = o.scan_step(*args)
        S, Ss = o.scan_step(*args, absolute=True)
        _near("o", out, want, S, N)
        live = range(B) if slots is None else [int(s) for s in slots if 0 <= s < B + 2]
        _near("state", state, ws, Ss, 2)
        rest = [i for i in range(B + 2) if i not in live]
        assert torch.equal(state[rest], before[rest])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_tokens_are_the_prompt(cuda_lib, dtype):
    """One token at a time gives the prompt's rows and its last state."""
    c = Scan(cuda_lib, 2, 70, 4, 2, 24, 32, dtype=dtype, seed=11)
    oo, last, _ = c.forward(save=False)
    state = c.S0.clone()
    rows = [cuda_lib.gated_scan_step(c.q[:, t], c.k[:, t], c.v[:, t], c.g[:, t], state, scale=c.scale) for t in range(70)]
    want, _, _ = o.scan_fwd(*c.args(), c.sp)
    S, Sl, _ = o.scan_fwd(*c.args(), c.sp, absolute=True)
    _near("tokens", torch.stack(rows, 1), want, S, c.count)
    _near("state", state, _np(last), 2 * Sl, c.count)


# ---------------------------------------------------------------- rms norm

WIDTHS = [1, 2, 7, 8, 31, 64, 250, 256, 257, 512, 1000, 1001, 1002, 1024, 1032, 2048, 2049, 4096, 5000, 8191, 16384, 16383]


def _norm_case(M, D, dtype, pad, seed, residual=True):
    r = np.random.default_rng(seed)
    def rows(scale=1.0):
        return torch.from_numpy(r.normal(size=(M, D + pad)) * scale).to(dtype).to(DEV)[:, :D]
    x, res, dy, dr = rows(), rows(3.0) if residual else None, rows(), rows() if residual else None
    w = torch.from_numpy(1 + 0.1 * r.normal(size=D)).float().to(DEV)
    return x, res, w, dy, dr


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("pad", [0, 3, 8])
@pytest.mark.parametrize("D", WIDTHS)
def test_norm(cuda_lib, D, pad, dtype):
    mg = cuda_lib
    M = 5 if D > 1000 else 37
    residual = D % 3 != 0
    x, res, w, dy, dr = _norm_case(M, D, dtype, pad, D, residual)
    y, r, rstd = mg.rms_norm_fwd(x, w, res, out=(_nan((M, D), dtype), _nan((M, D), dtype), _nan((M,))))
    want_r = x if res is None else x + res          # torch rounds the float32 sum once
    assert torch.equal(r, want_r)
    want, want_rstd = o.norm_fwd(_np(r), _np(w), 1e-5)
    _near("y", y, want, np.abs(want), 8)
    _near("rstd", rstd, want_rstd, want_rstd, D)
    dx, dw = mg.rms_norm_bwd(dy, rstd, r, w, dr, out=(_nan((M, D), dtype), _nan((D,))))
    args = (_np(dy), _np(r), _np(w), 1e-5, None if dr is None else _np(dr))
    for name, a, b, s in zip(("dx", "dw"), (dx, dw), o.norm_bwd(*args), o.norm_bwd(*args, absolute=True)):
        _near(name, a, b, s, D if name == "dx" else M)


def test_norm_of_many_rows(cuda_lib):
    """More rows than the gradients' blocks: every block walks over several."""
    for D, dtype in ((40, BF16), (24, F32), (1001, F32), (2048, BF16)):
        M = 6007 if D < 100 else 2500
        x, res, w, dy, dr = _norm_case(M, D, dtype, 0, D)
        y, r, rstd = cuda_lib.rms_norm_fwd(x, w, res)
        args = (_np(dy), _np(r), _np(w), 1e-5, _np(dr))
        _near("y", y, o.norm_fwd(_np(r), _np(w), 1e-5)[0], np.abs(o.norm_fwd(_np(r), _np(w), 1e-5)[0]), 8)
        for name, a, b, s in zip(("dx", "dw"), cuda_lib.rms_norm_bwd(dy, rstd, r, w, dr), o.norm_bwd(*args), o.norm_bwd(*args, absolute=True)):
            _near(name, a, b, s, D if name == "dx" else M)


def _check_quant(q, scale, y, block):
    """q and scale against the oracle's, from y in float64.  scale: float32
    arithmetic on y's own error of a few 2^-24.  q: half a step of e4m3, 2^-4 of
    the value (2^-10 below 2^-6), for a value that itself is off by 2^-20."""
    want, ws = o.norm_quant(y, block)
    got, gs = _np(q.float()), _np(scale)
    assert np.all(np.abs(gs - ws) <= 2.0 ** -20 * ws), np.max(np.abs(gs - ws) / ws)
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10) + 2.0 ** -20 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("D,block", [(1, None), (7, None), (64, 32), (96, 32), (256, 256), (512, 256), (1024, 64), (1001, None),
                                     (1002, None), (2048, 128), (4096, None), (4096, 128), (4352, 256), (16384, 32), (16383, None)])
@pytest.mark.parametrize("pad", [0, 3])
def test_norm_in_8_bits(cuda_lib, D, block, pad, dtype):
    mg = cuda_lib
    M = 19 if D < 1000 else 4
    x, res, w, _, _ = _norm_case(M, D, dtype, pad, D + 1, D != 64)
    blocks = D // block if block else 1
    q, scale, r = mg.rms_norm_quant(x, w, res, block=block, out=(torch.full((M, D), 3.0, device=DEV).to(torch.float8_e4m3fn), _nan((M, blocks)), None))
    assert torch.equal(r, x if res is None else x + res)
    _check_quant(q, scale, o.norm_fwd(_np(r), _np(w), 1e-5)[0], block or D)


def test_norm_values_at_the_border(cuda_lib):
    """Rows of zeros, of one value, with an infinity and with a NaN."""
    mg = cuda_lib
    x, w = torch.randn(5, 64, device=DEV), torch.ones(64, device=DEV)
    x[0], x[1], x[2, 40], x[3, 40] = 0.0, 2.0, float("inf"), float("nan")
    y, _, rstd = mg.rms_norm_fwd(x, w, eps=0.0)
    assert torch.isnan(y[0]).all() and torch.allclose(y[1], torch.ones(64, device=DEV)) and torch.isnan(y[3]).all()
    q, scale, _ = mg.rms_norm_quant(x, w, block=32)
    f = q.float()
    assert not f[0].any() and torch.equal(scale[0], torch.full((2,), 1e-30, device=DEV) / 448)
    assert (f[1] == 448).all()
    assert torch.isnan(f[3]).all() and torch.isnan(scale[3]).all()
    assert torch.equal(f[4], mg.rms_norm_quant(x[4:], w, block=32)[0].float()[0])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_norm_in_place_and_shapes(cuda_lib, dtype):
    mg = cuda_lib
    x, res = (torch.randn(2, 3, 5, 72, device=DEV).to(dtype) for _ in range(2))
    w = torch.rand(72, device=DEV)
    y, r, rstd = mg.rms_norm_fwd(x, w, res)
    assert y.shape == x.shape and rstd.shape == x.shape[:-1]
    stream = res.clone()
    y2, r2, _ = mg.rms_norm_fwd(x, w, stream, out=(None, stream, None))
    assert r2 is stream and torch.equal(stream, r) and torch.equal(y2, y)
    stream = res.clone()
    q, scale, r3 = mg.rms_norm_quant(x, w, stream, out=(None, None, stream))
    assert torch.equal(stream, r) and scale.shape == (2, 3, 5, 1)
    y4, r4, _ = mg.rms_norm_fwd(x, w)
    assert r4 is x and torch.equal(mg.rms_norm_fwd(x.transpose(0, 2), w)[0].transpose(0, 2), y4)
    dx, dw = mg.rms_norm_bwd(x[:0], rstd[:0], x[:0], w)
    assert dx.shape == (0, 3, 5, 72) and not dw.any()
    assert mg.rms_norm_fwd(x[:0], w, res[:0])[0].shape == (0, 3, 5, 72)


# ------------------------------------------------------ streams and graphs

def test_on_another_stream_and_in_a_graph(cuda_lib):
    """The calls on a stream of their own and captured: a replay takes the
    inputs that then lie in the buffers and gives an eager call's bits."""
    mg = cuda_lib
    c, d = (Scan(mg, 2, 200, 4, 2, 48, 32, dtype=BF16, seed=s) for s in (12, 13))
    x, res, w, dy, dr = _norm_case(33, 256, BF16, 0, 14)

    def calls():
        oo, last, saved = mg.gated_scan_fwd(c.q, c.k, c.v, c.g, c.S0, scale=c.scale, save=True)
        y, r, rstd = mg.rms_norm_fwd(x, w, res)
        return [oo, last, *mg.gated_scan_bwd(c.do, saved, c.q, c.k, c.v, c.g, c.S0, c.dl, scale=c.scale), y, r,
                *mg.rms_norm_bwd(dy, rstd, r, w, dr), *mg.rms_norm_quant(x, w, res, block=64)[:2]]

    bits = lambda t: t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t  # noqa: E731
    want = calls()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    oo, last, _ = mg.gated_scan_fwd(c.q, c.k, c.v, c.g, c.S0, scale=c.scale, stream=side)
    side.synchronize()
    assert torch.equal(oo, want[0]) and torch.equal(last, want[1])
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = calls()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
        for n in ("q", "k", "v", "g", "S0", "do", "dl"):
            getattr(c, n).copy_(getattr(d, n))
        want = calls()
        torch.cuda.synchronize()


def test_refusals(cuda_lib):
    mg = cuda_lib
    c = Scan(mg, 1, 8, 4, 2, 16, 16, dtype=BF16, seed=15)
    fwd = lambda **k: mg.gated_scan_fwd(*{**dict(q=c.q, k=c.k, v=c.v, g=c.g, S0=c.S0), **k}.values())  # noqa: E731
    for bad in (dict(q=c.q.float()), dict(q=c.q[:, :4]), dict(k=c.k[..., :8]), dict(g=c.g.half()), dict(g=c.g[..., :2]), dict(S0=c.S0[:, :2]),
                dict(v=c.v[0]), dict(v=c.v.half()), dict(v=c.v.cpu()), dict(q=c.q.expand(1, 8, 2, 16)[:, :, :1].expand(1, 8, 3, 16), k=c.k[:, :, :1].expand(1, 8, 3, 16))):
        with pytest.raises(ValueError):
            fwd(**bad)
    wide = torch.zeros(1, 8, 1, 129, device=DEV)
    with pytest.raises(ValueError):
        mg.gated_scan_fwd(wide, wide, c.v.float(), c.g)
    with pytest.raises(mg.MgScanError):
        mg.gated_scan_fwd(c.q, c.k, c.v, c.g, scale=float("nan"))
    with pytest.raises(ValueError):
        mg.gated_scan_bwd(c.do, None, c.q, c.k, c.v, c.g)
    with pytest.raises(ValueError):
        mg.gated_scan_bwd(c.do, torch.zeros(3, device=DEV), c.q, c.k, c.v, c.g)
    with pytest.raises(ValueError):
        mg.gated_scan_step(c.q[0], c.k[0], c.v[0], c.g[0], torch.zeros(8, 4, 16, 16, device=DEV).half())
    with pytest.raises(ValueError):
        mg.gated_scan_step(c.q[0], c.k[0], c.v[0], c.g[0], torch.zeros(4, 4, 16, 16, device=DEV))
    x, w = torch.zeros(4, 64, device=DEV), torch.ones(64, device=DEV)
    for f in (lambda: mg.rms_norm_fwd(x, w[:32]), lambda: mg.rms_norm_fwd(x, None), lambda: mg.rms_norm_fwd(x, w, x[:2]),
              lambda: mg.rms_norm_fwd(x, w, x.bfloat16()), lambda: mg.rms_norm_quant(x, w, block=48), lambda: mg.rms_norm_quant(x, w, block=128),
              lambda: mg.rms_norm_bwd(x, None, x, w), lambda: mg.rms_norm_bwd(x, torch.zeros(3, device=DEV), x, w), lambda: mg.rms_norm_fwd(x, w.cpu())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: mg.rms_norm_fwd(x, w, eps=-1.0), lambda: mg.rms_norm_fwd(torch.zeros(1, 16385, device=DEV), torch.ones(16385, device=DEV)),
              lambda: mg.rms_norm_fwd(x, w, out=(x, None, None))):
        with pytest.raises(mg.MgScanError):
            f()


# --------------------------------------- blocks of several heads, big buffers

@pytest.mark.parametrize("sizes", [(20, 129, 5, 1, 16, 8), (20, 129, 5, 1, 17, 9), (20, 129, 5, 1, 72, 16), (20, 129, 5, 1, 16, 72),
                                   (20, 129, 9, 1, 40, 24), (20, 128, 18, 2, 8, 8)], ids=str)
def test_groups_of_heads_in_parts(cuda_lib, sizes):
    """Batches whose gradients take a group's heads in parts of several, the last
    one smaller, with and without rows on 16-byte boundaries."""
    Scan(cuda_lib, *sizes, dtype=BF16, seed=31).check()


def test_groups_of_heads_in_parts_packed(cuda_lib):
    cu = [0] + list(np.cumsum([129, 1, 0, 128, 257, 300] * 4))
    Scan(cuda_lib, 1, int(cu[-1]), 9, 1, 24, 16, dtype=BF16, cu=[int(x) for x in cu], seed=32).check()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_two_calls_at_once(cuda_lib, dtype):
    """Different inputs on two streams, the calls of both in flight together."""
    mg, n = cuda_lib, 6
    cases = [Scan(mg, 2, 300, 4, 2, 64, 64, dtype=dtype, seed=33 + i) for i in range(2)]
    norms = [_norm_case(500, 384, dtype, 0, 35 + i) for i in range(2)]

    def calls(c, norm):
        x, res, w, dy, dr = norm
        oo, last, saved = mg.gated_scan_fwd(c.q, c.k, c.v, c.g, c.S0, scale=c.scale, save=True)
        _, r, rstd = mg.rms_norm_fwd(x, w, res)
        return [oo, last, *mg.gated_scan_bwd(c.do, saved, c.q, c.k, c.v, c.g, c.S0, c.dl, scale=c.scale), *mg.rms_norm_bwd(dy, rstd, r, w, dr)]

    want = [calls(c, x) for c, x in zip(cases, norms)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(n):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(cases[i], norms[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rows_far_apart(cuda_lib, dtype):
    """Row offsets beyond 2^31 values: the same bits as from dense rows."""
    mg, T, H, N, P = cuda_lib, 2200, 2, 24, 40
    wide = torch.empty(1, T, 1 << 20, dtype=dtype, device=DEV)
    gen = torch.Generator(DEV).manual_seed(37)
    at, far = 0, []
    for width in (N, N, P, P):
        part = wide[..., at:at + H * width]
        part.copy_(torch.randn(1, T, H * width, generator=gen, device=DEV))
        far.append(part.unflatten(-1, (H, width)))
        at += H * width
    g = torch.nn.functional.logsigmoid(torch.randn(1, T, H, generator=gen, device=DEV) + 2)
    got = []
    for q, k, v, do in (far, [t.contiguous() for t in far]):
        oo, last, saved = mg.gated_scan_fwd(q, k, v, g, save=True)
        got.append([oo, last, *mg.gated_scan_bwd(do, saved, q, k, v, g)[:4]])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    x, res, dy = (wide[0, :, i * 96:(i + 1) * 96] for i in range(1, 4))
    w = torch.randn(96, generator=gen, device=DEV)
    for t in (x, res, dy):
        t.normal_(generator=gen)
    got = []
    for a, b, c in ((x, res, dy), tuple(t.contiguous() for t in (x, res, dy))):
        y, r, rstd = mg.rms_norm_fwd(a, w, b)
        q8, sc, _ = mg.rms_norm_quant(a, w, b, block=32)
        got.append([y, r, rstd, q8.view(torch.uint8), sc, *mg.rms_norm_bwd(c, rstd, r, w, b)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_a_pool_of_many_states(cuda_lib):
    """Slots whose states begin beyond 2^31 values."""
    mg, H, N, P = cuda_lib, 32, 128, 128
    pool = torch.empty(4100, H, N, P, device=DEV)
    slots = torch.tensor([4099, 0, -1, 4096, 1 << 40], device=DEV)
    gen = torch.Generator(DEV).manual_seed(38)
    q, k = (torch.randn(5, 4, N, generator=gen, device=DEV) for _ in range(2))
    v, g = torch.randn(5, H, P, generator=gen, device=DEV), -torch.rand(5, H, generator=gen, device=DEV)
    own = torch.randn(5, H, N, P, generator=gen, device=DEV)
    for i in (0, 1, 3):
        pool[slots[i]] = own[i]
    want = mg.gated_scan_step(q, k, v, g, own, scale=0.1)
    got = mg.gated_scan_step(q, k, v, g, pool, slots=slots, scale=0.1)
    assert torch.equal(got[[0, 1, 3]], want[[0, 1, 3]]) and not got[[2, 4]].any()
    assert all(torch.equal(pool[slots[i]], own[i]) for i in (0, 1, 3))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_signalling_nans_do_not_pass_through_a_workspace(cuda_lib, dtype):
    """Gates and states whose bits are those of a look-back record's tag, then a
    scan that looks back in the same workspace: its results are a fresh one's."""
    mg = cuda_lib
    c = Scan(mg, 1, 700, 4, 2, 32, 32, dtype=dtype, seed=39)
    a, b = torch.rand(2, 700, 96, device=DEV), torch.randn(2, 700, 96, device=DEV)
    want = mg.linear_scan_fwd(a, b)
    size = max(mg.load().mg_gated_scan_workspace_size(1, 700, 4, 2, 32, 32, 1, 0, mg._DT[dtype], back) for back in (0, 1))
    ws = mg.new_workspace(max(size, mg.linear_workspace_size(2, 700, 96)), device=DEV)
    for epoch in range(1, 5):
        for t in (c.g, c.S0, c.dl):
            t.view(torch.int32).fill_((0xffa00000 | epoch) - (1 << 32))
        _, _, saved = mg.gated_scan_fwd(c.q, c.k, c.v, c.g, c.S0, scale=c.scale, save=True, ws=ws)
        mg.gated_scan_bwd(c.do, saved, c.q, c.k, c.v, c.g, c.S0, c.dl, scale=c.scale, ws=ws)
        got = mg.linear_scan_fwd(a, b, ws=ws)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
