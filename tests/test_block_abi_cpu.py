"""Host-side checks of the gated block's C entry points that need no GPU:
sizes, types, strides, buffers and workspaces are refused before any launch
(the addresses here are made up and never read)."""
from __future__ import annotations

import ctypes
import struct

import pytest

import linear_recurrence_scans_gb300 as mg

BASE = 1 << 40
INVALID, UNSUPPORTED = mg.MG_ERR_INVALID_ARG, mg.MG_ERR_UNSUPPORTED


def at(i):
    return BASE + (i << 34)


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


def _fwd(lib, **k):
    v = dict(q=at(1), ldq=8, k=at(2), ldk=8, v=at(3), ldv=12, g=at(4), ldg=4, dt=0, scale=1.0, S0=None, cu=None, nseq=2, o=at(5),
             last=at(6), saved=None, B=2, T=6, H=4, G=2, N=4, P=3, ws=at(7), wsb=1 << 30)
    v.update(k)
    return lib.mg_gated_scan_fwd(*v.values(), None)


def _bwd(lib, **k):
    v = dict(do=at(1), lddo=12, saved=at(2), q=at(3), ldq=8, k=at(4), ldk=8, v=at(5), ldv=12, g=at(6), ldg=4, dt=1, scale=1.0, dl=None,
             cu=None, nseq=2, dq=at(7), dk=at(8), dv=at(9), dg=at(10), dS0=None, B=2, T=6, H=4, G=2, N=4, P=3, ws=at(11), wsb=1 << 30)
    v.update(k)
    return lib.mg_gated_scan_bwd(*v.values(), None)


SCAN = [
    (dict(dt=7), UNSUPPORTED, b"dtype"), (dict(B=-1), INVALID, b"negative"), (dict(N=129), UNSUPPORTED, b"N = 129"),
    (dict(P=0), UNSUPPORTED, b"P = 0"), (dict(P=129), UNSUPPORTED, b"P = 129"), (dict(G=3), INVALID, b"multiple"), (dict(G=0), INVALID, b"multiple"),
    (dict(ldq=7), INVALID, b"row stride"), (dict(ldv=11), INVALID, b"row stride"), (dict(ldg=3), INVALID, b"row stride"),
    (dict(nseq=3), INVALID, b"nseq"), (dict(cu=at(12), nseq=3), INVALID, b"B must be 1"), (dict(cu=at(12) + 4, nseq=3, B=1), INVALID, b"aligned"),
    (dict(ws=None), INVALID, b"workspace"), (dict(ws=at(13) + 16), INVALID, b"aligned"), (dict(wsb=8), INVALID, b"needed"),
    (dict(q=None), INVALID, b"q is NULL"), (dict(v=at(3) + 8), INVALID, b"aligned"), (dict(scale=float("inf")), INVALID, b"scale"),
    (dict(T=1 << 36), UNSUPPORTED, b"2^36"), (dict(H=1 << 17, G=1, ldv=3 << 17, ldg=1 << 17), UNSUPPORTED, b"heads"),
]


@pytest.mark.parametrize("bad,status,word", SCAN + [
    (dict(o=at(1)), INVALID, b"overlaps"), (dict(last=at(5) + 16), INVALID, b"overlaps"), (dict(saved=at(6)), INVALID, b"overlaps")])
def test_scan_refusals(lib, bad, status, word):
    assert _fwd(lib, **bad) == status and word in lib.mg_last_error_detail(), lib.mg_last_error_detail()


@pytest.mark.parametrize("bad,status,word", SCAN + [
    (dict(saved=None), INVALID, b"saved is NULL"), (dict(dq=at(8)), INVALID, b"overlaps"), (dict(dg=None), INVALID, b"dg is NULL"),
    (dict(lddo=5), INVALID, b"row stride")])
def test_scan_gradients_refusals(lib, bad, status, word):
    assert _bwd(lib, **bad) == status and word in lib.mg_last_error_detail(), lib.mg_last_error_detail()


def test_step_refusals(lib):
    def step(nslots=4, slots=at(6), state=at(5), B=2, o=at(7), N=4):
        return lib.mg_gated_scan_step(at(1), 8, at(2), 8, at(3), 12, at(4), 4, 0, 1.0, state, nslots, slots, o, B, 4, 2, N, 3, None)
    assert step(nslots=-1) == INVALID and step(N=200) == UNSUPPORTED
    assert step(nslots=1, slots=None) == INVALID and b"states" in lib.mg_last_error_detail()
    assert step(slots=at(6) + 4) == INVALID
    assert step(state=None) == INVALID and b"state" in lib.mg_last_error_detail()
    assert step(state=at(1)) == INVALID and b"overlaps" in lib.mg_last_error_detail()
    assert step(B=0, o=None) == mg.MG_OK


def test_norm_refusals(lib):
    def fwd(x=at(1), ldx=64, res=at(2), ldres=64, dt=0, w=at(3), eps=1e-5, y=at(4), r=at(5), M=6, D=64):
        return lib.mg_rms_norm_fwd(x, ldx, res, ldres, dt, w, eps, y, r, None, M, D, None)
    assert fwd(D=16385, ldx=16385, ldres=16385) == UNSUPPORTED and fwd(dt=3) == UNSUPPORTED
    assert fwd(ldx=63) == INVALID and fwd(ldres=63) == INVALID and fwd(M=-1) == INVALID
    assert fwd(res=None) == INVALID and fwd(r=None) == INVALID
    assert fwd(eps=-1.0) == INVALID and fwd(eps=float("nan")) == INVALID and fwd(eps=float("inf")) == INVALID
    assert fwd(y=at(1)) == INVALID and b"overlaps" in lib.mg_last_error_detail()
    assert fwd(r=at(2), ldres=72) == INVALID and b"overlaps" in lib.mg_last_error_detail()   # in place only where both are dense
    assert fwd(w=None) == INVALID and fwd(M=0, x=None) == mg.MG_OK

    def quant(block=32, D=64, q=at(4), scale=at(6)):
        return lib.mg_rms_norm_quant(at(1), D, None, D, 1, at(3), 1e-5, q, scale, None, block, 6, D, None)
    assert quant(block=48) == UNSUPPORTED and quant(block=128) == INVALID and quant(block=-32) == UNSUPPORTED
    assert quant(scale=None) == INVALID and quant(q=at(1)) == INVALID

    def bwd(ldr=64, dw=at(5), ws=at(6), wsb=1 << 30, dx=at(4), M=6):
        return lib.mg_rms_norm_bwd(at(1), 64, at(2), at(3), ldr, None, 64, 0, at(7), dx, dw, M, 64, ws, wsb, None)
    assert bwd(ldr=1) == INVALID and bwd(ws=None) == INVALID and bwd(wsb=256) == INVALID and bwd(dw=None) == INVALID
    assert bwd(dx=at(3)) == INVALID


def test_sizes(lib):
    size = lib.mg_gated_scan_workspace_size
    assert size(2, 6, 4, 2, 4, 3, 2, 0, 0, 0) >= 256 and size(2, 6, 4, 3, 4, 3, 2, 0, 0, 0) == 0
    assert size(2, 6, 4, 2, 129, 3, 2, 0, 1, 1) == 0 and size(0, 6, 4, 2, 4, 3, 0, 0, 1, 1) == 256
    saved = lib.mg_gated_scan_saved_size
    assert saved(2, 6, 4, 4, 3, 2, 0, 0) == 2 * 4 * 12 * 4
    # a packed batch has room for a chunk that every sequence leaves unfilled
    assert saved(1, 6, 4, 4, 3, 2, 1, 0) == 2 * 4 * 12 * 4 and saved(1, 6, 4, 4, 3, 9, 1, 0) == 6 * 4 * 12 * 4
    assert lib.mg_rms_norm_workspace_size(6, 64) > 256 and lib.mg_rms_norm_workspace_size(6, 16385) == 0


def test_calls_by_words(lib):
    """The packed form takes as many words as its call has arguments."""
    for op, n in ((0, 25), (1, 30), (2, 20), (3, 13), (4, 14), (5, 16)):
        assert lib.mg_block_call(op, struct.pack("q", 0), n + 1) == INVALID and b"%d expected" % n in lib.mg_last_error_detail()
    assert lib.mg_block_call(9, struct.pack("q", 0), 1) == INVALID
    assert lib.mg_block_call(0, ctypes.c_char_p(None), 25) == INVALID
    from linear_recurrence_scans_gb300 import block
    assert {n: c for n, (_, _, c) in block._OPS.items()} == dict(zip(block._OPS, (25, 30, 20, 13, 14, 16)))
