"""Host-side checks of the mixer operators' C entry points that need no GPU:
sizes, types, strides, buffers and workspaces are refused before any launch
(the addresses here are made up and never read)."""
from __future__ import annotations

import pytest

import linear_recurrence_scans_gb300 as mg

BASE = 1 << 40


def at(i):
    return BASE + (i << 32)


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


def _scan(lib, **k):
    v = dict(x=at(1), ldx=8, raw=at(2), ldraw=8, A=at(3), Bm=at(4), ldb=4, Cm=at(5), ldc=4, dt=0, D_=None, bias=None,
             sp=1, h0=None, cu=None, nseq=2, y=at(6), last=at(7), saved=None, B=2, T=6, D=8, N=4, G=1, ws=at(8),
             wsb=1 << 30)
    v.update(k)
    return lib.mg_selective_scan_fwd(*v.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(dt=7), mg.MG_ERR_UNSUPPORTED, b"dtype"),
    (dict(B=-1), mg.MG_ERR_INVALID_ARG, b"negative"),
    (dict(N=65), mg.MG_ERR_UNSUPPORTED, b"N = 65"),
    (dict(N=0), mg.MG_ERR_UNSUPPORTED, b"N = 0"),
    (dict(G=3), mg.MG_ERR_INVALID_ARG, b"multiple"),
    (dict(G=0), mg.MG_ERR_INVALID_ARG, b"multiple"),
    (dict(ldx=7), mg.MG_ERR_INVALID_ARG, b"row stride"),
    (dict(ldb=3), mg.MG_ERR_INVALID_ARG, b"row stride"),
    (dict(nseq=3), mg.MG_ERR_INVALID_ARG, b"nseq"),
    (dict(cu=at(9), nseq=3), mg.MG_ERR_INVALID_ARG, b"B must be 1"),
    (dict(cu=at(9) + 4, nseq=3, B=1), mg.MG_ERR_INVALID_ARG, b"aligned"),
    (dict(ws=None), mg.MG_ERR_INVALID_ARG, b"workspace"),
    (dict(ws=at(8) + 16), mg.MG_ERR_INVALID_ARG, b"aligned"),
    (dict(wsb=8), mg.MG_ERR_INVALID_ARG, b"needed"),
    (dict(x=None), mg.MG_ERR_INVALID_ARG, b"x is NULL"),
    (dict(x=at(1) + 8), mg.MG_ERR_INVALID_ARG, b"aligned"),
    (dict(y=at(1)), mg.MG_ERR_INVALID_ARG, b"overlaps"),
    (dict(last=at(6) + 16), mg.MG_ERR_INVALID_ARG, b"overlaps"),
    (dict(T=1 << 36), mg.MG_ERR_UNSUPPORTED, b"2^36"),
])
def test_scan_refusals(lib, bad, status, word):
    assert _scan(lib, **bad) == status
    assert word in lib.mg_last_error_detail(), lib.mg_last_error_detail()


def test_calls_without_channels_are_ok(lib):
    assert _scan(lib, D=0, G=1) == mg.MG_OK
    assert lib.mg_causal_conv_step(None, 8, 0, None, None, None, 0, None, 1, None, 0, 8, 4, None) == mg.MG_OK
    assert lib.mg_selective_scan_step(None, 8, None, 8, None, None, 4, None, 4, 0, None, None, 1, None, 0, None, None,
                                      0, 8, 4, 1, None) == mg.MG_OK
    assert lib.mg_group_norm_fwd(None, 8, None, 8, 0, None, None, 1e-5, 0, 0, 1, None, None, 0, 8, 1, None) == mg.MG_OK


def test_step_refusals(lib):
    def step(nslots=4, slots=at(5), state=at(4), B=2):
        return lib.mg_selective_scan_step(at(1), 8, at(2), 8, at(3), at(6), 4, at(7), 4, 0, None, None, 1, state,
                                          nslots, slots, at(9), B, 8, 4, 1, None)
    assert step(nslots=-1) == mg.MG_ERR_INVALID_ARG
    assert step(nslots=1, slots=None) == mg.MG_ERR_INVALID_ARG and b"states" in lib.mg_last_error_detail()
    assert step(slots=at(5) + 4) == mg.MG_ERR_INVALID_ARG
    assert step(state=None) == mg.MG_ERR_INVALID_ARG and b"state" in lib.mg_last_error_detail()
    assert step(state=at(1)) == mg.MG_ERR_INVALID_ARG and b"overlaps" in lib.mg_last_error_detail()


def test_conv_and_norm_refusals(lib):
    conv = lambda W, ld=8: lib.mg_causal_conv_fwd(at(1), ld, 0, at(2), None, None, None, 2, 1, at(3), None, 2, 6, 8, W, at(4), 1 << 20, None)  # noqa: E731
    assert conv(0) == mg.MG_ERR_UNSUPPORTED and conv(9) == mg.MG_ERR_UNSUPPORTED
    assert conv(4, 7) == mg.MG_ERR_INVALID_ARG

    def norm(gate=0, z=None, G=1, D=8, eps=1e-5):
        return lib.mg_group_norm_fwd(at(1), D, z, D, 0, at(3), None, eps, 0, gate, 1, at(4), None, 6, D, G, None)
    assert norm(G=3) == mg.MG_ERR_INVALID_ARG
    assert norm(gate=1) == mg.MG_ERR_INVALID_ARG and norm(z=at(2)) == mg.MG_ERR_INVALID_ARG
    assert norm(gate=5, z=at(2)) == mg.MG_ERR_INVALID_ARG
    assert norm(D=16385) == mg.MG_ERR_UNSUPPORTED
    assert norm(eps=float("nan")) == mg.MG_ERR_INVALID_ARG


def test_sizes(lib):
    assert lib.mg_selective_scan_fwd_workspace_size(2, 6, 8, 4, 1, 2) >= 256
    assert lib.mg_selective_scan_bwd_workspace_size(2, 6, 8, 65, 1, 2) == 0
    assert lib.mg_selective_scan_fwd_workspace_size(2, 6, 8, 4, 3, 2) == 0
    rows = lib.mg_selective_scan_saved_rows()
    assert lib.mg_selective_scan_saved_size(2, rows + 1, 8, 4) == 2 * 2 * 8 * 4 * 4
    assert lib.mg_causal_conv_workspace_size(2, 6, 8, 9) == 0
    assert lib.mg_causal_conv_workspace_size(2, 6, 8, 4) > 256
    assert lib.mg_group_norm_workspace_size(6, 8, 3) == 0 and lib.mg_group_norm_workspace_size(6, 8, 2) > 256
