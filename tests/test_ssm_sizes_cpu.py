"""Sizes whose launches a grid does not hold are refused before any launch (the
addresses here are made up, far apart, and never read)."""
from __future__ import annotations

import pytest

import linear_recurrence_scans_gb300 as mg

WS, WSB = 1 << 60, 1 << 60


def at(i):
    return i << 48


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


def _refused(lib, status, word=b"blocks"):
    assert status == mg.MG_ERR_UNSUPPORTED and word in lib.mg_last_error_detail(), (status, lib.mg_last_error_detail())


def _scan_fwd(lib, B, T, D, N, G, dt=0):
    return lib.mg_selective_scan_fwd(at(1), D, at(2), D, at(3), at(4), G * N, at(5), G * N, dt, None, None, 1, None,
                                     None, B, at(6), None, None, B, T, D, N, G, WS, WSB, None)


def _scan_bwd(lib, B, T, D, N, G, dt=0):
    return lib.mg_selective_scan_bwd(at(1), D, at(2), at(3), D, at(4), D, at(5), at(6), G * N, at(7), G * N, dt, None,
                                     None, 1, None, None, None, B, at(8), at(9), at(10), at(11), at(12), None, None,
                                     None, B, T, D, N, G, WS, WSB, None)


@pytest.mark.parametrize("dt", [0, 1])
def test_scan_blocks(lib, dt):
    many = (4097, 1, 1 << 20, 1, 1 << 20)   # 2^32 + 2^20 tiles of one channel: 2^20 in 32 bits
    _refused(lib, _scan_fwd(lib, *many, dt))
    _refused(lib, _scan_bwd(lib, *many, dt))
    _refused(lib, _scan_fwd(lib, 2048, 1, 1 << 20, 1, 1 << 20, dt))   # 2^31
    _refused(lib, _scan_bwd(lib, 1, 1, 1 << 30, 64, 1, dt))           # the sums of the parts
    _refused(lib, _scan_bwd(lib, 1, 1 << 30, 16, 64, 16, dt))         # dB and dC


@pytest.mark.parametrize("dt", [0, 1])
def test_sums_of_parts(lib, dt):
    D = 1 << 33
    _refused(lib, lib.mg_causal_conv_bwd(at(1), D, at(2), D, dt, at(3), None, None, None, None, 1, 1, at(4), at(5), None,
                                         None, 1, 1, D, 8, WS, WSB, None))
    D = 1 << 36
    _refused(lib, lib.mg_group_norm_bwd(at(1), D, at(2), at(3), D, None, D, dt, at(4), None, 0, 0, 1, at(5), None, at(6),
                                        None, 1, D, 1 << 22, WS, WSB, None))


def test_token_blocks(lib):
    B, D = 1 << 33, 1
    _refused(lib, lib.mg_selective_scan_step(at(1), D, at(2), D, at(3), at(4), 1, at(5), 1, 0, None, None, 1, at(6), B,
                                             None, at(7), B, D, 1, 1, None))


def test_norm_rows(lib):
    """M G is held in 32 bits: 2^31 is one too many."""
    for M, G in ((1 << 31, 1), (1 << 30, 2), (1 << 28, 8)):
        fwd = lambda M: lib.mg_group_norm_fwd(at(1), G, None, G, 1, at(3), None, 1e-5, 0, 0, 1, at(4), None, M, G, G, None)  # noqa: E731
        _refused(lib, fwd(M), b"M G")
        _refused(lib, lib.mg_group_norm_bwd(at(1), G, at(2), at(3), G, None, G, 1, at(4), None, 0, 0, 1, at(5), None,
                                            at(6), None, M, G, G, WS, WSB, None), b"M G")
        assert lib.mg_group_norm_workspace_size(M, G, G) == 0 and lib.mg_group_norm_workspace_size(M - 1, G, G) > 0
