"""Host-side checks of the gated block's operators beside test_block_abi_cpu.py's:
sizes of nothing, copies' ranges, calls by name (no GPU needed)."""
from __future__ import annotations

import inspect
import subprocess

import pytest
import torch

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


FLAT = r"""
#include "flat_rows.h"
#include <cstdio>
int main()
{
    long bad = 0;
    for (int wide = 4; wide <= 8; wide += 4)
        for (long D = 1; D < 200; ++D)
            for (long M = 1; M < 70; ++M)
                for (long r = 0; r < M; ++r) {
                    const long b = mg::flat_copy_begin(r, D, wide), e = mg::flat_copy_end(r, D, M, wide);
                    bad += b % wide != 0 || e % wide != 0 || b < 0 || b > r * D;
                    if (e > b) bad += e > M * D || e - b > D + 2 * wide - 2;      // the array's end; a slot's room
                    // what is left out: less than a piece, of the array's last one
                    for (long v = r * D; v < (r + 1) * D; ++v)
                        if (v >= e) bad += v < M * D / wide * wide;
                }
    std::printf("%ld\n", bad);
}
"""


def test_copies_of_flat_rows_stay_in_the_array(tmp_path):
    """The ranges that the norm's gradients copy (csrc/flat_rows.h), compiled as
    the kernels compile them."""
    from linear_recurrence_scans_gb300 import _build
    (tmp_path / "flat.cpp").write_text(FLAT)
    subprocess.run(["g++", "-std=c++17", "-I", _build.CSRC, "-o", tmp_path / "flat", tmp_path / "flat.cpp"], check=True)
    assert subprocess.run([tmp_path / "flat"], capture_output=True, text=True, check=True).stdout == "0\n"


CALLS = ("gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "rms_norm_fwd", "rms_norm_quant", "rms_norm_bwd")


@pytest.mark.parametrize("name", CALLS)
def test_every_argument_has_its_name(name):
    """What the signature shows may be given by name, the first tensor and the
    stream too: the call gets as far as its checks of tensors."""
    f = getattr(mg, name)
    shown = inspect.signature(f).parameters
    assert "stream" in shown
    tensors = {n: torch.zeros(1, 1, 1, 1) for n, p in shown.items() if p.default is inspect.Parameter.empty}
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        f(**tensors, stream=None)
    with pytest.raises(TypeError, match="missing"):
        f()


@pytest.mark.parametrize("value", [1e39, -1e39, 3.5e38, float("inf"), float("nan")])
def test_factors_beyond_float32(lib, value):
    """scale and eps are float32 in the kernels: what is infinite there is refused."""
    at = lambda i: (1 << 40) + (i << 34)  # noqa: E731
    size = (2, 6, 4, 2, 4, 3)
    fwd = lib.mg_gated_scan_fwd(at(1), 8, at(2), 8, at(3), 12, at(4), 4, 0, value, None, None, 2, at(5), at(6), None, *size, at(7), 1 << 30, None)
    assert fwd == mg.MG_ERR_INVALID_ARG and b"scale" in lib.mg_last_error_detail()
    bwd = lib.mg_gated_scan_bwd(at(1), 12, at(2), at(3), 8, at(4), 8, at(5), 12, at(6), 4, 0, value, None, None, 2, at(7), at(8), at(9), at(10), None,
                                *size, at(11), 1 << 30, None)
    assert bwd == mg.MG_ERR_INVALID_ARG and b"scale" in lib.mg_last_error_detail()
    step = lib.mg_gated_scan_step(at(1), 8, at(2), 8, at(3), 12, at(4), 4, 0, value, at(5), 4, at(6), at(7), 2, 4, 2, 4, 3, None)
    assert step == mg.MG_ERR_INVALID_ARG and b"scale" in lib.mg_last_error_detail()
    norm = lib.mg_rms_norm_fwd(at(1), 64, None, 64, 0, at(3), value, at(4), None, None, 6, 64, None)
    assert norm == mg.MG_ERR_INVALID_ARG and b"eps" in lib.mg_last_error_detail()
    quant = lib.mg_rms_norm_quant(at(1), 64, None, 64, 0, at(3), value, at(4), at(5), None, 32, 6, 64, None)
    assert quant == mg.MG_ERR_INVALID_ARG and b"eps" in lib.mg_last_error_detail()


def test_rows_without_channels(lib):
    """They have no mean: refused, as their statistics would stay unwritten."""
    at = lambda i: (1 << 40) + (i << 34)  # noqa: E731
    assert lib.mg_rms_norm_fwd(at(1), 0, None, 0, 0, at(2), 1e-5, at(3), None, at(4), 6, 0, None) == mg.MG_ERR_INVALID_ARG
    assert b"channels" in lib.mg_last_error_detail()
    assert lib.mg_rms_norm_quant(at(1), 0, None, 0, 1, at(2), 1e-5, at(3), at(4), None, 0, 6, 0, None) == mg.MG_ERR_INVALID_ARG
    assert lib.mg_rms_norm_fwd(None, 0, None, 0, 0, None, 1e-5, None, None, None, 0, 0, None) == mg.MG_OK
    assert lib.mg_rms_norm_fwd(None, 64, None, 64, 0, None, 1e-5, None, None, None, 0, 64, None) == mg.MG_OK
