"""The words of the look-back's records in a workspace: their tags have bits
that no value left there by an op has."""
from __future__ import annotations

import numpy as np
import pytest

import linear_recurrence_scans_gb300 as mg

EPOCHS = 1 << 21   # after so many launches the tags begin again


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


def test_no_computed_value_has_a_tags_bits(lib):
    """Neither a finite float nor an infinity nor the GPU's NaN, for any launch."""
    epochs = [*range(4096), *range(4096, EPOCHS, 61), EPOCHS - 1, EPOCHS, 3 * EPOCHS + 5, (1 << 49) - 1, (1 << 64) - 1]
    tags = np.array([lib.mg_testing_record_tag(e) for e in epochs], dtype=np.uint32)
    assert np.isnan(tags.view(np.float32)).all()
    assert not (tags == 0x7fffffff).any() and not (tags & 0x00400000).any()   # signalling


def test_tags_are_neither_zeros_nor_flags_nor_each_others(lib):
    tags = np.array([lib.mg_testing_record_tag(e) for e in range(EPOCHS)], dtype=np.uint32)
    assert np.unique(tags).size == EPOCHS and (tags != 0).all()
    assert not ((tags >> 19) == 0x1fff).any()   # a flag's upper half: its top 13 bits are set
    assert lib.mg_testing_record_tag(EPOCHS + 7) == tags[7]
