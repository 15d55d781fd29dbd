"""The words of the look-back's records in a workspace: their tags have bits
that no value left there by an op has."""
from __future__ import annotations

import numpy as np
import pytest

import linear_recurrence_scans_gb300 as mg

BITS = 21   # of the launch's number in a tag: the low ones at even places, the next at odd


@pytest.fixture(scope="module")
def lib():
    from linear_recurrence_scans_gb300 import _build
    _build.build()
    return mg.load()


def _tags(lib, epochs):
    return np.array([[lib.mg_testing_record_tag(e, odd) for odd in (0, 1)] for e in epochs], dtype=np.uint32)


EPOCHS = [*range(4096), *range(4096, 1 << BITS, 61), *((1 << k) + d for k in (BITS, 2 * BITS, 49) for d in (-1, 0, 1)),
          *range(0, 1 << (2 * BITS), (1 << 27) + 12345), (1 << 64) - 1]


def test_no_computed_value_has_a_tags_bits(lib):
    """Neither a finite float nor an infinity nor the GPU's NaN, for any launch."""
    tags = _tags(lib, EPOCHS)
    assert np.isnan(tags.view(np.float32)).all()
    assert not (tags == 0x7fffffff).any() and not (tags & 0x00400000).any()   # signalling


def test_tags_are_neither_zeros_nor_flags_nor_each_others(lib):
    tags = _tags(lib, EPOCHS)
    assert (tags != 0).all()
    assert not ((tags >> 19) == 0x1fff).any()   # a flag's upper half: its top 13 bits are set
    pairs = tags[:, 0].astype(np.uint64) << np.uint64(32) | tags[:, 1].astype(np.uint64)
    assert np.unique(pairs).size == len({e % (1 << (2 * BITS)) for e in EPOCHS})
    low = np.array([lib.mg_testing_record_tag(e, 0) for e in range(1 << BITS)], dtype=np.uint32)
    assert np.unique(low).size == 1 << BITS
