"""Attention of many rows whose keys are cut into parts, joined by 16 rows a workgroup and by 128: ragged sequences
without new tokens and with a few among them, every head size and type."""
from __future__ import annotations

import pytest

from kvsingle import KINDS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_parts_of_ragged_sequences(dev, dim, kinds):
    for window in (0, 700):
        check(dev, [2500, 900, 0, 1700], [40, 3, 0, 130], 2, 1, dim, kinds, 8.0, window=window, parts=32, seed=3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kinds", [KINDS[0], KINDS[1], KINDS[3]])
def test_parts_joined_by_whole_tiles(dev, kinds, causal):
    """Three tiles of 64 heads, which are more than 128: a workgroup joins all rows of one."""
    check(dev, [1300], [300], 64, 64, 64, kinds, 8.0, causal=causal, parts=8, seed=5)
