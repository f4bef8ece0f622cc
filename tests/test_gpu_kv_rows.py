"""Attention over rows of q whose values are far apart: each as exact as the terms that it is taken in allow."""
from __future__ import annotations

import pytest

from kvsingle import KINDS, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_q_values_apart(dev, dim, kinds):
    """A row's values down to 2^-15 of its largest, each of which is one key's score."""
    for spread in (1.0, 4.0):
        check(dev, [32, 20, 7], [1, 2, 3], 4, 2, dim, kinds, spread, smallest=15)
        check(dev, [32, 30], [32, 20], 4, 2, dim, kinds, spread, smallest=15)
