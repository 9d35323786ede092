"""The training example runs its operators together, and both losses fall."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_losses_fall():
    import train_indexer
    losses = train_indexer.main(steps=12, S=256, vocab=2003)
    assert losses[-1][0] < 0.9 * losses[0][0]
    assert losses[-1][1] < 0.5 * losses[0][1]
