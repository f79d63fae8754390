"""The training example end to end: norm with dropout, loss, gradients and
descent learn the synthetic language, and the chain drafts it."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_training_example_learns_to_draft():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import train_head
    finally:
        sys.path.pop(0)
    losses, right = train_head.main(steps=300)
    assert losses[0] > 5.0                   # about log 256
    assert losses[-1] < 0.5 * losses[0]
    assert right > 0.5                       # chance: 0.4 %
