"""examples/moe_layer.py end to end."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_moe_layer_example(monkeypatch):
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    monkeypatch.setattr(sys, "argv", ["moe_layer.py", "--tokens", "96"])
    import moe_layer
    worst, losses = moe_layer.main()
    # bf16 rows of a residual stream: a few half steps of 2^-8
    assert worst < 3 * 2.0 ** -8
    assert losses[-1] < losses[0]
