"""The example layer: its training steps fit a target, its 4-bit copy answers like it."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "moe_layer.py")


def test_moe_layer_trains_and_decodes():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.main(say=lambda *_: None)
    # 30 steps of plain gradient descent take the loss well below where it began; 16
    # levels over a normal group's range of about six deviations are off by
    # 6 / 15 / sqrt(12) = 0.12 of one, in three weight matrices of the block.
    assert got["losses"][-1] < 0.7 * got["losses"][0]
    assert got["decode_off"] < 3 * 0.12
