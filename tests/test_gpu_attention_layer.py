"""The products, the 4-bit cache and the attention together, as examples/attention_layer.py runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")


@pytest.mark.parametrize("args", [
    ["--steps", "3", "--context", "70", "--tokens", "1"],
    ["--steps", "2", "--context", "500", "--tokens", "4"],
    ["--steps", "2", "--context", "700", "--tokens", "3", "--window", "100", "--sinks", "4"],
])
def test_attention_layer(args):
    spec = importlib.util.spec_from_file_location("attention_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(args) < 1e-5   # fp32 attention: 22 bits of each factor, scores of order ten
