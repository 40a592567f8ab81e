"""A decoder layer and the head, as examples/decoder_layer.py runs them: every operator between the products checked
on its own inputs in 64 bits."""
import pytest

from examples import decoder_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("args", [["--steps", "5"], ["--steps", "2", "--context", "1", "--tokens", "1"], ["--steps", "3", "--context", "777", "--tokens", "4"]])
def test_the_operators_of_a_step_agree_with_64_bits(args):
    assert decoder_layer.main(args) < 1e-5  # fp32 attention: 22 bits of each factor, scores of order ten; the others nearer
