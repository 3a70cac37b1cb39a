"""examples/quantize_and_serve.py: a prompt through the rounded experts, and a
gradient back."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_prompt_through_the_experts_and_back():
    spec = importlib.util.spec_from_file_location("quantize_and_serve", os.path.join(ROOT, "examples", "quantize_and_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    res = mod.main(["--hidden", "320", "--ffn", "448", "--experts", "6", "--top-k", "3", "--tokens", "200"])
    # A rounding to bfloat16 is 2^-8 / sqrt(3) of a value in the mean square at most.
    # Forward there are five (both inner products, the activation, the down product,
    # the result), whose sum no independence is needed for: 0.0113.
    assert res["expert layer against the rounded weights"] < 2.0 ** -6, res
    # Backward eight, two of them of weights: 0.018; and the two checkpoints: a step of
    # 1 / 63.75 of the largest of 32 values at most, that is of about 2.1 deviations (2.5 for
    # one block in three), an error of a step / sqrt(12): 0.0113 of a deviation each, in
    # independent terms.  0.018 + 0.016.
    assert res["its gradient against the rounded weights"] < 0.034, res
