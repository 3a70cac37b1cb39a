"""examples/quantize_and_serve.py: rounding, packing, a prompt, decoding steps
through experts and a gradient, together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_quantize_and_serve():
    spec = importlib.util.spec_from_file_location("quantize_and_serve", os.path.join(ROOT, "examples", "quantize_and_serve.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    res = mod.main(["--hidden", "256", "--ffn", "320", "--experts", "4", "--tokens", "130"])
    # results are rounded to bfloat16 once (2^-8 / sqrt(3) in the mean square of
    # a uniform rounding), the gradient's weights once more
    for what in ("prompt", "experts", "gradient"):
        assert res[f"{what} against the rounded weights"] < 2.0 ** -7, res
    # four bits with groups of 64: steps of about 1/3 of the weights' deviation,
    # an error of a step / sqrt(12) each
    assert res["rounded prompt against float32"] < 0.25, res
