"""The example of a layer with its own keys and values: append, prompt attention and decode
together, each step against the same layer over the whole sequences at once."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "grouped_head_layer", os.path.join(ROOT, "examples", "grouped_head_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_bf16_cache(example):
    # |o| <= max |v| < 6.  Both sides attend the same bf16 q, k and v: each rounds its weights
    # to bf16 (2^-8 of a weighted mean of |v|, itself under 6) and its result (2^-8 of |o|).
    assert example.run(False) <= 4 * 6 * 2.0 ** -8


def test_fp8_cache(example):
    # Keys and values are rounded to e4m3: by 2^-4 of each at most, uniformly, so 2^-4 / sqrt(3)
    # = 0.036 of it (one sigma).  A score, a sum of 128 products of unit variance over sqrt(128),
    # is then off by 0.036 (one sigma), a weight by as much of itself; a value by 0.036 |v|, |v|
    # < 6.  Where one key has all the weight, o is off by a value's own error, 2^-4 * 6; where
    # several share it, the weights' errors add 0.036 * 6 a sigma: five sigma.
    assert example.run(True) <= 6 * (2.0 ** -4 + 5 * 0.036)
