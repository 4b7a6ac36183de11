"""The example's hybrid model: stepping token by token and taking the same tokens in windows agree.

Both runs round every layer's outputs to bf16 (relative 2^-8 each) from sums in other orders; two layers and the output
product leave differences of a few such roundings of the largest logit, which lies within six standard deviations."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_steps_and_windows_agree(cuda, cache):
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # an e4m3 cache turns a bf16 rounding into one of e4m3's (2^-4) for the values on its boundaries
    assert example.main(["--prompt", "130", "--tokens", "9", "--cache", cache]) <= 6 * 4 * 2 ** -8 * (2 if cache == "e4m3" else 1)
