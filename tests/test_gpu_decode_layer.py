"""examples/decode_layer.py: the serving calls together, prompts in one chunk and then tokens one at a time from a
CUDA graph, against the layer in 32 bits over an unquantised cache.

The two differ by the cache's rounding. A code is off by at most half a step: in e4m3 2^-4 of its value, evenly
spread (a relative error of 2^-4 / sqrt(3) in the mean square), in int8 1/2 of 1/127 of its block's largest value.
Values' errors are averaged with the values themselves, so the branch is off by about as much, and keys' errors
move the weights by a comparable amount: 2 * 2^-4 bounds either with room for both."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["e4m3", "int8"])
def test_decode_layer(cache):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst = example.main(steps=6, cache=cache)
    assert len(worst) == 7 and max(worst) < 2 * 2.0 ** -4
