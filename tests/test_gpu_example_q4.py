"""examples/serve_layer.py with its cache in 4 bits: it runs, and decoding token
by token stays near the whole sequences at once (GPU).

Both runs append the same tokens, but from activations that decoding and
prefill round apart, so here and there an element falls on another code: its
key or value then differs by d, an eighth of its block's largest element.  An
output is a weighted mean of values, and a logit a sum of 5120 products of
outputs: for every element of every block to differ by all of d would be 1/8
of the attention's part of a logit, of size 1.4; a code that differs is the
exception, one in hundreds, and half the size of all is ample.
"""
import importlib.util
import os

import pytest

from gpu_common import lib

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")


@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 4)])
def test_a_layer_with_its_cache_in_4_bits(window, sinks):
    lib()
    spec = importlib.util.spec_from_file_location("serve_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(steps=4, window=window, sinks=sinks, verbose=False, cache_kind="q4") < 0.5 * 1.4 / 8
