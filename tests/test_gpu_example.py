"""examples/serve_layer.py: the operators and the matmuls as one served layer
(GPU).

Decoding token by token and running the whole sequences at once take other
kernels and other splits of the work for the same sums.  The layer's output
adds to a residual of size 1 with a spread of about 1.4 sqrt(5120) 0.02 a
logit; what differs is rounding of activations to bfloat16 (2^-8 a matmul
input, in four places) and the decode matmuls' 15-bit x, averaged over 5120
terms: well under 2^-8 * 4 * 2 = 0.03 of a logit's size, 2.
"""
import importlib.util
import os

import pytest

from gpu_common import lib

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")


@pytest.mark.parametrize("window,sinks", [(0, 0), (64, 4)])
def test_decoding_agrees_with_the_whole_sequences(window, sinks):
    lib()
    spec = importlib.util.spec_from_file_location("serve_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main(steps=4, window=window, sinks=sinks, verbose=False) < 0.06
