"""A block whose fp32 scale underflows to 0 is one of zeros to the oracle too:
no infinite quotient becomes a code."""
import numpy as np

import oracle


def test_codes_of_a_block_without_a_scale():
    w = np.zeros((4, 32), dtype=np.float32)
    least = np.float32(2.0 ** -149)
    for i, top in enumerate((1, -1, 4, -4)):
        w[i, 3], w[i, 9], w[i, 20], w[i, 31] = top * least, -least, least, -top * least
    q = oracle.get().quantize(w)
    assert (q[:, 2:] == 0x88).all()
    # the scale's sign is that of the largest element, turned
    assert [int(x) for x in q[:, :2].copy().view(np.uint16)[:, 0]] == [0x8000, 0, 0x8000, 0]


def test_the_least_scale_still_has_codes():
    w = np.zeros((1, 32), dtype=np.float32)
    w[0, 3], w[0, 4] = np.float32(2.0 ** -146), np.float32(-(2.0 ** -147))
    q = oracle.get().quantize(w)
    assert q[0, 2 + 3] & 15 == 0 and q[0, 2 + 4] & 15 == 12
