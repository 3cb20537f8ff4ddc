"""attention_q4 where a row's scale leaves fp32's or binary16's comfort (GPU):
scores up to 2^30, and queries and scales whose product underflows.

Four keys of n have the largest score, the rest next to no weight (scores of
2^10 and more) or the same as far as fp32 can tell (products that underflow), so
the output is a mean of values: to within their rounding to binary16, 2^-11
each, that of the equal weights, which are powers of two times a common factor
(another 2^-11), and 2^-16 for fp32 sums.
"""
import math

import pytest
import torch

from gpu_common import lib
from serving_ref_q4 import Batch

pytestmark = pytest.mark.gpu


def batch(new, dim, best):
    """Keys with 1 in their first element at `best`, else 7/8."""
    b = Batch([new, new], [200, 300], 16, 1, dim, seed=4)
    b.tokens = []
    for s, n in enumerate(b.kv):
        k = torch.zeros(n, 1, dim)
        k[:, :, 0], k[:, :, 1] = 7 / 8, 1.0
        k[best, :, 0] = 1.0
        b.tokens.append(b.put(s, k, torch.randn(n, 1, dim, generator=b.g)))
        assert torch.equal(b.tokens[-1][0], k.double())
    return b


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 60])
@pytest.mark.parametrize("size", [10, 20.3, 25.99, 26.01, 30])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_large_scores(size, new, dim, sign):
    """c s of 2^size (times 7/8 where it is the lesser of two that counts)."""
    q4, best = lib(), [0, 3, 64, 130]
    b = batch(new, dim, best)
    q = torch.zeros(b.rows, 4, dim)
    q[..., 0] = sign
    scale = 2 ** size * math.log(2)
    lse = torch.empty(b.rows, 4, device="cuda")
    out = q4.attention_q4(q.bfloat16().cuda(), *b.cuda(), max_q_len=new, scale=scale, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    for row in range(b.rows):
        s, pos = row // new, b.kv[row // new] - new + row % new
        v = b.tokens[s][1][:pos + 1, 0].cuda()
        count = len(best) if sign > 0 else pos + 1 - len(best)
        assert pos >= max(best)
        mine = v[best] if sign > 0 else v[[j for j in range(pos + 1) if j not in best]]
        tol = (2 * 2 ** -11 + 2 ** -16) * mine.abs().mean(0) + 2 ** -25
        assert ((out[row].double() - mine.mean(0)).abs() <= tol).all()
        want = (scale if sign > 0 else -scale * 7 / 8) + math.log(count)
        assert ((lse[row].double() - want).abs() <= 2 ** -20 * abs(want)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("q_size,scale", [(1e-30, 1e-30), (1e-38, 1e-20), (1.0, 1e-44)])
def test_products_that_underflow(q_size, scale, new, dim):
    """Scores of next to nothing: every key that is seen counts the same, and
    what is not seen does not."""
    q4 = lib()
    b = batch(new, dim, [0, 3])
    q = (torch.randn(b.rows, 4, dim, generator=torch.Generator().manual_seed(6)) * q_size).bfloat16()
    lse = torch.empty(b.rows, 4, device="cuda")
    out = q4.attention_q4(q.cuda(), *b.cuda(), max_q_len=new, scale=scale, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    for row in range(b.rows):
        s, pos = row // new, b.kv[row // new] - new + row % new
        v = b.tokens[s][1][:pos + 1, 0].cuda()
        tol = (2 * 2 ** -11 + 2 ** -16) * v.abs().mean(0) + 2 ** -25
        assert ((out[row].double() - v.mean(0)).abs() <= tol).all()
        assert ((lse[row].double() - math.log(pos + 1)).abs() <= 2 ** -16).all()
