"""q4_0_attention on scores whose products with log2 e are rounded by more than
an exponent holds (GPU).

Queries and keys have one element each, whose products are exact in fp32, so
scores differ by exactly 0 or by so much that only the largest counts.
Tolerance as for other attention outputs, without the scores' part: 2^-8 +
2^-16 of the mean of |v|; the logarithm, 2^-22 of its size (the scale's, its
product's and log2 e's rounding, and two of the result).
"""
import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new,kv", [([1], [1]), ([1], [1000]), ([1, 300, 90], [3000, 300, 700])])
@pytest.mark.parametrize("exponent", [22, 30, 31, 36, 50, 100])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("distinct", [False, True])
def test_scores_far_from_zero(dim, new, kv, exponent, sign, distinct):
    q4 = lib()
    b = ref.Batch(new, kv, 16, 2, dim, seed=25).write_tokens()
    heads, group = 6, 3
    # the score of key j is sign * 2^exponent * (128 + j mod 101) / 128: 2^(exponent - 7) apart at least
    for s, n in enumerate(kv):
        k, v = b.tokens[s]
        k.zero_()
        step = torch.arange(n) % 101 if distinct else torch.zeros(n)
        k[:, :, 5] = ((128 + step) / 128 * 2.0 ** (exponent // 2))[:, None].bfloat16()
        b.put(s, k, v)
    b.cuda()
    q = torch.zeros(b.rows, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[:, :, 5] = sign * 2.0 ** (exponent - exponent // 2)
    lse = torch.empty(b.rows, heads, device="cuda")
    out = q4.attention(q, *b.dev, max_q_len=max(new), scale=1.0, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    row = 0
    for s, (n, length) in enumerate(zip(new, kv)):
        k, v = (t.double().repeat_interleave(group, 1).cuda() for t in b.tokens[s])
        seen = torch.arange(length, device="cuda") <= (length - n + torch.arange(n, device="cuda"))[:, None]
        score = torch.einsum("ih,jh->hij", q[row:row + n, :, 5].double(), k[:, :, 5])
        score = score.masked_fill(~seen, -torch.inf)
        p = score.softmax(-1)
        want, weight = torch.einsum("hij,jhd->ihd", p, v), torch.einsum("hij,jhd->ihd", p, v.abs())
        got = out[row:row + n].double()
        assert ((got - want).abs() <= (2 ** -8 + 2 ** -16) * weight).all(), (got - want).abs().max()
        want = score.logsumexp(-1).T
        assert ((lse[row:row + n].double() - want).abs() <= 2 ** -22 * (want.abs() + 16)).all()
        row += n
