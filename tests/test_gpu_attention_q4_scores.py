"""Scores of attention_q4's sequences of few rows (GPU): keys are exact there,
and every sum is one of fp32.

A row with a single key has the score as its logarithm of the softmax sum, to
within the rounding of the logarithm itself.  Tolerance of a score: a block's
dot product is sum_i q_i code_i - 8 sum_i q_i, 33 terms whose partial sums are
at most 15 sum_i |q_i|, each addition off by at most a step, 2^-23, of that
(tensor cores cut off); the blocks' scales and sums add a few roundings of the
same size.  So e = scale (33 + blocks) 2^-23 sum_b |d_b| 15 sum_{i in b} |q_i|.
The unit that undoes the query's scaling, the logarithm of 2 and their products
are 2^-21 of the score, the logarithm of a power of two 2^-20.
"""
import math

import pytest
import torch

import serving_ref as ref
from gpu_common import lib
from serving_ref_q4 import Batch

pytestmark = pytest.mark.gpu

# group 8: one tile of 8 rows; 16 and 12: two
HEADS = [(8, 1, 64), (8, 1, 128), (16, 1, 64), (16, 1, 128), (24, 2, 128), (10, 2, 64)]


def score_error(q, scales):
    """Per (token of the cache, query head): the tolerance of a score, without
    the softmax scale.  q [heads, dim], scales [tokens, kv_heads, blocks]."""
    heads, dim = q.shape
    kv_heads, blocks = scales.shape[-2:]
    d = scales.double().abs().repeat_interleave(heads // kv_heads, -2)
    size = q.double().abs().view(heads, blocks, 32).sum(-1)
    return (33 + blocks) * 2 ** -23 * 15 * (d * size).sum(-1)


def queries(rows, heads, dim, factor, seed):
    """One element of each is `factor` times the rest, in block 0."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(rows, heads, dim, generator=g)
    at = torch.randint(0, 32, (rows, heads, 1), generator=g)
    return q.scatter(2, at, q.gather(2, at).sign() * factor).bfloat16()


@pytest.mark.parametrize("factor", [1.0, 100.0, 1000.0, 20000.0])
@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
def test_a_dominant_element_costs_the_others_nothing(q_heads, kv_heads, dim, factor):
    """The dominant element meets a block of zeros: what remains is the other
    blocks' dot product, and their error."""
    q4, n = lib(), 64
    b = Batch([1] * n, [1] * n, 8, kv_heads, dim, seed=3)
    b.tokens, scales = [], []
    for s in range(n):
        k = torch.randn(1, kv_heads, dim, generator=b.g)
        k[..., :32] = 0
        b.tokens.append(b.put(s, k, torch.randn(1, kv_heads, dim, generator=b.g)))
        page, off = b.place(s, 0)
        scales.append(b.cache[1][page, :, off])
    q = queries(n, q_heads, dim, factor, 5)
    lse = torch.empty(n, q_heads, device="cuda")
    out = q4.attention_q4(q.cuda(), *b.cuda(), max_q_len=1, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    scale, group = dim ** -0.5, q_heads // kv_heads
    for s in range(n):
        k, v = (t[0].repeat_interleave(group, 0) for t in b.tokens[s])
        want = scale * (q[s].double() * k).sum(-1)
        tol = scale * score_error(q[s], scales[s]) + 2 ** -21 * want.abs() + 2 ** -20
        off = (lse[s].cpu().double() - want).abs()
        assert (off <= tol).all(), (s, (off / tol).max())
        # a single key is seen with certainty; values are rounded to binary16
        assert ((out[s].cpu().double() - v).abs() <= 2 ** -11 * v.abs() + 2 ** -25).all()


@pytest.mark.parametrize("factor", [1.0, 100.0, 1000.0])
@pytest.mark.parametrize("new", [1, 2])
@pytest.mark.parametrize("q_heads,kv_heads,dim", [(8, 1, 64), (8, 1, 128), (16, 2, 128), (5, 5, 64)])
def test_outputs_without_the_allowance_for_rounded_keys(q_heads, kv_heads, dim, new, factor):
    """Many keys: an error e in the scores moves a row's logarithm by e and its
    output by at most 2 e sum_j w_j |v_j|; rounding the weights and the values
    to binary16, 2^-11 each of the same and 2^-25 of the values' sizes."""
    q4, kv = lib(), [2, 33, 129, 700, 1025]
    b = Batch([new] * 5, kv, 16, kv_heads, dim, seed=9).write_tokens()
    q = queries(b.rows, q_heads, dim, factor, 7).cuda()
    scale = dim ** -0.5 / max(1.0, factor / 10)
    lse = torch.empty(b.rows, q_heads, device="cuda")
    out = q4.attention_q4(q, *b.cuda(), max_q_len=new, scale=scale, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    want, want_lse, weight, _ = ref.attention(q, b, 0, 0, scale)
    for row in range(b.rows):
        s = row // new
        j = torch.arange(kv[s])
        k_scales = b.cache[1][b.table[s, j // 16].long(), :, j % 16]
        e = scale * score_error(q[row].cpu(), k_scales).amax(0).cuda() + 2 ** -20
        largest = float(b.tokens[s][1].abs().max())
        tol = weight[row] * (2 * 2 ** -11 + 2 ** -16 + 2 * e[:, None]) + 2 ** -25 * (1 + kv[s] * largest)
        off = (out[row].double() - want[row]).abs()
        assert (off <= tol).all(), (row, (off / tol).max())
        at = want_lse[row]
        assert ((lse[row].double() - at).abs() <= e + 2 ** -20 * (1 + at.abs())).all()
        assert math.isfinite(float(at.abs().max()))
