"""attention_q4 over long caches in which one key outweighs each of the others
by far, and all the others together count (GPU).

The first token's score is 25.6 above the others' in log2; its value is 0 and
theirs are 1, so a row that sees n others gives M / (1 + M), M = n 2^-25.6, and
its logarithm is 25.6 log 2 + log(1 + M).  Pages repeat: the cache is two pages
whatever the length.

Tolerance.  A weight is rounded to binary16 in a unit 2^7 above the weight of
the largest: 2^-11 of each, or 2^-32 of the largest below the normal range.
Sums of n terms in fp32, of which the sequential part of each of 64 partial
sums (16 of a tcgen05 row: four chains of 32 pairs a tile, of which one starts
from the total) is n / 64 (n / 16) additions: 2^-24 n / 16 of the total.
"""
import math

import pytest
import torch

import serving_ref_q4 as ref4
from gpu_common import lib

pytestmark = pytest.mark.gpu
ABOVE = 25.6
PAGE = 64


def run(dim, sequences, new, tokens, group):
    q4 = lib()
    k, v = torch.zeros(2, 1, PAGE, dim), torch.ones(2, 1, PAGE, dim)
    k[0, 0, 0, 0], v[0, 0, 0] = 1.0, 0.0
    cache = q4.kv_cache_q4(2, 1, PAGE, dim)
    for at, x in ((0, k), (2, v)):
        for t, part in zip(cache[at:at + 2], ref4.blocks(x)):
            t.copy_(part.cuda())
    table = torch.ones(sequences, -(-tokens // PAGE), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    starts = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * new
    lengths = torch.full((sequences,), tokens, dtype=torch.int32, device="cuda")
    q = torch.zeros(sequences * new, group, dim, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    lse = torch.empty(sequences * new, group, device="cuda")
    out = q4.attention_q4(q, cache, table, starts, lengths, max_q_len=new, scale=ABOVE * math.log(2),
                          out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    others = (tokens - new + torch.arange(new, dtype=torch.float64, device="cuda")).repeat(sequences)[:, None]
    mass = others * 2 ** -ABOVE
    want, want_lse = mass / (1 + mass), ABOVE * math.log(2) + torch.log1p(mass)
    sums = tokens / 16 * 2 ** -24
    tol = (mass * 2 ** -11 + tokens * 2 ** -32) / (1 + mass) + want * (sums + 2 ** -16)
    off = (out.double() - want[..., None]).abs()
    assert (off <= tol[..., None]).all(), (off / tol[..., None]).max()
    assert ((lse.double() - want_lse).abs() <= sums + 2 ** -20 * (1 + want_lse)).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [8, 16])
def test_single_tokens(dim, group):
    """Enough sequences that each is whole in one block of threads."""
    run(dim, 304, 1, 1 << 20, group)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("new", [8, 32])
def test_prompts(dim, new):
    """64 and 256 rows: an item of one tile and of two."""
    run(dim, 152, new, 1 << 18, 8)
