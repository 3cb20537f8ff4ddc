"""A sequence's rows of q4_0_attention depend on that sequence only: not on the
queries of others, nor on what kernels that ran before left behind (GPU).  Bits are compared: the split of the work follows the lengths,
which are the same."""
import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu

HEADS = [(40, 8, 128), (24, 4, 64), (28, 4, 128), (9, 3, 128)]   # 128 is no multiple of 5, 6, 7, 3


def attend(q4, b, q, window, sinks):
    return q4.attention(q, *b.dev, max_q_len=max(b.new), window=window, sinks=sinks, out_dtype=torch.float32)


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5)])
def test_same_bits_after_other_kernels(q_heads, kv_heads, dim, window, sinks):
    q4 = lib()
    b = ref.Batch([700, 1, 333, 60], [1500, 900, 333, 2000], 32, kv_heads, dim, seed=23).write_tokens()
    b.cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(b.rows, q_heads, dim, generator=g, device="cuda").bfloat16()
    want = attend(q4, b, q, window, sinks)
    for size in (1e-3, 1.0, 30.0, 1e4):
        # every SM's shared memory holds these afterwards
        logits = (torch.randn(608, 65536, generator=g, device="cuda") * size).bfloat16()
        q4.token_logprobs(logits, torch.zeros(608, dtype=torch.int64, device="cuda"))
        attend(q4, b, (torch.randn(b.rows, q_heads, dim, generator=g, device="cuda") * size).bfloat16(), window, sinks)
        assert torch.equal(attend(q4, b, q, window, sinks), want), size
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("new,kv", [([60, 70], [400, 300]), ([1, 1, 1, 1], [900, 700, 500, 300]),
                                    ([300, 5, 44], [300, 800, 600])])
def test_other_sequences_queries_do_not_matter(q_heads, kv_heads, dim, new, kv):
    q4 = lib()
    b = ref.Batch(new, kv, 16, kv_heads, dim, seed=24).write_tokens()
    b.cuda()
    q = torch.randn(b.rows, q_heads, dim, device="cuda").bfloat16()
    want = attend(q4, b, q, 0, 0)
    for s in range(len(new)):
        lo, hi = int(b.q_start[s]), int(b.q_start[s + 1])
        other = (torch.randn(b.rows, q_heads, dim, device="cuda") * 100).bfloat16()
        other[lo:hi] = q[lo:hi]
        assert torch.equal(attend(q4, b, other, 0, 0)[lo:hi], want[lo:hi]), s
    assert q4.device_error() == q4.OK
