"""Calls on another stream than the current one beside work that is still
queued on it (GPU): neither's memory is the other's."""
import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu


def append(q4):
    b = ref.Batch([1, 90], [500, 300], 16, 2, 128, seed=26)
    dev = b.cuda()
    qkv, cs = torch.randn(b.rows, 14 * 128, device="cuda"), torch.randn(512, 128, device="cuda")
    return lambda s: (q4.kv_append(qkv, cs, *dev, q_heads=10, stream=s),), [b.rows * 10 * 128 * 2]


def attend(q4):
    b = ref.Batch([1, 90], [500, 300], 16, 2, 128, seed=27).write_tokens()
    dev = b.cuda()
    q = torch.randn(b.rows, 10, 128, device="cuda").bfloat16()
    sizes = [b.rows * 10 * 128 * 4, q4.attention_workspace_bytes(b.rows, 10, 2, 128, 90)]
    return lambda s: (q4.attention(q, *dev, max_q_len=90, out_dtype=torch.float32, stream=s),), sizes


def score(q4):
    x, t = torch.randn(500, 9000, device="cuda"), torch.arange(500, device="cuda")
    return lambda s: q4.token_logprobs(x, t, top=20, stream=s), [500 * 4, 500 * 4, 500 * 20 * 4, 500 * 20 * 8]


@pytest.mark.parametrize("make", [append, attend, score])
@pytest.mark.parametrize("handle", [False, True])
def test_blocks_that_queued_work_still_uses(make, handle):
    q4 = lib()
    call, sizes = make(q4)
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(100_000_000)                     # some 50 ms
        kept = [b.clone() for b in blocks]
        for b in blocks:
            b.fill_(3)
        del b, blocks                                      # free for the current stream, in its order
        got = call(side.cuda_stream if handle else side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all((k == 7).all() for k in kept)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("make", [append, attend, score])
def test_results_outlive_their_last_use(make):
    """A result that is dropped while the current stream still reads it is not
    handed out again before that."""
    q4 = lib()
    call, _ = make(q4)
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    read = [g.clone() for g in got]
    del got
    with torch.cuda.stream(side):
        for _ in range(3):
            for w in want:
                torch.empty_like(w).fill_(1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read, want))
