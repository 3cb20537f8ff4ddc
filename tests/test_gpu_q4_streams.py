"""The operators of the 4-bit cache on another stream than the current one,
beside work that is still queued on it (GPU): neither's memory is the
other's."""
import pytest
import torch

from gpu_common import lib
from serving_ref_q4 import Batch

pytestmark = pytest.mark.gpu


def append(q4):
    b = Batch([1, 90], [500, 300], 16, 2, 128, seed=26)
    dev = b.cuda()
    qkv, cs = torch.randn(b.rows, 14 * 128, device="cuda"), torch.randn(512, 128, device="cuda")
    return lambda s: (q4.kv_append_q4(qkv, cs, *dev, q_heads=10, stream=s),), [b.rows * 10 * 128 * 2]


def read(q4):
    b = Batch([1, 90], [500, 300], 16, 2, 128, seed=27).write_tokens()
    dev = b.cuda()
    return lambda s: q4.kv_read_q4(*dev, rows=b.rows, stream=s), [b.rows * 2 * 128 * 2] * 2


def attend(q4):
    b = Batch([1, 90], [500, 300], 16, 2, 128, seed=28).write_tokens()
    dev = b.cuda()
    q = torch.randn(b.rows, 10, 128, device="cuda").bfloat16()
    sizes = [b.rows * 10 * 128 * 4, q4.attention_q4_workspace_bytes(b.rows, 10, 2, 128, 90)]
    return lambda s: (q4.attention_q4(q, *dev, max_q_len=90, out_dtype=torch.float32, stream=s),), sizes


@pytest.mark.parametrize("make", [append, read, attend])
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


@pytest.mark.parametrize("make", [append, read, attend])
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
    read_ = [g.clone() for g in got]
    del got
    with torch.cuda.stream(side):
        for _ in range(3):
            for w in want:
                torch.empty_like(w).fill_(1)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(read_, want))


def test_two_captured_graphs_with_workspaces_of_their_own_and_one_shared():
    """Two graphs replayed in turn: each with its own workspace, and both
    with one that their order on the stream keeps apart."""
    q4 = lib()
    batches = [Batch([1] * 4, [700, 90, 333, 64 + i], 16, 2, 128, seed=30 + i).write_tokens() for i in range(2)]
    qs = [torch.randn(4, 10, 128, device="cuda").bfloat16() for _ in batches]
    need = q4.attention_q4_workspace_bytes(4, 10, 2, 128, 1)
    for shared in (False, True):
        one = torch.empty(need, dtype=torch.uint8, device="cuda")
        graphs, outs, wants = [], [], []
        for b, q in zip(batches, qs):
            dev = b.cuda()
            ws = one if shared else torch.empty(need, dtype=torch.uint8, device="cuda")
            out = torch.empty(4, 10, 128, device="cuda")
            def call():
                q4.attention_q4(q, *dev, max_q_len=1, out=out, out_dtype=torch.float32, workspace=ws)

            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                call()
            torch.cuda.synchronize()
            wants.append(out.clone())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                call()
            graphs.append(graph), outs.append(out)
        for o in outs:
            o.zero_()
        for _ in range(3):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, wants))
    assert q4.device_error() == q4.OK
