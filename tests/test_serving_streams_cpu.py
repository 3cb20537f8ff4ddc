"""Where the memory of a call on another stream comes from, on a machine
without a GPU: the binding runs against a library and streams that only record
what they are asked for."""
import contextlib
import types

import pytest
import torch

from q4_weight_only_gb300 import serving


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Block:
    """What torch.empty gives: the stream it was made under, and those that
    were told of it."""

    def __init__(self, shape, under):
        self.shape, self.under, self.told = shape, under, []

    def data_ptr(self):
        return 1 << 20

    def numel(self):
        return 1 << 20

    def record_stream(self, s):
        self.told.append(s.cuda_stream)


@pytest.fixture
def blocks(monkeypatch):
    made, current = [], [0]

    @contextlib.contextmanager
    def under(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def empty(shape, dtype=None, device=None):
        made.append(Block(shape, current[-1]))
        return made[-1]

    class Torch(types.ModuleType):
        def __getattr__(self, name):
            return getattr(torch, name)

    fake = Torch("torch")
    fake.empty = empty
    fake._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda device: current[-1])
    fake.cuda = types.SimpleNamespace(current_device=lambda: -1, stream=under, Stream=Stream, ExternalStream=Stream,
                                      current_stream=lambda device=None: Stream(current[-1]))
    ok = types.SimpleNamespace(q4_0_kv_append=lambda *a: 0, q4_0_attention=lambda *a: 0,
                               q4_0_token_logprobs=lambda *a: 0)
    monkeypatch.setattr(serving, "torch", fake)
    monkeypatch.setattr(serving, "lib", lambda: ok)
    monkeypatch.setattr(serving, "_ws_bytes", lambda *a: 4096)
    return made


def calls():
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(2, 1, 8, 64, dtype=torch.bfloat16)
    batch = (k, k.clone(), ints(1)[None], ints(0, 1), ints(1))
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    return {
        "kv_append": lambda s: serving.kv_append(torch.zeros(1, 4 * 64), torch.zeros(8, 64), *batch, q_heads=2, stream=s),
        "attention": lambda s: serving.attention(q, *batch, max_q_len=1, stream=s),
        "token_logprobs": lambda s: serving.token_logprobs(torch.zeros(1, 9), torch.zeros(1, dtype=torch.int64), top=2,
                                                           stream=s),
    }


@pytest.mark.parametrize("what,results,scratch", [("kv_append", 1, 0), ("attention", 1, 1), ("token_logprobs", 4, 0)])
@pytest.mark.parametrize("stream", [Stream(5), 5])
def test_memory_of_the_stream_that_writes_it(blocks, what, results, scratch, stream):
    calls()[what](stream)
    assert len(blocks) == results + scratch
    assert [b.under for b in blocks] == [5] * len(blocks)
    # results are used on the current stream afterwards
    assert [b.told for b in blocks[:results]] == [[0]] * results


@pytest.mark.parametrize("what", ["kv_append", "attention", "token_logprobs"])
@pytest.mark.parametrize("stream", [None, 0, Stream(0)])
def test_the_current_stream_needs_no_more(blocks, what, stream):
    calls()[what](stream)
    assert blocks and all(b.under == 0 and not b.told for b in blocks)
