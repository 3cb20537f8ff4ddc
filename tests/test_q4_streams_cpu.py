"""Where the memory of a 4-bit cache's calls on another stream comes from, on
a machine without a GPU: as test_serving_streams_cpu.py, whose recording
library and streams it uses."""
import types

import pytest
import torch

from q4_weight_only_gb300 import serving
from test_serving_streams_cpu import Stream, blocks  # noqa: F401


@pytest.fixture
def made(blocks, monkeypatch):  # noqa: F811
    ok = types.SimpleNamespace(q4_0_kv_append_q4=lambda *a: 0, q4_0_kv_read_q4=lambda *a: 0,
                               q4_0_attention_q4=lambda *a: 0)
    monkeypatch.setattr(serving, "lib", lambda: ok)
    return blocks


def calls():
    ints = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    codes, scales = torch.zeros(2, 1, 8, 32, dtype=torch.uint8), torch.zeros(2, 1, 8, 2, dtype=torch.float16)
    batch = ((codes, scales, codes.clone(), scales.clone()), ints(1)[None], ints(0, 1), ints(1))
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    return {
        "append": lambda s: serving.kv_append_q4(torch.zeros(1, 4 * 64), torch.zeros(8, 64), *batch, q_heads=2,
                                                 stream=s),
        "read": lambda s: serving.kv_read_q4(*batch, rows=1, stream=s),
        "attention": lambda s: serving.attention_q4(q, *batch, max_q_len=1, stream=s),
    }


@pytest.mark.parametrize("what,results,scratch", [("append", 1, 0), ("read", 2, 0), ("attention", 1, 1)])
@pytest.mark.parametrize("stream", [Stream(5), 5])
def test_memory_of_the_stream_that_writes_it(made, what, results, scratch, stream):
    calls()[what](stream)
    assert len(made) == results + scratch
    assert [b.under for b in made] == [5] * len(made)
    assert [b.told for b in made[:results]] == [[0]] * results   # results are used on the current stream afterwards


@pytest.mark.parametrize("what", ["append", "read", "attention"])
@pytest.mark.parametrize("stream", [None, 0, Stream(0)])
def test_the_current_stream_needs_no_more(made, what, stream):
    calls()[what](stream)
    assert made and all(b.under == 0 and not b.told for b in made)
