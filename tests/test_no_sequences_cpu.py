"""A batch without a sequence: its arrays have no elements, and a tensor
without elements has no address (no GPU: such a call ends after the checks)."""
import pytest

from test_serving_cpu import append, attention, cache, lib  # noqa: F401


@pytest.mark.parametrize("call", [append, attention])
def test_empty_arrays(lib, call):  # noqa: F811
    assert call(lib, cache(sequences=0, page_table=0, kv_len=0)) == 0
    assert call(lib, cache(sequences=0, page_table=0, kv_len=0, q_start=0)) == 0
    assert call(lib, cache(sequences=1, page_table=0)) == -1
