"""q4_0_kv_append without a rotation: what it asks of the table (no GPU: a
call of no rows ends after the checks)."""
from test_serving_cpu import GOOD, append, lib  # noqa: F401


def test_no_table_is_needed(lib):  # noqa: F811
    for change in (dict(cos_sin=None, positions=0), dict(cos_sin=None, positions=1), dict(cos_sin=GOOD, positions=0)):
        assert append(lib, rows=0, rot=0, **change) == 0, change
    assert append(lib, rows=0, rot=0, positions=-1) == -1
    assert append(lib, rows=0, rot=8, positions=0) == -1
    assert append(lib, rows=0, rot=8, cos_sin=None) == -1
