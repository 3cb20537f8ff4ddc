"""The operators around the matmuls on a machine without a GPU: their entry
points refuse bad arguments before any CUDA call, and the binding checks its
tensors."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
GOOD = 1 << 20           # never dereferenced: validation fails first

FIELDS = ["k", "v", "k_page_stride", "k_head_stride", "k_token_stride", "v_page_stride", "v_head_stride",
          "v_token_stride", "pages", "page_size", "kv_heads", "head_dim", "page_table", "table_stride", "table_width",
          "q_start", "kv_len", "sequences"]


@pytest.fixture(scope="module")
def lib():
    from q4_weight_only_gb300 import _lib, build
    build.build()
    return _lib.lib()


def cache(**change):
    c = dict(k=GOOD, v=GOOD, k_page_stride=16 * 2 * 64, k_head_stride=16 * 64, k_token_stride=64,
             v_page_stride=16 * 2 * 64, v_head_stride=16 * 64, v_token_stride=64, pages=10, page_size=16, kv_heads=2,
             head_dim=64, page_table=GOOD, table_stride=5, table_width=5, q_start=GOOD, kv_len=GOOD, sequences=3)
    c.update(change)
    return (ctypes.c_int64 * len(FIELDS))(*(c[f] for f in FIELDS))


def append(lib, c=None, **change):
    a = dict(qkv=GOOD, type=0, stride=8 * 64, rows=3, q_heads=4, cos_sin=GOOD, positions=9, rot=64, interleaved=0,
             row_positions=None, out=GOOD)
    a.update(change)
    return lib.q4_0_kv_append(*a.values(), c if c is not None else cache(), None)


def attention(lib, c=None, **change):
    a = dict(q=GOOD, row=4 * 64, head=64, out=GOOD, type=1, lse=None, rows=3, q_heads=4, max_q_len=1, scale=0.1,
             window=0, sinks=0, cache=c if c is not None else cache(), workspace=GOOD, bytes=1 << 40, stream=None)
    a.update(change)
    return lib.q4_0_attention(*a.values())


def logprobs(lib, **change):
    a = dict(logits=GOOD, type=0, stride=100, rows=4, vocab=100, tokens=GOOD, top=3, logprob=GOOD, entropy=GOOD,
             top_logprob=GOOD, top_ids=GOOD, stream=None)
    a.update(change)
    return lib.q4_0_token_logprobs(*a.values())


BAD_CACHES = [dict(k=0), dict(v=0), dict(page_table=0), dict(q_start=0), dict(kv_len=0), dict(k=GOOD + 8),
              dict(v=GOOD + 2), dict(page_table=GOOD + 2), dict(pages=0), dict(page_size=0), dict(kv_heads=0),
              dict(head_dim=0), dict(sequences=-1), dict(table_width=0), dict(table_stride=4),
              dict(k_page_stride=1001), dict(v_token_stride=60), dict(k_head_stride=-64)]
HUGE_CACHES = [dict(pages=1 << 31), dict(page_size=1 << 21, table_width=1, table_stride=1), dict(kv_heads=2000),
               dict(head_dim=2048), dict(sequences=1 << 21), dict(table_width=1 << 28, table_stride=1 << 28),
               dict(k_page_stride=1 << 39)]


@pytest.mark.parametrize("call", [append, attention])
def test_caches_are_checked(lib, call):
    for change in BAD_CACHES:
        assert call(lib, cache(**change)) == -1, change
    for change in HUGE_CACHES:
        assert call(lib, cache(**change)) == -2, change
    assert call(lib, rows=0) == 0
    assert call(lib, cache(sequences=0)) == 0


def test_append_arguments(lib):
    for change in (dict(qkv=None), dict(cos_sin=None), dict(out=None), dict(type=2), dict(rows=-1), dict(q_heads=0),
                   dict(positions=0), dict(rot=72), dict(rot=12), dict(rot=-8), dict(stride=8 * 64 - 4),
                   dict(stride=8 * 64 + 2), dict(qkv=GOOD + 4), dict(out=GOOD + 8), dict(cos_sin=GOOD + 4),
                   dict(row_positions=GOOD + 1), dict(type=1, stride=8 * 64 + 4)):
        assert append(lib, **change) == -1, change
    assert append(lib, cache(head_dim=68, k_token_stride=72, v_token_stride=72), stride=8 * 68, rot=64) == -1
    for change in (dict(rows=1 << 31), dict(q_heads=5000, stride=1 << 30), dict(positions=1 << 31)):
        assert append(lib, **change) == -2, change


def test_attention_arguments(lib):
    nan = float("nan")
    for change in (dict(q=None), dict(out=None), dict(type=3), dict(window=-1), dict(sinks=-1), dict(scale=0.0),
                   dict(scale=-1.0), dict(scale=nan), dict(q_heads=3), dict(max_q_len=0), dict(rows=-1),
                   dict(row=4 * 64 + 4), dict(head=60), dict(head=0), dict(q=GOOD + 8), dict(out=GOOD + 16),
                   dict(lse=GOOD + 2)):
        assert attention(lib, **change) == -1, change
    for c in (dict(head_dim=96), dict(page_size=12), dict(head_dim=256)):
        assert attention(lib, cache(**c)) == -2, c
    assert attention(lib, q_heads=2 * 129) == -2
    need = lib.q4_0_attention_workspace_bytes(3, 4, 2, 64, 1)
    if need:                                       # a device is needed to know the workspace
        assert attention(lib, workspace=None, bytes=0) == -5
        assert attention(lib, bytes=need - 1) == -5
        assert attention(lib, workspace=GOOD + 128) == -5
    for bad in ((0, 4, 2, 64, 1), (3, 4, 3, 64, 1), (3, 4, 2, 80, 1), (3, 4, 2, 64, 0)):
        assert lib.q4_0_attention_workspace_bytes(*bad) == 0


def test_logprobs_arguments(lib):
    for change in (dict(logits=None), dict(type=2), dict(stride=99), dict(rows=-1), dict(vocab=0), dict(top=-1),
                   dict(top=101, vocab=100), dict(entropy=None), dict(logprob=None), dict(top_logprob=None),
                   dict(top_ids=None), dict(logits=GOOD + 2), dict(type=1, logits=GOOD + 1), dict(tokens=GOOD + 4),
                   dict(top_ids=GOOD + 4), dict(entropy=GOOD + 2)):
        assert logprobs(lib, **change) == -1, change
    for change in (dict(top=33), dict(rows=1 << 31), dict(vocab=1 << 31, stride=1 << 31)):
        assert logprobs(lib, **change) == -2, change
    assert logprobs(lib, rows=0) == 0


def test_status_text(lib):
    assert b"index" in lib.q4_0_status_string(-6)


def test_binding_refuses_host_tensors(monkeypatch):
    import q4_weight_only_gb300 as q4
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    t = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        q4.token_logprobs(t, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        q4.token_logprobs(t.double(), torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError):
        q4.kv_append(t.half(), t, t, t, t, t, t, q_heads=1)
    with pytest.raises(ValueError):
        q4.attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16), t, t, t, t, t, max_q_len=1)
    with pytest.raises(TypeError):
        q4.attention(None, t, t, t, t, t, max_q_len=1)
