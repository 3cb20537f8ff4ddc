"""Python binding of the operators around the matmuls: kv_append, attention
and token_logprobs (argument marshalling only, see include/q4_0.h).

A paged cache is a pair of bfloat16 tensors [pages, kv_heads, page_size,
head_dim] in any memory order whose head_dim elements are adjacent (a
[pages, page_size, kv_heads, head_dim] cache is passed as its transpose(1,
2)).  A batch is described by three int32 device tensors: page_table
[sequences, max_pages], q_start [sequences + 1] (the rows of each sequence)
and kv_len [sequences] (its tokens in the cache, the new ones included).
They are read on the device only, so a captured CUDA graph follows them.
"""
import ctypes

import torch

from ._lib import Y_BF16, Y_F32, _check, _need, _stream, _workspace, _ws_bytes, lib

MAX_TOP = 32

_TYPES = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}


class _KvCache(ctypes.Structure):
    _fields_ = ([("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]
                + [(n, ctypes.c_int64) for n in ("k_page_stride", "k_head_stride", "k_token_stride", "v_page_stride",
                                                 "v_head_stride", "v_token_stride", "pages", "page_size", "kv_heads",
                                                 "head_dim")]
                + [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64),
                   ("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("sequences", ctypes.c_int64)])


def _strided(t, name, dtype, ndim):
    """As _need, but only the last dimension has to be contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a {ndim}-D tensor with adjacent elements in its last dimension")


def _same_device(*tensors):
    """Every tensor on the current device: the library launches there."""
    current = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != current:
            raise ValueError(f"every tensor must be on the current device (cuda:{current}), got {t.device}")


def _keep(stream, *tensors):
    """Memory made here for work on another stream than the current one is
    not handed out again before that work is done."""
    if stream is None:
        return
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    for t in tensors:
        if t is not None and s.cuda_stream != torch.cuda.current_stream().cuda_stream:
            t.record_stream(s)


def _cache(k_cache, v_cache, page_table, q_start, kv_len):
    _strided(k_cache, "k_cache", torch.bfloat16, 4)
    _strided(v_cache, "v_cache", torch.bfloat16, 4)
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    _strided(page_table, "page_table", torch.int32, 2)
    _need(q_start, "q_start", torch.int32, 1)
    _need(kv_len, "kv_len", torch.int32, 1)
    n = kv_len.shape[0]
    if q_start.shape[0] != n + 1 or page_table.shape[0] != n:
        raise ValueError("page_table, q_start and kv_len must be of sequences, sequences + 1 and sequences rows")
    _same_device(k_cache, v_cache, page_table, q_start, kv_len)
    pages, heads, size, dim = k_cache.shape
    # a dimension of one row has no stride to speak of
    stride = page_table.stride(0) if n > 1 else page_table.shape[1]
    return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.stride()[:3], *v_cache.stride()[:3], pages, size,
                    heads, dim, page_table.data_ptr(), stride, page_table.shape[1], q_start.data_ptr(),
                    kv_len.data_ptr(), n)


def _row_stride(t):
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def kv_append(qkv: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              page_table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, *, q_heads: int,
              interleaved: bool = False, positions: torch.Tensor = None, out: torch.Tensor = None,
              stream=None) -> torch.Tensor:
    """Rotate the queries and keys of qkv [rows, (q_heads + 2 kv_heads) *
    head_dim] (fp32 or bf16: query, key and value heads) by position, append
    keys and values to the cache in place, and return the queries, bf16
    [rows, q_heads, head_dim].

    cos_sin: fp32 [positions, rot], cosines then sines of the rot / 2 pairs
    (halves of the first rot elements, or neighbours when interleaved).
    positions: int32 [rows], the row of cos_sin to use instead of the
    position in the sequence."""
    _strided(qkv, "qkv", (torch.float32, torch.bfloat16), 2)
    _need(cos_sin, "cos_sin", torch.float32, 2)
    c = _cache(k_cache, v_cache, page_table, q_start, kv_len)
    rows = qkv.shape[0]
    if qkv.shape[1] != (q_heads + 2 * c.kv_heads) * c.head_dim:
        raise ValueError("qkv must be [rows, (q_heads + 2 * kv_heads) * head_dim]")
    if positions is not None:
        _need(positions, "positions", torch.int32, 1)
        if positions.shape[0] != rows:
            raise ValueError("positions must have one element per row")
    given = out
    if out is None:
        out = torch.empty((rows, q_heads, c.head_dim), dtype=torch.bfloat16, device=qkv.device)
    _need(out, "out", torch.bfloat16, 3)
    if tuple(out.shape) != (rows, q_heads, c.head_dim):
        raise ValueError("out must be [rows, q_heads, head_dim]")
    _same_device(qkv, cos_sin, positions, out)
    if rows == 0:
        return out
    _check(lib().q4_0_kv_append(qkv.data_ptr(), _TYPES[qkv.dtype], _row_stride(qkv), rows, q_heads,
                                cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)),
                                positions.data_ptr() if positions is not None else None, out.data_ptr(),
                                ctypes.byref(c), _stream(stream)), "q4_0_kv_append")
    if given is None:
        _keep(stream, out)
    return out


def attention_workspace_bytes(rows: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int) -> int:
    """Scratch of attention on the current device (0 for sizes it refuses)."""
    return _ws_bytes("q4_0_attention_workspace_bytes", rows, q_heads, kv_heads, head_dim, max_q_len)


def attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
              q_start: torch.Tensor, kv_len: torch.Tensor, *, max_q_len: int, scale: float = None, window: int = 0,
              sinks: int = 0, out: torch.Tensor = None, out_dtype=torch.bfloat16, lse: torch.Tensor = None,
              workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Causal attention of q [rows, q_heads, head_dim] (bf16, any strides of
    rows and heads) over the paged cache, the rows' own tokens included:
    [rows, q_heads, head_dim] of out_dtype (bf16 or fp32).

    max_q_len: the most new tokens of a sequence.  scale: head_dim ** -0.5
    when not given.  window, sinks: a row sees its latest `window` tokens (0:
    all) and the first `sinks`.  lse: fp32 [rows, q_heads] to receive the
    natural logarithms of the softmax sums."""
    if out_dtype not in _TYPES:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    _strided(q, "q", torch.bfloat16, 3)
    c = _cache(k_cache, v_cache, page_table, q_start, kv_len)
    rows, q_heads, dim = q.shape
    if dim != c.head_dim:
        raise ValueError("q and the cache must have the same head_dim")
    given = out
    if out is None:
        out = torch.empty((rows, q_heads, dim), dtype=out_dtype, device=q.device)
    _need(out, "out", out_dtype, 3)
    if tuple(out.shape) != (rows, q_heads, dim):
        raise ValueError("out must be [rows, q_heads, head_dim]")
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
        if tuple(lse.shape) != (rows, q_heads):
            raise ValueError("lse must be [rows, q_heads]")
    _same_device(q, out, lse, workspace)
    if rows == 0:
        return out
    ws, wsb = _workspace(attention_workspace_bytes(rows, q_heads, c.kv_heads, dim, max_q_len), q.device, workspace)
    _check(lib().q4_0_attention(q.data_ptr(), q.stride(0), q.stride(1), out.data_ptr(), _TYPES[out_dtype],
                                lse.data_ptr() if lse is not None else None, rows, q_heads, max_q_len,
                                dim ** -0.5 if scale is None else scale, window, sinks, ctypes.byref(c),
                                ws.data_ptr() if ws is not None else None, wsb, _stream(stream)), "q4_0_attention")
    _keep(stream, out if given is None else None, ws if workspace is None else None)
    return out


def token_logprobs_workspace_bytes(rows: int, vocab: int, top: int) -> int:
    """Scratch of token_logprobs on the current device."""
    return _ws_bytes("q4_0_token_logprobs_workspace_bytes", rows, vocab, top)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top: int = 0, workspace: torch.Tensor = None,
                   stream=None):
    """(logprob, entropy, top_logprob, top_ids) of logits [rows, vocab] (fp32
    or bf16): the log probability of tokens[row] (int64; negative: none, 0),
    the row's entropy in nats, and its `top` largest log probabilities with
    their ids ([rows, top], largest first, equal logits by lowest id)."""
    _strided(logits, "logits", (torch.float32, torch.bfloat16), 2)
    _need(tokens, "tokens", torch.int64, 1)
    rows, vocab = logits.shape
    if tokens.shape[0] != rows:
        raise ValueError("tokens must have one element per row of logits")
    _same_device(logits, tokens, workspace)
    dev = logits.device
    stats = torch.empty((2, rows), dtype=torch.float32, device=dev)
    top_logprob = torch.empty((rows, max(top, 0)), dtype=torch.float32, device=dev)
    top_ids = torch.empty((rows, max(top, 0)), dtype=torch.int64, device=dev)
    if rows == 0:
        return stats[0], stats[1], top_logprob, top_ids
    ws, wsb = _workspace(token_logprobs_workspace_bytes(rows, vocab, top), dev, workspace)
    _check(lib().q4_0_token_logprobs(logits.data_ptr(), _TYPES[logits.dtype], _row_stride(logits), rows, vocab,
                                     tokens.data_ptr(), top, stats[0].data_ptr(), stats[1].data_ptr(),
                                     top_logprob.data_ptr() if top else None, top_ids.data_ptr() if top else None,
                                     ws.data_ptr() if ws is not None else None, wsb, _stream(stream)),
           "q4_0_token_logprobs")
    _keep(stream, stats, top_logprob, top_ids, ws if workspace is None else None)
    return stats[0], stats[1], top_logprob, top_ids
