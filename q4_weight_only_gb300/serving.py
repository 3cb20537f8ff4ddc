"""Python binding of the operators around the matmuls: kv_append, attention
and token_logprobs, and kv_append_q4, kv_read_q4 and attention_q4 for a cache
in 4 bits (argument marshalling only, see include/q4_0.h).

A paged cache is a pair of bfloat16 tensors [pages, kv_heads, page_size,
head_dim] in any memory order whose head_dim elements are adjacent (a
[pages, page_size, kv_heads, head_dim] cache is passed as its transpose(1,
2)).  A batch is described by three int32 device tensors: page_table
[sequences, max_pages], q_start [sequences + 1] (the rows of each sequence)
and kv_len [sequences] (its tokens in the cache, the new ones included).
They are read on the device only, so a captured CUDA graph follows them.

A cache in 4 bits is a KVCacheQ4: codes uint8 [pages, kv_heads, page_size,
head_dim / 2] and scales float16 [pages, kv_heads, page_size, head_dim / 32] of
keys and of values, in any memory order of the outer dimensions as above
(kv_cache_q4 makes one).  An element is scale * (code - 8), in blocks of 32.

A call with `stream` reads its inputs and writes its results there: that
stream waits for whoever writes the inputs, and whoever reads the results
waits for it, both in the caller's hands.  Results and workspaces that are not
given are that stream's own memory.
"""
import struct
from typing import NamedTuple

import torch

from ._lib import Y_BF16, Y_F32, _check, _need, _ws_bytes, lib

MAX_TOP = 32

_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64
_F16, _U8 = torch.float16, torch.uint8
_TYPES = {_F32: Y_F32, _BF16: Y_BF16}

# q4_0_kv_cache: two pointers, six strides, four sizes, the table and its two
# sizes, two pointers and a size, all 64 bits
_KV_CACHE = struct.Struct("=18q")

# q4_0_kv_cache_q4: four pointers, twelve strides, four sizes and the batch
_KV_CACHE_Q4 = struct.Struct("=26q")


class KVCacheQ4(NamedTuple):
    """A paged cache in Q4_0 blocks."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


# The checks of a call run on every decode step and cost as much as its
# launches: each tensor gets one short test, and only a misfit goes on to the
# function that names what is wrong with it.

def _strided(t, name, dtypes, ndim):
    """As _need, but only the last dimension has to be contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != ndim or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must be a {ndim}-D tensor with adjacent elements in its last dimension")


def _misplaced(t, name, device):
    raise ValueError(f"{name} must be on the current device (cuda:{device}), where the call launches, got {t.device}")


def _plain(t, name, dtype, ndim, device):
    """A contiguous tensor of the current device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()
            and t.get_device() == device):
        _need(t, name, dtype, ndim)
        _misplaced(t, name, device)


def _rows(t, name, dtypes, ndim, device):
    """A tensor of the current device with adjacent last elements; its
    strides."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == ndim and t.get_device() == device:
        stride = t.stride()
        if stride[-1] == 1 or t.shape[-1] <= 1:
            return stride
    _strided(t, name, dtypes, ndim)
    _misplaced(t, name, device)


def _stream_of(stream, device):
    """The raw handle of `stream`, the current one when None."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _other(stream, device):
    """`stream` as a torch stream where it is not the current one, else None."""
    if stream is None or _stream_of(stream, device) == _stream_of(None, device):
        return None
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))


def _empty(shape, dtype, device, other, result=True):
    """Memory for a call on the stream `other` (None: the current one).  It
    comes from that stream's pool: a block of the current stream's may be in
    use by work that is still queued there.  A result goes back to its pool
    only after what the current stream does with it."""
    if other is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(other):
        t = torch.empty(shape, dtype=dtype, device=device)
    if result:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _scratch(nbytes, device, workspace, other):
    """The caller's workspace or one made here, or None where none is needed."""
    if workspace is not None:
        _plain(workspace, "workspace", torch.uint8, 1, device)
        if workspace.numel() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return _empty(nbytes, torch.uint8, device, other, result=False) if nbytes else None


def _cache(k_cache, v_cache, page_table, q_start, kv_len, device):
    """The q4_0_kv_cache of these tensors, packed, and its heads and head_dim."""
    ks = _rows(k_cache, "k_cache", (_BF16,), 4, device)
    vs = _rows(v_cache, "v_cache", (_BF16,), 4, device)
    ts = _rows(page_table, "page_table", (_I32,), 2, device)
    _plain(q_start, "q_start", _I32, 1, device)
    _plain(kv_len, "kv_len", _I32, 1, device)
    shape = k_cache.shape
    if shape != v_cache.shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    n = kv_len.shape[0]
    sequences, width = page_table.shape
    if q_start.shape[0] != n + 1 or sequences != n:
        raise ValueError("page_table, q_start and kv_len must be of sequences, sequences + 1 and sequences rows")
    pages, heads, size, dim = shape
    packed = _KV_CACHE.pack(k_cache.data_ptr(), v_cache.data_ptr(), ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], pages,
                            size, heads, dim, page_table.data_ptr(),
                            ts[0] if n > 1 else width,  # one row has no stride to speak of
                            width, q_start.data_ptr(), kv_len.data_ptr(), n)
    return packed, heads, dim


def kv_cache_q4(pages: int, kv_heads: int, page_size: int, head_dim: int, *, token_major: bool = False) -> KVCacheQ4:
    """A cache of `pages` pages on the current device, all zeros; token_major:
    a page holds [page_size, kv_heads, ...] instead of [kv_heads, page_size,
    ...] (the tensors' shapes are the same)."""
    if head_dim < 32 or head_dim % 32:
        raise ValueError("head_dim must be a positive multiple of 32")

    def make(width, dtype):
        if token_major:
            return torch.zeros((pages, page_size, kv_heads, width), dtype=dtype, device="cuda").transpose(1, 2)
        return torch.zeros((pages, kv_heads, page_size, width), dtype=dtype, device="cuda")

    return KVCacheQ4(*(make(*kind) for kind in ((head_dim // 2, _U8), (head_dim // 32, _F16)) * 2))


_BYTE, _HALF = (_U8,), (_F16,)


def _cache_q4(cache, page_table, q_start, kv_len, device):
    """The q4_0_kv_cache_q4 of these tensors, packed, and its heads and head_dim."""
    k, k_scale, v, v_scale = cache
    ks, vs = _rows(k, "k_codes", _BYTE, 4, device), _rows(v, "v_codes", _BYTE, 4, device)
    kss, vss = _rows(k_scale, "k_scales", _HALF, 4, device), _rows(v_scale, "v_scales", _HALF, 4, device)
    ts = _rows(page_table, "page_table", (_I32,), 2, device)
    _plain(q_start, "q_start", _I32, 1, device)
    _plain(kv_len, "kv_len", _I32, 1, device)
    shape, scales = k.shape, k_scale.shape
    if shape != v.shape or scales != v_scale.shape:
        raise ValueError("keys and values must have the same shapes")
    pages, heads, size, half = shape
    if half % 16 or scales != (pages, heads, size, half // 16):
        raise ValueError("codes must be [pages, kv_heads, page_size, head_dim / 2] and scales [pages, kv_heads, "
                         "page_size, head_dim / 32]")
    n = kv_len.shape[0]
    sequences, width = page_table.shape
    if q_start.shape[0] != n + 1 or sequences != n:
        raise ValueError("page_table, q_start and kv_len must be of sequences, sequences + 1 and sequences rows")
    packed = _KV_CACHE_Q4.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                               *ks[:3], *vs[:3], *kss[:3], *vss[:3], pages, size, heads, 2 * half,
                               page_table.data_ptr(), ts[0] if n > 1 else width, width, q_start.data_ptr(),
                               kv_len.data_ptr(), n)
    return packed, heads, 2 * half


def _append(entry, cache_of, batch, qkv, cos_sin, q_heads, interleaved, positions, out, stream, dev):
    """What both appends do with their arguments."""
    qs = _rows(qkv, "qkv", _TYPES, 2, dev)
    _plain(cos_sin, "cos_sin", _F32, 2, dev)
    cache, kv_heads, dim = cache_of(*batch)
    rows, width = qkv.shape
    if width != (q_heads + 2 * kv_heads) * dim:
        raise ValueError("qkv must be [rows, (q_heads + 2 * kv_heads) * head_dim]")
    if positions is not None:
        _plain(positions, "positions", _I32, 1, dev)
        if positions.shape[0] != rows:
            raise ValueError("positions must have one element per row")
    if out is None:
        out = _empty((rows, q_heads, dim), _BF16, dev, _other(stream, dev))
    else:
        _plain(out, "out", _BF16, 3, dev)
        if tuple(out.shape) != (rows, q_heads, dim):
            raise ValueError("out must be [rows, q_heads, head_dim]")
    if rows == 0:
        return out
    turns, rot = cos_sin.shape
    st = getattr(lib(), entry)(qkv.data_ptr(), _TYPES[qkv.dtype], qs[0] if rows > 1 else width, rows, q_heads,
                               cos_sin.data_ptr(), turns, rot, 1 if interleaved else 0,
                               positions.data_ptr() if positions is not None else None, out.data_ptr(), cache,
                               _stream_of(stream, dev))
    if st:
        _check(st, entry)
    return out


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
    dev = torch.cuda.current_device()
    return _append("q4_0_kv_append", _cache, (k_cache, v_cache, page_table, q_start, kv_len, dev), qkv, cos_sin,
                   q_heads, interleaved, positions, out, stream, dev)


def attention_workspace_bytes(rows: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int) -> int:
    """Scratch of attention on the current device (0 for sizes it refuses)."""
    return _ws_bytes("q4_0_attention_workspace_bytes", rows, q_heads, kv_heads, head_dim, max_q_len)


def _attend(entry, cache_of, batch, q, max_q_len, scale, window, sinks, out, out_dtype, lse, workspace, stream, dev):
    """What both attentions do with their arguments."""
    if out_dtype not in _TYPES:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    qs = _rows(q, "q", (_BF16,), 3, dev)
    cache, kv_heads, cache_dim = cache_of(*batch)
    rows, q_heads, dim = shape = q.shape
    if dim != cache_dim:
        raise ValueError("q and the cache must have the same head_dim")
    other = _other(stream, dev)
    if out is None:
        out = _empty(shape, out_dtype, dev, other)
    else:
        _plain(out, "out", out_dtype, 3, dev)
        if out.shape != shape:
            raise ValueError("out must be [rows, q_heads, head_dim]")
    if lse is not None:
        _plain(lse, "lse", _F32, 2, dev)
        if tuple(lse.shape) != (rows, q_heads):
            raise ValueError("lse must be [rows, q_heads]")
    if rows == 0:
        return out
    ws = _scratch(_ws_bytes(entry + "_workspace_bytes", rows, q_heads, kv_heads, dim, max_q_len), dev, workspace, other)
    st = getattr(lib(), entry)(q.data_ptr(), qs[0], qs[1], out.data_ptr(), _TYPES[out_dtype],
                               lse.data_ptr() if lse is not None else None, rows, q_heads, max_q_len,
                               dim ** -0.5 if scale is None else scale, window, sinks, cache,
                               ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                               _stream_of(stream, dev))
    if st:
        _check(st, entry)
    return out


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
    dev = torch.cuda.current_device()
    return _attend("q4_0_attention", _cache, (k_cache, v_cache, page_table, q_start, kv_len, dev), q, max_q_len,
                   scale, window, sinks, out, out_dtype, lse, workspace, stream, dev)


def kv_append_q4(qkv: torch.Tensor, cos_sin: torch.Tensor, cache: KVCacheQ4, page_table: torch.Tensor,
                 q_start: torch.Tensor, kv_len: torch.Tensor, *, q_heads: int, interleaved: bool = False,
                 positions: torch.Tensor = None, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """kv_append into a cache in 4 bits: keys and values are quantised as they
    are written.  A block of 32 elements with a NaN or one past 65504 in size
    reads back as NaN."""
    dev = torch.cuda.current_device()
    return _append("q4_0_kv_append_q4", _cache_q4, (cache, page_table, q_start, kv_len, dev), qkv, cos_sin,
                   q_heads, interleaved, positions, out, stream, dev)


def kv_read_q4(cache: KVCacheQ4, page_table: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, *, rows: int,
               out_dtype=torch.bfloat16, out=None, stream=None):
    """(k, v) of a batch's rows read back, each [rows, kv_heads, head_dim] of
    out_dtype (bf16, or fp32, which is exact): row q_start[b] + i is the token
    at position kv_len[b] - (q_start[b + 1] - q_start[b]) + i of sequence b --
    what an append of this batch wrote, or whole sequences where q_start counts
    all their tokens up.  rows: q_start[-1], known to the host; rows of no
    sequence are left as they were.  out: a pair of tensors to write to."""
    if out_dtype not in _TYPES:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    dev = torch.cuda.current_device()
    packed, kv_heads, dim = _cache_q4(cache, page_table, q_start, kv_len, dev)
    if rows < 0:
        raise ValueError("rows must not be negative")
    shape = (rows, kv_heads, dim)
    if out is None:
        other = _other(stream, dev)
        k, v = _empty(shape, out_dtype, dev, other), _empty(shape, out_dtype, dev, other)
    else:
        k, v = out
        for t, name in ((k, "out[0]"), (v, "out[1]")):
            _plain(t, name, out_dtype, 3, dev)
            if tuple(t.shape) != shape:
                raise ValueError("out must be a pair of [rows, kv_heads, head_dim]")
    if rows == 0:
        return k, v
    st = lib().q4_0_kv_read_q4(k.data_ptr(), v.data_ptr(), _TYPES[out_dtype], rows, packed, _stream_of(stream, dev))
    if st:
        _check(st, "q4_0_kv_read_q4")
    return k, v


def attention_q4_workspace_bytes(rows: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int) -> int:
    """Scratch of attention_q4 on the current device (0 for sizes it refuses)."""
    return _ws_bytes("q4_0_attention_q4_workspace_bytes", rows, q_heads, kv_heads, head_dim, max_q_len)


def attention_q4(q: torch.Tensor, cache: KVCacheQ4, page_table: torch.Tensor, q_start: torch.Tensor,
                 kv_len: torch.Tensor, *, max_q_len: int, scale: float = None, window: int = 0, sinks: int = 0,
                 out: torch.Tensor = None, out_dtype=torch.bfloat16, lse: torch.Tensor = None,
                 workspace: torch.Tensor = None, stream=None) -> torch.Tensor:
    """attention over a cache in 4 bits (attention_q4_workspace_bytes is its
    scratch)."""
    dev = torch.cuda.current_device()
    return _attend("q4_0_attention_q4", _cache_q4, (cache, page_table, q_start, kv_len, dev), q, max_q_len,
                   scale, window, sinks, out, out_dtype, lse, workspace, stream, dev)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, *, top: int = 0, stream=None):
    """(logprob, entropy, top_logprob, top_ids) of logits [rows, vocab] (fp32
    or bf16): the log probability of tokens[row] (int64; negative: none, 0),
    the row's entropy in nats, and its `top` largest log probabilities with
    their ids ([rows, top], largest first, equal logits by lowest id)."""
    dev = torch.cuda.current_device()
    ls = _rows(logits, "logits", _TYPES, 2, dev)
    _plain(tokens, "tokens", _I64, 1, dev)
    rows, vocab = logits.shape
    if tokens.shape[0] != rows:
        raise ValueError("tokens must have one element per row of logits")
    other = _other(stream, dev)
    logprob = _empty(rows, _F32, dev, other)
    entropy = _empty(rows, _F32, dev, other)
    top_logprob = _empty((rows, max(top, 0)), _F32, dev, other)
    top_ids = _empty((rows, max(top, 0)), _I64, dev, other)
    if rows == 0:
        return logprob, entropy, top_logprob, top_ids
    st = lib().q4_0_token_logprobs(logits.data_ptr(), _TYPES[logits.dtype], ls[0] if rows > 1 else vocab, rows, vocab,
                                   tokens.data_ptr(), top, logprob.data_ptr(), entropy.data_ptr(),
                                   top_logprob.data_ptr() if top else None, top_ids.data_ptr() if top else None,
                                   _stream_of(stream, dev))
    if st:
        _check(st, "q4_0_token_logprobs")
    return logprob, entropy, top_logprob, top_ids
