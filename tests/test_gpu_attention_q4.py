"""q4_0_attention_q4 against 64-bit attention over the blocks' values (GPU).

Tolerance, per element, from the kernels' roundings.  u = 2^-11 is half a step
of binary16 (relative), 2^-25 half a step below its normal range.
* p_j is rounded to binary16 in units of a reference whose own p is 1 and in
  the sum: u of each moves the output by at most u sum_j w_j |v_j| (w the
  softmax weights), and 2^-25 of each by at most 2^-25 sum_j |v_j|.
* a value is rounded to binary16: u |v_j| + 2^-25, another u sum_j w_j |v_j|
  + 2^-25.
* a score is a sum of D products in fp32, off by at most D 2^-23 sum_i |q_i
  k_i| (times the scale), and by u sum_i |q_i k_i| more where keys are rounded
  to binary16 too (prompts); an error e in every score moves the output by at
  most 2 e sum_j w_j |v_j| and the row's logarithm by e.
* everything else (exponentials, sums, the division) is fp32, for which 2^-16
  of the same size is ample.
A bfloat16 output adds its own rounding, 2^-8 of the value.
"""
import math

import pytest
import torch

import serving_ref as ref
from gpu_common import lib
from serving_ref_q4 import Batch

pytestmark = pytest.mark.gpu
U = 2 ** -11


def run(b, q_heads, window=0, sinks=0, scale=None, out_dtype=torch.float32, q_scale=1.0, seed=1, q=None, **kw):
    q4 = lib()
    if q is None:
        g = torch.Generator().manual_seed(seed)
        q = (torch.randn(b.rows, q_heads, b.dim, generator=g) * q_scale).bfloat16().cuda()
    lse = torch.full((b.rows, q_heads), 7.0, device="cuda")
    dev = b.dev if hasattr(b, "dev") else b.cuda()
    out = q4.attention_q4(q, *dev, max_q_len=max(b.new + [1]), window=window, sinks=sinks, scale=scale,
                          out_dtype=out_dtype, lse=lse, **kw)
    assert q4.device_error() == q4.OK
    return q, out, lse


def check(b, q, out, lse, window=0, sinks=0, scale=None):
    s = b.dim ** -0.5 if scale is None else scale
    want, want_lse, weight, bound = ref.attention(q, b, window, sinks, s)
    inside = torch.zeros(b.rows, dtype=torch.bool, device="cuda")
    inside[int(b.q_start[0]):int(b.q_start[-1])] = True
    e = s * (b.dim * 2 ** -23 + U) * bound
    largest = max([float(v.abs().max()) for _, v in b.tokens if len(v)] + [0.0])
    tol = weight * (2 * U + 2 ** -16 + 2 * e[..., None]) + 2 ** -25 * (1 + max(b.kv) * largest)
    if out.dtype == torch.bfloat16:
        tol = tol + 2 ** -8 * (want.abs() + tol)
    off = (out.double() - want).abs()
    assert (off <= tol)[inside].all(), (off - tol)[inside].max()
    finite = inside[:, None] & torch.isfinite(want_lse)
    assert ((lse.double() - want_lse).abs() <= e + 2 ** -16 * (1 + want_lse.abs()))[finite].all()
    assert (lse == -math.inf)[inside[:, None] & ~finite].all()
    assert (lse == 7.0)[~inside].all()              # rows of no sequence are not written


HEADS = [(40, 8, 128), (8, 8, 64), (7, 1, 128), (32, 2, 64), (128, 1, 64), (9, 3, 128)]


@pytest.mark.parametrize("q_heads,kv_heads,dim", HEADS)
@pytest.mark.parametrize("new,kv", [
    ([1], [1]), ([1], [2]), ([1], [127]), ([1], [128]), ([1], [129]), ([1], [700]),
    ([1, 1, 1, 1, 1], [5, 1, 300, 64, 1025]),
    ([4, 0, 7, 2], [4, 9, 200, 260]),
    ([60], [60]), ([129], [500]),
    ([33, 1, 0, 1, 300], [33, 900, 0, 1, 420]),
    ([1, 2, 3, 1], [31, 33, 64, 512]),
    ([6, 3], [6, 1000]),
])
def test_lengths_and_heads(q_heads, kv_heads, dim, new, kv):
    b = Batch(new, kv, 16, kv_heads, dim, seed=len(new) + kv[0]).write_tokens()
    check(b, *run(b, q_heads))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page,token_major", [(8, False), (16, True), (24, False), (48, True), (128, False),
                                              (256, True), (200, False)])
def test_pages(dim, page, token_major):
    """Pages that end inside a tile, and that hold several."""
    b = Batch([1, 50, 3], [300, 333, 129], page, 2, dim, seed=page, token_major=token_major).write_tokens()
    q, out, lse = run(b, 6)
    check(b, q, out, lse)
    q, out, lse = run(b, 6, window=100, sinks=3)
    check(b, q, out, lse, 100, 3)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (64, 0), (127, 4), (128, 128), (129, 130), (300, 5),
                                          (5000, 7)])
def test_windows_and_sinks(dim, window, sinks):
    b = Batch([1, 90, 1, 5], [1000, 700, 40, 2000], 32, 2, dim, seed=window).write_tokens()
    q, out, lse = run(b, 10, window=window, sinks=sinks)
    check(b, q, out, lse, window, sinks)


@pytest.mark.parametrize("new,kv", [([1, 5, 1], [300, 200, 129]), ([70, 1], [450, 1000])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 3)])
def test_unseen_memory_does_not_matter(new, kv, window, sinks):
    """NaN in every slot and page that no query sees, and no page at all in
    the table where none is seen."""
    b = Batch(new, kv, 16, 2, 128, seed=9, fill=(255, math.nan)).write_tokens()
    for s, (n, length) in enumerate(zip(new, kv)):
        gone = range(sinks, max(sinks, length - n - window + 1)) if window else ()
        for j in gone:
            page, off = b.place(s, j)
            for t in b.cache:
                t[page, :, off] = 77 if t.dtype == torch.uint8 else math.inf
        for first in range(0, length, 16):
            if all(j in gone for j in range(first, min(first + 16, length))):
                b.table[s, first // 16] = -1
    q, out, lse = run(b, 4, window=window, sinks=sinks)
    check(b, q, out, lse, window, sinks)


@pytest.mark.parametrize("new,kv", [([5], [3]), ([4, 1], [0, 6]), ([60, 2], [30, 1])])
def test_rows_that_see_nothing(new, kv):
    """More new tokens than the cache holds: the first rows are at positions
    before the sequence, give 0 and -infinity, and disturb nobody."""
    b = Batch(new, kv, 16, 1, 64, seed=10).write_tokens()
    check(b, *run(b, 5))


def test_rows_of_no_sequence_and_empty_batches():
    b = Batch([2, 0, 3], [2, 0, 80], 16, 1, 64, seed=11, extra_rows=3).write_tokens()
    check(b, *run(b, 3))
    b = Batch([0, 0], [5, 0], 16, 1, 64, extra_rows=2).write_tokens()
    q, out, lse = run(b, 3)
    assert (lse == 7.0).all()


@pytest.mark.parametrize("rise", [2.0, 40.0, 300.0, -300.0])
@pytest.mark.parametrize("dim", [64, 128])
def test_scores_that_rise_along_the_keys(rise, dim):
    """Every tile's maximum far above (or below) the last one's: the running
    reference has to follow it."""
    b = Batch([1, 64], [1000, 900], 16, 1, dim, seed=12).write_tokens()
    for s, kv in enumerate(b.kv):
        k, v = b.tokens[s]
        k = k.clone()
        k[:, :, :32] = 0.0
        k[:, :, 0] = (torch.arange(kv) / kv * rise)[:, None]
        b.tokens[s] = b.put(s, k, v)
    q = torch.randn(b.rows, 4, dim, generator=torch.Generator().manual_seed(2))
    q[..., 0] = 8.0
    q = q.bfloat16().cuda()
    _, out, lse = run(b, 4, q=q)
    check(b, q, out, lse)


@pytest.mark.parametrize("new", [1, 3, 40])
def test_nan_scales_reach_the_rows_that_see_them(new):
    """A key's NaN reaches only the rows that see it; so does a value's among
    rows that are further apart than the documented distance."""
    b = Batch([new, new], [50, 300], 16, 1, 64, seed=23).write_tokens()
    q, want, want_lse = run(b, 4)
    page, off = b.place(0, 49)                                   # the last token of sequence 0
    for i in (1, 3):
        cache = list(b.cache)
        cache[i] = cache[i].clone()
        cache[i][page, 0, off, 1] = math.nan
        dev = (tuple(t.cuda() for t in cache), *b.dev[1:])
        q4 = lib()
        out = q4.attention_q4(q, *dev, max_q_len=new, out_dtype=torch.float32)
        assert out[new - 1].isnan().any()
        if i == 1:
            assert out[new - 1].isnan().all() and torch.equal(out[:new - 1], want[:new - 1])
        else:
            assert out[new - 1, :, 32:].isnan().all() and torch.equal(out[:, :, :32], want[:, :, :32])
        assert torch.equal(out[new:], want[new:])


@pytest.mark.parametrize("q_scale", [2 ** -60, 2 ** -20, 2 ** 10])
def test_queries_of_any_size(q_scale):
    b = Batch([1, 40], [300, 200], 16, 2, 128, seed=24).write_tokens()
    q, out, lse = run(b, 4, q_scale=q_scale, scale=0.1 / q_scale)
    check(b, q, out, lse, scale=0.1 / q_scale)


def test_certain_keys():
    """Scores far apart: one key has all the weight and its value comes back
    with nothing but its rounding to binary16."""
    b = Batch([1, 30], [400, 90], 16, 1, 128, seed=25).write_tokens()
    q, out, lse = run(b, 2, q_scale=64.0, scale=1000.0)
    s = torch.einsum("hd,jd->hj", q[0].double(), b.tokens[0][0][:, 0].cuda())
    best = b.tokens[0][1][:, 0].cuda()[s.argmax(-1)]
    assert ((out[0].double() - best).abs() <= U * best.abs() + 2 ** -25).all()


def test_scale_and_bf16_output():
    b = Batch([1, 40], [600, 333], 64, 2, 128, seed=13).write_tokens()
    q, out, lse = run(b, 10, scale=0.5, out_dtype=torch.bfloat16)
    check(b, q, out, lse, scale=0.5)


def test_long_context_and_many_sequences():
    b = Batch([1], [40000], 64, 2, 128, seed=14).write_tokens()
    check(b, *run(b, 10))
    n = 900
    b = Batch([(i % 5 == 0) + (i % 7 == 0) * 20 for i in range(n)], [30 + i % 150 for i in range(n)], 16, 1, 64,
                  seed=15).write_tokens()
    check(b, *run(b, 4))


@pytest.mark.parametrize("q_heads,kv_heads,dim", [(40, 8, 128), (16, 8, 64), (32, 2, 128), (80, 8, 64)])
@pytest.mark.parametrize("longest,window", [(128, 0), (300, 0), (300, 20), (5, 0)])
def test_many_short_sequences(q_heads, kv_heads, dim, longest, window):
    """Many items of one or two key tiles in every share."""
    n = 140 * 8 // kv_heads
    b = Batch([1] * n, [1 + (i * 37) % longest for i in range(n)], 16, kv_heads, dim, seed=21).write_tokens()
    q, out, lse = run(b, q_heads, window=window)
    check(b, q, out, lse, window)


@pytest.mark.parametrize("new,longest", [(7, 120), (20, 130), (33, 200)])
def test_many_short_drafts(new, longest):
    b = Batch([new] * 150, [new + (i * 29) % longest for i in range(150)], 16, 8, 128, seed=22).write_tokens()
    check(b, *run(b, 40))
    b = Batch([new, 1] * 90, [new + (i * 29) % longest for i in range(180)], 16, 8, 128, seed=23).write_tokens()
    check(b, *run(b, 40))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window", [0, 90])
def test_items_of_one_and_two_tiles_in_turn(dim, window):
    """A CTA's share of some thousand items mixes both kinds at any offset."""
    new = [(1, 60, 3, 129, 40, 1, 1, 26)[i % 8] + (i % 3 == 0) * 25 for i in range(400)]
    b = Batch(new, [n + 37 * (i % 11) for i, n in enumerate(new)], 32, 2, dim, seed=20).write_tokens()
    check(b, *run(b, 10, window=window, sinks=2 if window else 0), window, 2 if window else 0)


@pytest.mark.parametrize("q_heads,kv_heads", [(10, 2), (40, 2)])
@pytest.mark.parametrize("max_q_len", [2, 9, 30, 5000])
def test_a_bound_above_the_batch(q_heads, kv_heads, max_q_len):
    """max_q_len is a bound: single tokens under one that lets both kernels
    run, or that is above the number of rows."""
    b = Batch([1] * 30, [3 + 37 * i for i in range(30)], 16, kv_heads, 64, seed=19).write_tokens()
    q = torch.randn(b.rows, q_heads, b.dim, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    q4, lse = lib(), torch.full((b.rows, q_heads), 7.0, device="cuda")
    out = q4.attention_q4(q, *b.cuda(), max_q_len=max_q_len, out_dtype=torch.float32, lse=lse)
    assert q4.device_error() == q4.OK
    check(b, q, out, lse)


@pytest.mark.parametrize("new,extra", [([5, 5, 5], 0), ([1, 5, 5], 4), ([5, 0, 2], 8), ([40, 40], 0), ([40, 1], 39),
                                       ([40, 25], 0), ([40, 3], 30), ([30], 0), ([2], 40), ([40, 4], 0), ([5, 3, 5], 1)])
def test_rows_enough_for_long_sequences_alone(new, extra):
    """Batches whose rows could all be of sequences too long for the kernel of
    few rows: in some they are, and in some a shorter sequence leaves rows of
    none."""
    b = Batch(new, [300 + 77 * i + n for i, n in enumerate(new)], 16, 2, 128, seed=20, extra_rows=extra).write_tokens()
    check(b, *run(b, 10))
    check(b, *run(b, 10, window=60, sinks=3), window=60, sinks=3)


def test_strided_queries():
    """Queries inside fused rows: row and head strides of their own."""
    b = Batch([1, 30], [100, 200], 16, 2, 64, seed=16).write_tokens()
    wide = torch.randn(b.rows, 14, 64, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    q = wide[:, 2:10]
    _, out, lse = run(b, 8, q=q)
    check(b, q, out, lse)
    q = wide.view(b.rows, 7, 2, 64)[:, :6, 1]
    _, out, lse = run(b, 6, q=q)
    check(b, q, out, lse)


def test_one_key_head_and_strides_of_single_dimensions():
    b = Batch([1], [50], 64, 1, 128, seed=17, spare=0).write_tokens()
    (k, ks, v, vs), *rest = b.cuda()
    b.dev = ((k.as_strided(k.shape, (1, 3, 64, 1)), ks.as_strided(ks.shape, (7, 1, 4, 1)),
              v.as_strided(v.shape, (5, 1, 64, 1)), vs.as_strided(vs.shape, (1, 3, 4, 1))), *rest)
    check(b, *run(b, 4))


def test_reads_past_32_bit_offsets():
    q4 = lib()
    pages, page, heads, dim = 550000, 16, 8, 128                # 4.5e9 bytes of codes
    cache = q4.kv_cache_q4(pages, heads, page, dim)
    b = Batch([1, 1], [200, 75], page, heads, dim, seed=18).write_tokens()
    shift = pages - b.pages
    small, table, *rest = b.cuda()
    for t, x in zip(cache, small):
        t[shift:] = x
    b.dev = (cache, torch.where(table >= 0, table + shift, table), *rest)
    check(b, *run(b, 16))
    assert q4.device_error() == q4.OK


def test_same_bits_twice_and_graph_replay_follows_lengths():
    q4 = lib()
    b = Batch([1] * 6, [700, 90, 1, 2000, 333, 64], 16, 2, 128, seed=19, width=130).write_tokens()
    q, out, lse = run(b, 10)
    _, again, lse2 = run(b, 10, q=q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    cache, table, q_start, kv_len = b.dev
    ws = torch.empty(q4.attention_q4_workspace_bytes(b.rows, 10, 2, 128, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(out)
    call = lambda: q4.attention_q4(q, cache, table, q_start, kv_len, max_q_len=1, out=out,  # noqa: E731
                                   out_dtype=torch.float32, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    b.kv = [650, 1, 1, 1999, 129, 64]
    b.tokens = [(kk[:n], vv[:n]) for (kk, vv), n in zip(b.tokens, b.kv)]
    kv_len.copy_(torch.tensor(b.kv, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    check(b, q, out, lse)


def test_another_stream():
    q4 = lib()
    b = Batch([1, 90], [500, 300], 16, 2, 128, seed=20).write_tokens()
    b.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = torch.randn(b.rows, 10, 128, device="cuda").bfloat16()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):                       # memory made for the side stream is not handed out meanwhile
        outs.append(q4.attention_q4(q, *b.dev, max_q_len=90, stream=side, out_dtype=torch.float32))
        torch.empty(1 << 22, device="cuda").fill_(math.nan)
    side.synchronize()
    _, want, lse = run(b, 10, q=q)
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("what", ["page", "page past the end", "kv_len", "q_start", "max_q_len"])
def test_bad_arrays_are_reported(what):
    """Indices out of range in device memory: never dereferenced, reported,
    and the sequences they do not concern keep their results."""
    q4 = lib()
    b = Batch([3, 2], [40, 90], 16, 1, 64, seed=21).write_tokens()
    q, want, _ = run(b, 4)
    cache, (table, q_start, kv_len) = b.dev[0], (t.clone() for t in b.dev[1:])
    limit = 3
    if what == "page":
        table[0, 1] = -3
    elif what == "page past the end":
        table[0, 1] = b.pages
    elif what == "kv_len":
        kv_len[0] = 10 ** 8
    elif what == "q_start":
        q_start[2] = 10 ** 6
    else:
        limit = 2
    out = q4.attention_q4(q, cache, table, q_start, kv_len, max_q_len=limit, out_dtype=torch.float32)
    assert q4.device_error() == q4.ERR_DEVICE_INDEX
    assert q4.device_error() == q4.OK
    if what != "q_start":
        assert (out[3:] - want[3:]).abs().max() <= 1e-5      # another split of the work, no other keys


def test_refusals():
    q4 = lib()
    b = Batch([1], [20], 16, 2, 64, seed=22).write_tokens()
    dev = b.cuda()
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    def good(**k):
        return q4.attention_q4(k.pop("q", q), *k.pop("dev", dev), max_q_len=k.pop("max_q_len", 1), **k)

    good()
    with pytest.raises(TypeError):
        good(q=q.float())
    with pytest.raises(ValueError):
        good(q=q[..., :32])
    with pytest.raises(ValueError):
        good(q=q.cpu())
    with pytest.raises(TypeError):
        good(out_dtype=torch.float16)
    with pytest.raises(ValueError):
        good(out=torch.zeros(1, 4, 32, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        good(lse=torch.zeros(1, 3, device="cuda"))
    with pytest.raises(ValueError):
        good(dev=((*dev[0][:2], dev[0][2][:, :1], dev[0][3]), *dev[1:]))
    with pytest.raises(ValueError):
        good(dev=((dev[0][0], dev[0][1][..., :1], *dev[0][2:]), *dev[1:]))
    with pytest.raises(TypeError):
        good(dev=((dev[0][0], dev[0][1].float(), *dev[0][2:]), *dev[1:]))
    with pytest.raises(TypeError):
        good(dev=((dev[0][1], dev[0][0], *dev[0][2:]), *dev[1:]))
    with pytest.raises(ValueError):
        good(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    for bad in ({"max_q_len": 0}, {"scale": 0.0}, {"scale": -1.0}, {"scale": math.nan}, {"window": -1}, {"sinks": -1},
                {"q": q[:, :3].contiguous()}):                # 3 query heads on 2 key heads
        with pytest.raises(q4.Q4Error) as e:
            good(**bad)
        assert e.value.status == q4.ERR_INVALID_ARG
    odd = Batch([1], [5], 12, 2, 64).write_tokens()        # page_size % 8
    with pytest.raises(q4.Q4Error) as e:
        good(dev=odd.cuda())
    assert e.value.status == q4.ERR_UNSUPPORTED
    wide = Batch([1], [5], 16, 2, 96).write_tokens()       # head_dim
    with pytest.raises(q4.Q4Error) as e:
        good(q=torch.zeros(1, 4, 96, dtype=torch.bfloat16, device="cuda"), dev=wide.cuda())
    assert e.value.status == q4.ERR_UNSUPPORTED
    assert good(q=q[:0]).shape == (0, 4, 64)
    assert q4.device_error() == q4.OK
