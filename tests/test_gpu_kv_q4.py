"""q4_0_kv_append_q4 and q4_0_kv_read_q4 (GPU).

The rotation is products and sums rounded to fp32 one by one, and the blocks
follow the weights' quantizer: numpy's fp32 arithmetic and the CPU oracle give
the same codes and scales bit for bit, and so are they compared.  Queries are
one rounding to bfloat16 of the same fp32 numbers.  Reading back multiplies a
binary16 scale by a whole number of four bits, exact in fp32.
"""
import math

import numpy as np
import pytest
import torch

import serving_ref_q4 as ref4
from gpu_common import lib
from serving_ref_q4 import Batch

pytestmark = pytest.mark.gpu


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def rotated(x, cos, sin, interleaved):
    """x [heads, rot] fp32 of one row, one rounding an operation."""
    x, cos, sin = x.numpy(), cos.numpy(), sin.numpy()
    half = x.shape[-1] // 2
    a, b = (x[:, 0::2], x[:, 1::2]) if interleaved else (x[:, :half], x[:, half:])
    c, d = a * cos - b * sin, b * cos + a * sin
    out = np.empty_like(x)
    if interleaved:
        out[:, 0::2], out[:, 1::2] = c, d
    else:
        out[:, :half], out[:, half:] = c, d
    assert out.dtype == np.float32
    return torch.from_numpy(out)


def expected(b, qkv, q_heads, rot, interleaved, cs, positions=None):
    """(queries, cache) after the append; rows of no sequence are zeros."""
    x = qkv.float().cpu().view(b.rows, -1, b.dim).clone()
    cache = tuple(t.clone() for t in b.cache)
    q = torch.zeros(b.rows, q_heads, b.dim, dtype=torch.bfloat16)
    for s, n in enumerate(b.new):
        for i in range(n):
            r, pos = int(b.q_start[s]) + i, b.kv[s] - n + i
            turn = pos if positions is None else int(positions[r])
            if rot:
                x[r, :q_heads + b.kv_heads, :rot] = rotated(x[r, :q_heads + b.kv_heads, :rot], cs[turn, :rot // 2],
                                                           cs[turn, rot // 2:], interleaved)
            q[r] = x[r, :q_heads].bfloat16()
            page, off = b.place(s, pos)
            for at, rows in ((0, x[r, q_heads:q_heads + b.kv_heads]), (2, x[r, q_heads + b.kv_heads:])):
                cache[at][page, :, off], cache[at + 1][page, :, off] = ref4.blocks(rows)
    return q, cache


def append(b, q_heads, rot, interleaved, dtype, positions=None, pad=0, seed=1, size=1.0):
    q4 = lib()
    width = (q_heads + 2 * b.kv_heads) * b.dim
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(b.rows, width + pad, generator=g) * size).to(dtype).cuda()[:, :width]
    cs = table(max(b.kv + [1]) + 64, rot)
    b.cuda()
    out = torch.zeros(b.rows, q_heads, b.dim, dtype=torch.bfloat16, device="cuda")
    got = q4.kv_append_q4(qkv, cs.cuda(), *b.dev, q_heads=q_heads, interleaved=interleaved, out=out,
                          positions=None if positions is None else positions.cuda())
    assert got is out and q4.device_error() == q4.OK
    want, cache = expected(b, qkv, q_heads, rot, interleaved, cs, positions)
    assert torch.equal(out.cpu(), want)
    for t, x in zip(b.dev[0], cache):
        assert torch.equal(t.cpu(), x)                # codes, scales and every slot that was not appended to
    return q4


SHAPES = [
    (40, 8, 128, 128, False, 16, False),
    (40, 8, 128, 64, True, 16, True),
    (4, 1, 64, 64, True, 1, False),
    (3, 3, 96, 24, False, 7, True),
    (2, 2, 256, 0, False, 128, False),
    (5, 1, 32, 8, True, 3, False),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q_heads,kv_heads,dim,rot,interleaved,page,token_major", SHAPES)
def test_codes_scales_and_places(dtype, q_heads, kv_heads, dim, rot, interleaved, page, token_major):
    b = Batch([1, 0, 5, 1, 33], [1, 4, 5, 100, 70], page, kv_heads, dim, seed=3, token_major=token_major, fill=(9, 0.5))
    append(b, q_heads, rot, interleaved, dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_in_several_pieces(dtype):
    """A row wider than one block of threads holds (32 KB)."""
    b = Batch([2, 3], [2, 90], 16, 48, 128, seed=4)
    append(b, 96, 128, False, dtype)
    b = Batch([2], [5], 16, 3, 1024, seed=4)
    append(b, 17, 1024, True, dtype)


def test_strided_rows_given_positions_and_rows_of_no_sequence():
    b = Batch([3, 2], [10, 2], 16, 2, 64, seed=5, extra_rows=2)
    positions = torch.tensor([7, 0, 3, 3, 40, 0, 0], dtype=torch.int32)
    append(b, 4, 32, False, torch.float32, positions=positions, pad=8)


@pytest.mark.parametrize("size", [1e-38, 1e-7, 1e-3, 5000.0])
def test_small_and_large_elements(size):
    """Scales below binary16's normal range, and below its smallest number."""
    b = Batch([20], [20], 16, 2, 64, seed=6)
    append(b, 2, 0, False, torch.float32, size=size)


def test_blocks_of_equals_zeros_and_halves():
    """Ties for the largest element and between two codes, and blocks of
    nothing but zeros."""
    q4 = lib()
    b = Batch([4], [4], 16, 1, 64, seed=7)
    x = torch.zeros(4, 3, 64)
    x[0, 1:, 5], x[0, 1:, 17], x[0, 1:, 40] = -3.0, 3.0, 2.0
    x[1, 1:, 20], x[1, 1:, 3], x[1, 1:, 33], x[1, 1:, 63] = 1.0, -1.0, 8.0, -8.0
    x[2, 1:] = torch.arange(-32, 32) / 4.0                        # steps of a quarter: halves of a code
    x[3, 1:] = -0.0
    qkv = x.view(4, -1).cuda()
    b.cuda()
    q4.kv_append_q4(qkv, torch.zeros(8, 0, device="cuda"), *b.dev, q_heads=1)
    _, cache = expected(b, qkv, 1, 0, False, None)
    for t, w in zip(b.dev[0], cache):
        assert torch.equal(t.cpu(), w)
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("size", [1.0, 3e-6, 8000.0])
def test_elements_next_to_half_a_code(size):
    """Every element within two units in the last place of the border of two
    codes, where the rounding of a quotient decides."""
    q4 = lib()
    b = Batch([40], [40], 16, 2, 128, seed=8)
    g = np.random.default_rng(8)
    top = (g.uniform(1, 8, (40, 5, 4, 1)) * g.choice([-1, 1], (40, 5, 4, 1)) * size).astype(np.float32)
    d = top * np.float32(-0.125)
    x = ((g.integers(-8, 8, (40, 5, 4, 32)) + 0.5).astype(np.float32) * d).astype(np.float32)
    for _ in range(2):
        away = g.integers(-1, 2, x.shape)
        x = np.where(away == 0, x, np.nextafter(x, np.where(away > 0, np.inf, -np.inf).astype(np.float32)))
    x = np.clip(x, -np.abs(top), np.abs(top))
    x[..., 7:8] = top
    qkv = torch.from_numpy(x.reshape(40, -1).astype(np.float32)).cuda()
    b.cuda()
    q4.kv_append_q4(qkv, torch.zeros(64, 0, device="cuda"), *b.dev, q_heads=1)
    _, cache = expected(b, qkv, 1, 0, False, None)
    for t, w in zip(b.dev[0], cache):
        assert torch.equal(t.cpu(), w)
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 65520.0, 1e30])
def test_elements_a_block_cannot_hold(bad):
    q4 = lib()
    b = Batch([2], [2], 16, 1, 64, seed=8)
    qkv = torch.randn(2, 3 * 64, device="cuda")
    qkv[0, 64 + 35] = bad                                         # second block of the key
    qkv[1, 2 * 64 + 3] = bad                                      # first block of the value
    qkv[1, 2 * 64 + 40] = -65504.0                                # the largest that fits
    b.cuda()
    q4.kv_append_q4(qkv, torch.zeros(8, 0, device="cuda"), *b.dev, q_heads=1)
    k, v = q4.kv_read_q4(*b.dev, rows=2, out_dtype=torch.float32)
    assert k[0, 0, 32:].isnan().all() and v[1, 0, :32].isnan().all()
    assert k[0, 0, :32].isfinite().all() and k[1].isfinite().all() and v[0].isfinite().all()
    assert v[1, 0, 40] == -65504.0
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("page,kv_heads,dim,token_major", [(16, 8, 128, False), (1, 1, 64, True), (7, 3, 96, False),
                                                           (64, 2, 1024, True), (5, 1, 32, True)])
def test_reading_back(out_dtype, page, kv_heads, dim, token_major):
    q4 = lib()
    b = Batch([1, 0, 5, 1, 33], [1, 4, 5, 100, 70], page, kv_heads, dim, seed=9, token_major=token_major,
              extra_rows=3).write_tokens()
    out = tuple(torch.full((b.rows, kv_heads, dim), 7.0, dtype=out_dtype, device="cuda") for _ in range(2))
    got = q4.kv_read_q4(*b.cuda(), rows=b.rows, out_dtype=out_dtype, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    for i in range(2):
        want = torch.cat([t[i][len(t[i]) - n:] for t, n in zip(b.tokens, b.new)]).to(out_dtype)
        assert torch.equal(got[i][:len(want)].cpu(), want)
        assert (got[i][len(want):] == 7.0).all()
    # whole sequences: q_start counts all their tokens
    starts = torch.tensor([0] + b.kv).cumsum(0).to(torch.int32).cuda()
    k, v = q4.kv_read_q4(b.dev[0], b.dev[1], starts, b.dev[3], rows=sum(b.kv), out_dtype=out_dtype)
    assert torch.equal(k.cpu(), torch.cat([t[0] for t in b.tokens]).to(out_dtype))
    assert torch.equal(v.cpu(), torch.cat([t[1] for t in b.tokens]).to(out_dtype))
    assert q4.device_error() == q4.OK


def test_many_sequences():
    n = 600
    new, kv = [i % 3 for i in range(n)], [i % 3 + i % 20 for i in range(n)]
    append(Batch(new, kv, 16, 1, 64, seed=10), 2, 64, False, torch.bfloat16)
    q4 = lib()
    b = Batch(new, kv, 16, 1, 64, seed=11).write_tokens()
    k, v = q4.kv_read_q4(*b.cuda(), rows=b.rows, out_dtype=torch.float32)
    assert torch.equal(v.double().cpu(), torch.cat([t[1][len(t[1]) - m:] for t, m in zip(b.tokens, new)]))


def test_past_32_bit_offsets():
    """A cache of more than 2^32 bytes of codes: the last page is reached."""
    q4 = lib()
    pages, page, heads, dim = 550000, 16, 8, 128
    cache = q4.kv_cache_q4(pages, heads, page, dim)
    qkv = torch.randn(1, (2 + 2 * heads) * dim)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = (cache, ints(pages - 1)[None], ints(0, 1), ints(6))
    q4.kv_append_q4(qkv.cuda(), torch.zeros(8, 0, device="cuda"), *batch, q_heads=2)
    x = qkv.view(18, dim)
    for i, rows in ((0, x[2:10]), (2, x[10:])):
        codes, scales = ref4.blocks(rows)
        assert torch.equal(cache[i][pages - 1, :, 5].cpu(), codes)
        assert torch.equal(cache[i + 1][pages - 1, :, 5].cpu(), scales)
        assert int(cache[i + 1].count_nonzero()) == scales.numel()
    k, _ = q4.kv_read_q4(*batch, rows=1, out_dtype=torch.float32)
    assert torch.equal(k[0].double().cpu(), ref4.values(*ref4.blocks(x[2:10])))
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("what", ["page", "page past the end", "long", "short", "turn"])
def test_bad_places_are_reported_and_skipped(what):
    q4 = lib()
    b = Batch([1, 1], [9, 5], 4, 1, 64, seed=12)
    cache, page_table, q_start, kv_len = b.cuda()
    positions = None
    if what == "page":
        page_table[0, 2] = -5
    elif what == "page past the end":
        page_table[0, 2] = b.pages
    elif what == "long":
        kv_len[0] = 10 ** 6
    elif what == "short":
        kv_len[0] = 0
    else:
        positions = torch.tensor([10 ** 6, 0], dtype=torch.int32).cuda()
    qkv = torch.randn(2, 3 * 64)
    batch = (cache, page_table, q_start, kv_len)
    q4.kv_append_q4(qkv.cuda(), table(64, 64).cuda(), *batch, q_heads=1, positions=positions)
    assert q4.device_error() == q4.ERR_DEVICE_INDEX
    assert q4.device_error() == q4.OK
    page, off = b.place(1, 4)
    codes, scales = ref4.blocks(qkv[1, 128:][None])
    want = (torch.zeros_like(cache[2]), torch.zeros_like(cache[3]))
    want[0][page, 0, off], want[1][page, 0, off] = codes[0].cuda(), scales[0].cuda()
    assert torch.equal(cache[2], want[0]) and torch.equal(cache[3], want[1])   # the good row, nothing else
    if what != "turn":
        out = tuple(torch.full((2, 1, 64), 7.0, device="cuda") for _ in range(2))
        q4.kv_read_q4(*batch, rows=2, out_dtype=torch.float32, out=out)
        assert q4.device_error() == q4.ERR_DEVICE_INDEX
        assert (out[0][0] == 7.0).all() and (out[1][0] == 7.0).all()
        assert torch.equal(out[1][1, 0].double().cpu(), ref4.values(codes, scales)[0])


def test_a_replayed_graph_follows_the_batch():
    """Append, read and attend captured once; the replay is at other lengths."""
    q4 = lib()
    b = Batch([1, 1], [40, 9], 16, 2, 64, seed=13, width=4).write_tokens()
    cache, page_table, q_start, kv_len = b.cuda()
    cs = table(64, 64).cuda()
    qkv = torch.randn(2, 8 * 64, device="cuda")
    batch = (cache, page_table, q_start, kv_len)

    def step():
        q = q4.kv_append_q4(qkv, cs, *batch, q_heads=4)
        return q4.attention_q4(q, *batch, max_q_len=1), *q4.kv_read_q4(*batch, rows=2)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    kv_len.copy_(torch.tensor([35, 12], dtype=torch.int32))
    qkv.copy_(torch.randn(2, 8 * 64))
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    assert all(torch.equal(a, w) for a, w in zip(got, want))
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("dim,kv_heads,q_heads,page,token_major", [(128, 8, 40, 16, False), (64, 1, 4, 48, True)])
def test_the_operators_together(dim, kv_heads, q_heads, page, token_major):
    """A prompt and then tokens one by one, as a server runs them: attention
    over what was appended is 64-bit attention over what reads back."""
    import serving_ref as ref
    q4 = lib()
    lengths, steps = [37, 5, 130], 3
    b = Batch(lengths, lengths, page, kv_heads, dim, seed=14, token_major=token_major, width=-(-(130 + steps) // page))
    g = torch.Generator().manual_seed(2)
    order = torch.randperm(len(lengths) * b.table.shape[1], generator=g).to(torch.int32)
    cache = q4.kv_cache_q4(order.numel(), kv_heads, page, dim, token_major=token_major)
    page_table, cs = order.view(len(lengths), -1).cuda(), table(256, dim).cuda()
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv = [0] * len(lengths)
    for step in range(1 + steps):
        new = lengths if step == 0 else [1] * len(lengths)
        kv = [k + n for k, n in zip(kv, new)]
        batch = (cache, page_table, ints([0] + new).cumsum(0).to(torch.int32), ints(kv))
        qkv = torch.randn(sum(new), (q_heads + 2 * kv_heads) * dim, generator=g).cuda()
        q = q4.kv_append_q4(qkv, cs, *batch, q_heads=q_heads)
        out = q4.attention_q4(q, *batch, max_q_len=max(new), out_dtype=torch.float32)
        k, v = q4.kv_read_q4(cache, page_table, ints([0] + kv).cumsum(0).to(torch.int32), ints(kv), rows=sum(kv),
                             out_dtype=torch.float32)
        b.new, b.kv, b.q_start = list(new), kv, batch[2].cpu()
        b.tokens = list(zip(k.split(kv), v.split(kv)))
        want, _, weight, bound = ref.attention(q, b, 0, 0, dim ** -0.5)
        e = dim ** -0.5 * (dim * 2 ** -23 + 2 ** -11) * bound       # as in test_gpu_attention_q4.py
        tol = weight * (2 ** -10 + 2 ** -16 + 2 * e[..., None]) + 2 ** -25 * (1 + max(kv) * float(v.abs().max()))
        assert ((out.double() - want).abs() <= tol).all()
    assert q4.device_error() == q4.OK


def test_refusals():
    q4 = lib()
    b = Batch([1], [1], 4, 2, 64)
    dev = b.cuda()
    qkv, cs = torch.zeros(1, 6 * 64, device="cuda"), table(4, 64).cuda()
    good = lambda **k: q4.kv_append_q4(k.pop("qkv", qkv), k.pop("cs", cs), *k.pop("dev", dev),  # noqa: E731
                                       q_heads=k.pop("q_heads", 2), **k)
    read = lambda **k: q4.kv_read_q4(*k.pop("dev", dev), rows=k.pop("rows", 1), **k)  # noqa: E731
    good(), read()
    with pytest.raises(TypeError):
        good(qkv=qkv.half())
    with pytest.raises(ValueError):
        good(q_heads=3)
    for call in (good, read):
        k, ks, v, vs = dev[0]
        with pytest.raises(TypeError):
            call(dev=((k, ks.float(), v, vs), *dev[1:]))
        with pytest.raises(TypeError):
            call(dev=(dev[0], dev[1].long(), *dev[2:]))
        with pytest.raises(ValueError):
            call(dev=((k, ks, v[:1], vs), *dev[1:]))
        with pytest.raises(ValueError):
            call(dev=((k, ks[..., :1], v, vs[..., :1]), *dev[1:]))
        with pytest.raises(ValueError):
            call(dev=((k.cpu(), ks, v, vs), *dev[1:]))
        with pytest.raises(ValueError):
            call(dev=(dev[0], dev[1], dev[2][:1], dev[3]))
        with pytest.raises(q4.Q4Error) as e:                       # rows of codes 8 bytes apart
            call(dev=((k.as_strided(k.shape, (256, 128, 8, 1)), ks, v, vs), *dev[1:]))
        assert e.value.status == q4.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        read(out=(torch.zeros(1, 2, 64, device="cuda"), torch.zeros(1, 1, 64, device="cuda")), out_dtype=torch.float32)
    with pytest.raises(TypeError):
        read(out_dtype=torch.float16)
    with pytest.raises(ValueError):
        read(rows=-1)
    with pytest.raises(ValueError):
        q4.kv_cache_q4(1, 1, 16, 48)
    assert good(qkv=qkv[:0]).shape == (0, 2, 64) and read(rows=0)[0].shape == (0, 2, 64)
    assert q4.device_error() == q4.OK
