"""q4_0_token_logprobs against 64-bit sums (GPU).

Tolerance.  All statistics are fp32.  With X the largest finite |logit| of the
row, every exponent, the reference m and the final lse are products and sums
of size at most 2 X log2 e: fewer than eight such roundings, each 2^-24 of
that, in log units below 16 * 2^-24 X.  A sum runs through at most vocab / 512
+ 64 additions in a row (a thread's share of one row, then a tree): a relative
error below that count times 2^-24, which is an absolute one in its logarithm;
the entropy has it times sum p |log p|.  Ids are exact.
"""
import math

import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu


def check(x, tokens, top):
    q4 = lib()
    logprob, entropy, value, ids = q4.token_logprobs(x, tokens, top=top)
    lp, h, v, i, spread = ref.logprobs(x, tokens, top)
    assert torch.equal(ids, i)
    finite = torch.where(torch.isfinite(x), x, 0).double().abs().amax(-1)
    count = x.shape[1] / 512 + 64
    tol = 16 * 2 ** -24 * finite + count * 2 ** -24 + 2 ** -22
    given = tokens >= 0
    off = torch.where(lp == logprob, 0.0, (logprob.double() - lp).abs())
    assert (off <= tol)[given].all(), (off / tol)[given].max()
    assert (logprob == 0)[~given].all()
    off = torch.where(v == value, 0.0, (value.double() - v).abs())
    assert (off <= tol[:, None]).all()
    assert ((entropy.double() - h).abs() <= tol * (1 + spread) + tol).all()
    assert (entropy >= 0).all()
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab,top", [
    (1, 1, 1), (1, 1, 0), (3, 5, 5), (2, 31, 20), (1, 33, 32), (5, 511, 4), (2, 4097, 32), (3, 8191, 1), (2, 8192, 20),
    (2, 8193, 20), (1, 32000, 5), (16, 128257, 20), (160, 3001, 8), (151, 20000, 0), (400, 16385, 32), (700, 50257, 20),
])
def test_shapes(dtype, rows, vocab, top):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(dtype)
    check(x, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), top)


ORDERS = {
    "ascending": lambda x: x.sort(-1)[0],
    "descending": lambda x: x.sort(-1, descending=True)[0],
    "constant": lambda x: torch.full_like(x, -2.5),
    "few values": lambda x: (x * 2).round(),
    "signed zeros": lambda x: torch.where(torch.arange(x.shape[1], device="cuda") % 2 == 1, -0.0, 0.0).to(x.dtype).expand(
        x.shape).contiguous(),
    "one in a thousand allowed": lambda x: torch.where(torch.arange(x.shape[1], device="cuda") % 977 == 5, x, -math.inf),
    "three allowed": lambda x: torch.where((torch.arange(x.shape[1], device="cuda") * 3) % x.shape[1] < 3, x, -math.inf),
    "lowest value": lambda x: torch.where(torch.arange(x.shape[1], device="cuda") % 3 == 0, x,
                                          torch.finfo(x.dtype).min).to(x.dtype),
    "far apart": lambda x: x * 1000,
}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", sorted(ORDERS))
@pytest.mark.parametrize("rows,vocab", [(2, 40000), (320, 20011)])
def test_orders_ties_and_masks(dtype, order, rows, vocab):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = ORDERS[order](torch.randn(rows, vocab, generator=g, device="cuda").to(dtype))
    check(x, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_and_unaligned_rows(dtype):
    wide = (torch.randn(37, 9011, device="cuda") * 2).to(dtype)
    for x in (wide[:, 1:9000], wide[::2, 3:8200], wide[:, 5:6], wide[1:2, 7:]):
        check(x, torch.randint(0, x.shape[1], (x.shape[0],), device="cuda"), min(3, x.shape[1]))


def test_rows_past_32_bit_offsets():
    x = torch.zeros(17000, 131072, dtype=torch.bfloat16, device="cuda")     # 2.2e9 logits
    x[-1, 5], x[-1, 131071] = 3.0, 9.0
    x[-2, 131071] = 4.0
    part = x[-3:]
    q4 = lib()
    logprob, entropy, value, ids = q4.token_logprobs(x, torch.full((17000,), 5, device="cuda"), top=2)
    lp, h, v, i, _ = ref.logprobs(part, torch.full((3,), 5, device="cuda"), 2)
    assert torch.equal(ids[-3:], i)
    assert (logprob[-3:].double() - lp).abs().max() < 1e-4 and (entropy[-3:].double() - h).abs().max() < 1e-3
    assert torch.equal(ids[0], torch.tensor([0, 1], device="cuda"))


@pytest.mark.parametrize("rows", [2, 400])
def test_rows_without_a_number(rows):
    """Nothing but -inf; NaN; +inf; the rows beside them keep their results."""
    q4 = lib()
    x = torch.randn(rows, 9000, device="cuda")
    t = torch.full((rows,), 17, device="cuda")
    clean = q4.token_logprobs(x, t, top=4)
    x[0] = -math.inf
    logprob, entropy, value, ids = q4.token_logprobs(x, t, top=4)
    assert logprob[0] == -math.inf and entropy[0] == 0 and (value[0] == -math.inf).all()
    assert ids[0].tolist() == [0, 1, 2, 3]
    for a, c in zip((logprob, entropy, value, ids), clean):
        assert torch.equal(a[1:], c[1:])
    x[0] = 1.0
    x[0, 8000] = x[0, 300] = math.nan
    logprob, entropy, value, ids = q4.token_logprobs(x, t, top=4)
    assert logprob[0].isnan() and entropy[0].isnan() and value[0].isnan().all()
    assert ids[0].tolist() == [300, 8000, 0, 1]
    x[0] = 1.0
    x[0, 8000] = math.inf
    logprob, entropy, value, ids = q4.token_logprobs(x, t, top=4)
    assert logprob[0].isnan() and ids[0].tolist() == [8000, 0, 1, 2]
    assert torch.equal(logprob[1:], clean[0][1:])
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [2, 400])
def test_rows_at_the_ends_of_the_range(dtype, rows):
    """A row of nothing but the type's lowest value (a mask that leaves
    nothing) is uniform, as is one of its highest; one allowed token among
    lowest values is certain."""
    q4 = lib()
    info = torch.finfo(dtype)
    x = torch.full((rows, 9000), info.min, dtype=dtype, device="cuda")
    x[0] = info.max
    x[-1, 77] = 2.0
    logprob, entropy, value, ids = q4.token_logprobs(x, torch.full((rows,), 77, device="cuda"), top=3)
    uniform = torch.full((rows - 1,), -math.log(9000), device="cuda")
    assert torch.allclose(logprob[:-1], uniform, rtol=0, atol=1e-4)
    assert torch.allclose(entropy[:-1], -uniform, rtol=0, atol=1e-4)
    assert torch.allclose(value[:-1], uniform[:, None].expand(-1, 3), rtol=0, atol=1e-4)
    assert (ids[:-1] == torch.arange(3, device="cuda")).all()
    assert logprob[-1] == 0 and entropy[-1] == 0 and ids[-1].tolist() == [77, 0, 1] and value[-1, 0] == 0
    assert q4.device_error() == q4.OK


def test_tokens_missing_and_out_of_range():
    q4 = lib()
    x = torch.randn(3, 500, device="cuda")
    check(x, torch.tensor([-1, 4, -100], device="cuda"), 2)
    logprob, *_ = q4.token_logprobs(x, torch.tensor([1, 500, 2], device="cuda"), top=2)
    assert q4.device_error() == q4.ERR_DEVICE_INDEX
    assert logprob[1].isnan() and torch.isfinite(logprob[[0, 2]]).all()


@pytest.mark.parametrize("vocab", [2049, 4100, 8195, 70001])
@pytest.mark.parametrize("rows", [1, 19, 38, 39, 76, 77, 152, 153])
def test_rows_shared_by_blocks(rows, vocab):
    """Row counts and vocabularies at which the blocks of a row change."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, generator=g, device="cuda")
    x[:, vocab // 2:] -= 30.0  # some blocks hold none of the top
    check(x, torch.randint(0, vocab, (rows,), generator=g, device="cuda"), 20)


def test_graph_replay_reads_new_logits():
    q4 = lib()
    x, t = torch.randn(3, 40000, device="cuda"), torch.tensor([5, -1, 39999], device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        q4.token_logprobs(x, t, top=7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = q4.token_logprobs(x, t, top=7)
    x.copy_(torch.randn(3, 40000, device="cuda"))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, q4.token_logprobs(x, t, top=7)))
    check(x, t, 7)


def test_same_bits_twice_and_another_stream():
    q4 = lib()
    x = torch.randn(5, 70001, device="cuda").bfloat16()
    t = torch.arange(5, device="cuda")
    a = q4.token_logprobs(x, t, top=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = q4.token_logprobs(x, t, top=20, stream=side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_refusals():
    q4 = lib()
    x, t = torch.zeros(2, 10, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        q4.token_logprobs(x.half(), t)
    with pytest.raises(TypeError):
        q4.token_logprobs(x, t.int())
    with pytest.raises(ValueError):
        q4.token_logprobs(x, t[:1])
    with pytest.raises(ValueError):
        q4.token_logprobs(x.cpu(), t)
    with pytest.raises(ValueError):
        q4.token_logprobs(x.t(), torch.zeros(10, dtype=torch.int64, device="cuda"))
    with pytest.raises(q4.Q4Error) as e:
        q4.token_logprobs(x, t, top=11)                        # more than the vocabulary
    assert e.value.status == q4.ERR_INVALID_ARG
    with pytest.raises(q4.Q4Error) as e:
        q4.token_logprobs(torch.zeros(2, 100, device="cuda"), t, top=33)
    assert e.value.status == q4.ERR_UNSUPPORTED
    with pytest.raises(q4.Q4Error) as e:
        q4.token_logprobs(x, t, top=-1)
    assert e.value.status == q4.ERR_INVALID_ARG
    out = q4.token_logprobs(x[:0], t[:0], top=3)
    assert [o.shape for o in out] == [(0,), (0,), (0, 3), (0, 3)]
