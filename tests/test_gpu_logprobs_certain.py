"""q4_0_token_logprobs where its log probabilities are near 0 or its logits
are far from it: certain tokens, masks, common offsets (GPU).

Tolerance, which does not grow with an offset of the row.  With m the row's
maximum, each p_j = exp(x_j - m) / sum comes from a difference and a product
(2^-24 of |x_j - m| each, as does the constant log2 e), an exponential (2^-22),
and shifts of the reference that add up to at most |x_j - m| (2^-24 of it
twice): in log units below 8 * 2^-24 sum p |x - m|, and 2^-22.  A sum adds its
additions in a row (vocab / 512 + 64) times 2^-24.  The difference of the
token's logit and m, the sum's logarithm and its product with ln 2 are rounded
too: 4 * 2^-24 of |x - m| and of ln sum.  In the entropy, sum p |x - m| has
the errors of its terms: those of p times |x - m|, so 8 * 2^-24 sum p (x - m)^2
and the additions times sum p |x - m|.
A token that is certain has p = 1 and sum = 1 exactly: 0, without tolerance,
and no log probability is above 0 in any row.
"""
import math

import pytest
import torch

import serving_ref as ref
from gpu_common import lib

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16]
ROWS = [(1, 32000), (2, 8192), (16, 9000), (400, 9000)]
# an ordinary logit's product with log2 e is rounded; 1e10 * log2 e is off by hundreds
LOGITS = [3.0, 12.7, 60.7, -27.9, 1000.3, 30000.5, 1e10, -3e18]


def check(x, tokens, top):
    q4 = lib()
    logprob, entropy, value, ids = q4.token_logprobs(x, tokens, top=top)
    lp, h, v, i, _ = ref.logprobs(x, tokens, top)
    assert torch.equal(ids, i)
    m = x.double().amax(-1, keepdim=True)
    below = (x.double() - m).clamp(min=-1e300)
    ln_sum = below.exp().sum(-1)
    p = below.exp() / ln_sum[:, None]
    ln_sum = ln_sum.log()
    near = torch.where(p > 0, -below, 0.0)
    size, square = (p * near).sum(-1), (p * near * near).sum(-1)
    count = x.shape[1] / 512 + 64
    tol = 8 * size + 4 * ln_sum + count + 16

    def close(got, want, bound):
        off = torch.where(got == want, 0.0, (got.double() - want).abs())
        assert (off <= 2 ** -24 * bound).all(), (off / bound * 2 ** 24).max()

    given = below.gather(1, tokens[:, None])[:, 0]
    close(logprob, lp, tol + 4 * given.abs())
    close(value, v, tol[:, None] + 4 * below.gather(1, i).abs())
    close(entropy, h, tol + 8 * square + count * size + 4 * h)
    assert (logprob <= 0).all() and (value <= 0).all() and (entropy >= 0).all()
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", ROWS)
@pytest.mark.parametrize("mask", ["infinity", "lowest"])
def test_the_one_allowed_token_is_certain(dtype, rows, vocab, mask):
    q4 = lib()
    nothing = -math.inf if mask == "infinity" else torch.finfo(dtype).min
    for logit in LOGITS:
        x = torch.full((rows, vocab), nothing, dtype=dtype, device="cuda")
        at = torch.arange(rows, device="cuda") * 7919 % vocab
        x[torch.arange(rows, device="cuda"), at] = logit
        logprob, entropy, value, ids = q4.token_logprobs(x, at, top=2)
        assert (logprob == 0).all() and (value[:, 0] == 0).all() and (entropy == 0).all(), (logit, logprob.max())
        assert torch.equal(ids[:, 0], at)
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", ROWS)
@pytest.mark.parametrize("allowed", [3, 400])
def test_a_few_allowed_tokens(dtype, rows, vocab, allowed):
    g = torch.Generator(device="cuda").manual_seed(rows + allowed)
    for offset in (0.0, 20.7, 100.3, -1000.3, 30000.5):
        for nothing in (-math.inf, torch.finfo(dtype).min):
            x = torch.randn(rows, vocab, generator=g, device="cuda") * 2 + offset
            keep = torch.rand(rows, vocab, generator=g, device="cuda").argsort(-1)[:, :allowed]
            masked = torch.full((rows, vocab), nothing, dtype=dtype, device="cuda")
            masked.scatter_(1, keep, x.gather(1, keep).to(dtype))
            check(masked, keep[:, 0].contiguous(), min(allowed, 20))


@pytest.mark.parametrize("rows,vocab", ROWS)
def test_an_offset_of_the_whole_row(rows, vocab):
    """Some of a row's chunks have a mask and some have none."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    for offset in (0.0, 100.3, -1000.3, 30000.5):
        x = torch.randn(rows, vocab, generator=g, device="cuda") * 2 + offset
        t = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        check(x, t, 20)
        x[:, vocab // 3:vocab // 2] = -math.inf
        t = torch.where((t >= vocab // 3) & (t < vocab // 2), 0, t)
        check(x, t, 20)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", ROWS)
def test_rows_of_one_large_value_are_uniform(dtype, rows, vocab):
    """A mask that leaves nothing may be any large negative number."""
    q4 = lib()
    for value in (-1e9, -1e10, -3e18, 1e30, -1e36, 3e37):
        x = torch.full((rows, vocab), value, dtype=dtype, device="cuda")
        logprob, entropy, best, ids = q4.token_logprobs(x, torch.full((rows,), vocab - 1, device="cuda"), top=3)
        want = math.log(vocab)
        tol = 2 ** -24 * (vocab / 512 + 64 + 16 + 4 * want)
        for got, sign in ((logprob, -1), (best, -1), (entropy, 1)):
            assert ((got.double() - sign * want).abs() <= tol).all(), (value, got.flatten()[:3])
        assert (ids == torch.arange(3, device="cuda")).all()
    assert q4.device_error() == q4.OK


@pytest.mark.parametrize("rows,vocab", ROWS)
def test_neighbours_among_large_values(rows, vocab):
    """One unit in the last place apart is far apart: the larger is certain."""
    q4 = lib()
    for value in (1e10, -1e10, 3e18, 2.02e37, 3.3e38, -3.3e38):
        x = torch.full((rows, vocab), value, device="cuda")
        x[:, vocab - 2] = torch.nextafter(x[0, 0], torch.tensor(math.inf, device="cuda"))
        logprob, entropy, best, ids = q4.token_logprobs(x, torch.full((rows,), vocab - 2, device="cuda"), top=1)
        assert (logprob == 0).all() and (entropy == 0).all() and (best == 0).all(), (value, logprob.max())
        assert (ids == vocab - 2).all()
    assert q4.device_error() == q4.OK
