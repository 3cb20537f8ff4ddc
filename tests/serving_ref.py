"""Plain 64-bit implementations of the operators around the matmuls, and the
paged batches the tests run them on.  Loops over sequences and rows; shares
no code with the library."""
import math

import torch

F64 = torch.float64


class Batch:
    """A ragged batch over a paged cache: `new` and `kv` are the new tokens
    of every sequence and its tokens in the cache, the new ones included."""

    def __init__(self, new, kv, page, kv_heads, dim, seed=0, token_major=False, extra_rows=0, spare=3, width=None,
                 fill=0.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.page, self.kv_heads, self.dim = list(new), list(kv), page, kv_heads, dim
        used = [-(-max(k, 0) // page) for k in self.kv]
        self.pages = sum(used) + spare
        width = width or max(used + [1])
        self.table = torch.full((len(used), width), -1, dtype=torch.int32)
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        at = 0
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_start = torch.tensor([0] + self.new).cumsum(0).to(torch.int32)
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32)
        self.rows = sum(self.new) + extra_rows
        shape = (self.pages, page, kv_heads, dim) if token_major else (self.pages, kv_heads, page, dim)
        self.k = torch.full(shape, fill, dtype=torch.bfloat16)
        self.v = torch.full(shape, fill, dtype=torch.bfloat16)
        if token_major:
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.g = g

    def place(self, b, j):
        """(page, offset) of token j of sequence b."""
        return int(self.table[b, j // self.page]), j % self.page

    def write_tokens(self, scale=1.0):
        """Random keys and values for every token of every sequence."""
        self.tokens = []
        for b, n in enumerate(self.kv):
            n = max(n, 0)
            k = (torch.randn(n, self.kv_heads, self.dim, generator=self.g) * scale).bfloat16()
            v = (torch.randn(n, self.kv_heads, self.dim, generator=self.g) + 0.25).bfloat16()
            self.put(b, k, v)
            self.tokens.append((k, v))
        return self

    def put(self, b, k, v, first=0):
        if not len(k):
            return
        j = torch.arange(first, first + len(k))
        where, offset = self.table[b, j // self.page].long(), j % self.page
        self.k[where, :, offset] = k
        self.v[where, :, offset] = v

    def cuda(self):
        keep = lambda t: t.transpose(1, 2).contiguous().cuda().transpose(1, 2) if not t.is_contiguous() else t.cuda()  # noqa: E731
        self.dev = (keep(self.k), keep(self.v), self.table.cuda(), self.q_start.cuda(), self.kv_len.cuda())
        return self.dev


def rotate(x, cos, sin, interleaved):
    """x [..., rot] float64; cos and sin [rot / 2] of its position."""
    out = x.clone()
    half = x.shape[-1] // 2
    for p in range(half):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        a, b = x[..., i], x[..., j]
        out[..., i], out[..., j] = a * cos[p] - b * sin[p], b * cos[p] + a * sin[p]
    return out


def attention(q, batch, window, sinks, scale):
    """(out, lse, weight) of q [rows, heads, dim]: weight is sum_j p_j |v_j|,
    the scale of the error that rounding the p_j makes; bound is the largest
    sum_i |q_i k_ij| a row meets, the scale of its scores' rounding."""
    rows, heads, dim = q.shape
    group = heads // batch.kv_heads
    out = torch.zeros(rows, heads, dim, dtype=F64, device="cuda")
    weight = torch.zeros_like(out)
    lse = torch.full((rows, heads), -math.inf, dtype=F64, device="cuda")
    bound = torch.zeros(rows, heads, dtype=F64, device="cuda")
    q = q.to("cuda", F64)
    for b, (n, kv) in enumerate(zip(batch.new, batch.kv)):
        row = int(batch.q_start[b])
        if not n or kv <= 0:
            continue
        k, v = (t.to("cuda", F64).repeat_interleave(group, 1) for t in batch.tokens[b])
        j = torch.arange(kv, device="cuda")
        pos = (kv - n + torch.arange(n, device="cuda"))[:, None]
        seen = j <= pos
        if window:
            seen &= (j > pos - window) | (j < sinks)
        qb = q[row:row + n]
        s = torch.einsum("ihd,jhd->hij", qb, k) * scale
        bound[row:row + n] = torch.einsum("ihd,jhd->hij", qb.abs(), k.abs()).amax(-1).T
        s = s.masked_fill(~seen, -math.inf)
        some = seen.any(1)
        p = torch.where(some[:, None], torch.softmax(s, -1), 0.0)
        out[row:row + n] = torch.einsum("hij,jhd->ihd", p, v)
        weight[row:row + n] = torch.einsum("hij,jhd->ihd", p, v.abs())
        lse[row:row + n] = torch.where(some, torch.logsumexp(s, -1), -math.inf).T
    return out, lse, weight, bound


def logprobs(logits, tokens, top):
    """(logprob, entropy, top_logprob, top_ids, spread): spread is
    sum p |x - lse|, the scale of the entropy's rounding."""
    x = logits.double()
    lse = torch.logsumexp(x, -1, keepdim=True)
    value, ids = torch.sort(x + 0.0, dim=-1, descending=True, stable=True)
    logp = x - lse
    p = logp.exp()
    h = torch.where(p > 0, p * logp, 0.0)
    given = logp.gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    return given, -h.sum(-1), (value - lse)[:, :top], ids[:, :top], h.abs().sum(-1)
