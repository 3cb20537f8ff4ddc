"""The paged batches of serving_ref with a cache in Q4_0 blocks.  Blocks are
made and read by the CPU oracle."""
import numpy as np
import torch

import oracle
import serving_ref as ref

F64 = torch.float64


def blocks(x):
    """(codes, scales) of x [..., dim] fp32: the oracle's blocks, taken apart."""
    n, dim = x.numel() // x.shape[-1], x.shape[-1]
    q = oracle.get().quantize(x.reshape(n, dim).numpy()).reshape(n, dim // 32, 18)
    scales = torch.from_numpy(np.ascontiguousarray(q[..., :2]).view(np.float16)[..., 0].copy())
    codes = torch.from_numpy(np.ascontiguousarray(q[..., 2:]).reshape(n, dim // 2).copy())
    return codes.view(*x.shape[:-1], dim // 2), scales.view(*x.shape[:-1], dim // 32)


def values(codes, scales):
    """What they stand for, by the oracle, in 64 bits."""
    n, dim = codes.numel() // codes.shape[-1], codes.shape[-1] * 2
    q = np.empty((n, dim // 32, 18), dtype=np.uint8)
    q[..., :2] = scales.reshape(n, dim // 32, 1).numpy().view(np.uint8)
    q[..., 2:] = codes.reshape(n, dim // 32, 16).numpy()
    v = oracle.get().dequantize(q.reshape(n, -1), n, dim)
    return torch.from_numpy(v).view(*codes.shape[:-1], dim)


class Batch(ref.Batch):
    """fill: what the slots without a token hold, as (codes, scale)."""

    def __init__(self, new, kv, page, kv_heads, dim, seed=0, token_major=False, extra_rows=0, spare=3, width=None,
                 fill=(0, 0.0)):
        super().__init__(new, kv, page, kv_heads, dim, seed, token_major, extra_rows, spare, width)
        del self.k, self.v
        shape = (self.pages, page, kv_heads) if token_major else (self.pages, kv_heads, page)
        make = lambda: (torch.full((*shape, dim // 2), fill[0], dtype=torch.uint8),                 # noqa: E731
                        torch.full((*shape, dim // 32), fill[1], dtype=torch.float16))
        self.cache = (*make(), *make())
        if token_major:
            self.cache = tuple(t.transpose(1, 2) for t in self.cache)

    def write_tokens(self, scale=1.0):
        """Random keys and values for every token; tokens holds what they
        read back as."""
        self.tokens = []
        for b, n in enumerate(self.kv):
            n = max(n, 0)
            k = torch.randn(n, self.kv_heads, self.dim, generator=self.g) * scale
            v = torch.randn(n, self.kv_heads, self.dim, generator=self.g) + 0.25
            self.tokens.append(self.put(b, k, v))
        return self

    def put(self, b, k, v, first=0):
        if not len(k):
            return k.double(), v.double()
        j = torch.arange(first, first + len(k))
        where, offset = self.table[b, j // self.page].long(), j % self.page
        back = []
        for i, x in ((0, k), (2, v)):
            codes, scales = blocks(x.float())
            self.cache[i][where, :, offset], self.cache[i + 1][where, :, offset] = codes, scales
            back.append(values(codes, scales))
        return tuple(back)

    def cuda(self):
        def keep(t):
            return t.cuda() if t.is_contiguous() else t.transpose(1, 2).contiguous().cuda().transpose(1, 2)

        self.dev = (tuple(keep(t) for t in self.cache), self.table.cuda(), self.q_start.cuda(), self.kv_len.cuda())
        return self.dev
