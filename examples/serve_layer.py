"""One served decoder layer end to end: Q4_0 matmuls with the operators
between and after them.

    python examples/serve_layer.py [--steps 8] [--window 0] [--sinks 0]

A batch of prompts goes through the layer in one call each of
  matmul(QKV) -> kv_append -> attention -> matmul(O) -> matmul(vocabulary)
  -> token_logprobs,
then every sequence decodes token by token on the same calls.  Weights and
prompts are random (no checkpoint is needed); the layer has 40 query and 8 key
heads of 128 on a hidden size of 5120, the QKV 7168 x 5120 and O 5120 x 5120
matrices of the benchmark.  The last step's log probabilities are compared
with the same layer run on the whole sequences at once, without a cache to
decode from.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import q4_weight_only_gb300 as q4  # noqa: E402

HIDDEN, Q_HEADS, KV_HEADS, DIM, VOCAB, PAGE = 5120, 40, 8, 128, 32000, 16


class Cache:
    """Pages of a key and a value cache, handed out as sequences grow."""

    def __init__(self, sequences, tokens):
        per_sequence = -(-tokens // PAGE)
        pages = sequences * per_sequence
        self.k = torch.empty(pages, KV_HEADS, PAGE, DIM, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(0))
        self.table = order.to(torch.int32).view(sequences, per_sequence).cuda()
        self.length = torch.zeros(sequences, dtype=torch.int32, device="cuda")


def rotation_table(positions):
    freq = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64) / DIM)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class Layer:
    def __init__(self, positions, window, sinks):
        g = torch.Generator(device="cuda").manual_seed(1)
        matrix = lambda n, k: q4.quantize(torch.randn(n, k, generator=g, device="cuda") * 0.02)  # noqa: E731
        self.width = (Q_HEADS + 2 * KV_HEADS) * DIM
        self.qkv, self.o, self.vocab = matrix(self.width, HIDDEN), matrix(HIDDEN, Q_HEADS * DIM), matrix(VOCAB, HIDDEN)
        self.embedding = torch.randn(VOCAB, HIDDEN, generator=g, device="cuda").bfloat16()
        self.cos_sin = rotation_table(positions)
        self.window, self.sinks = window, sinks

    def __call__(self, tokens, lengths, cache):
        """Logits after every new token: `tokens` of all sequences in a row,
        `lengths` of them new in each."""
        starts = torch.tensor([0] + lengths).cumsum(0).to(torch.int32).cuda()
        cache.length += torch.tensor(lengths, dtype=torch.int32, device="cuda")
        batch = (cache.k, cache.v, cache.table, starts, cache.length)
        x = self.embedding[tokens]
        qkv = q4.matmul(x, self.qkv, self.width, HIDDEN)
        q = q4.kv_append(qkv, self.cos_sin, *batch, q_heads=Q_HEADS)
        a = q4.attention(q, *batch, max_q_len=max(lengths), window=self.window, sinks=self.sinks)
        y = q4.matmul(a.view(len(tokens), Q_HEADS * DIM), self.o, HIDDEN, Q_HEADS * DIM, out_dtype=torch.bfloat16)
        return q4.matmul(x + y, self.vocab, VOCAB, HIDDEN)


def main(steps=8, window=0, sinks=0, verbose=True):
    lengths = [37, 5, 300, 128]
    layer = Layer(max(lengths) + steps + 1, window, sinks)
    g = torch.Generator(device="cuda").manual_seed(2)
    texts = [torch.randint(0, VOCAB, (n,), generator=g, device="cuda") for n in lengths]
    cache = Cache(len(texts), max(lengths) + steps + 1)

    # the prompts: each token's log probability after the ones before it
    logits = layer(torch.cat(texts), lengths, cache)
    following = torch.cat([torch.cat([t[1:], t.new_full((1,), -1)]) for t in texts])
    scores, entropy, _, _ = q4.token_logprobs(logits, following)
    ends = torch.tensor(lengths).cumsum(0) - 1
    for i, score in enumerate(scores.split(lengths)):
        if verbose:
            print(f"prompt {i}: {lengths[i]} tokens, log probability {score.sum().item():.2f}, "
                  f"entropy after it {entropy[ends[i]].item():.3f}")

    last = logits[ends.cuda()]
    for step in range(steps):
        # greedy: the best alternative is the next token
        nobody = torch.full((len(texts),), -1, device="cuda")
        _, entropy, best, ids = q4.token_logprobs(last, nobody, top=5)
        texts = [torch.cat([t, i]) for t, i in zip(texts, ids[:, :1])]
        if verbose:
            print(f"step {step}: tokens {ids[:, 0].tolist()}, log probabilities "
                  f"{[round(v, 3) for v in best[:, 0].tolist()]}")
        last = layer(ids[:, 0], [1] * len(texts), cache)

    # the same sequences at once, in a fresh cache
    whole = Cache(len(texts), max(lengths) + steps + 1)
    counts = [len(t) for t in texts]
    logits = layer(torch.cat(texts), counts, whole)[(torch.tensor(counts).cumsum(0) - 1).cuda()]
    tokens = torch.zeros(len(texts), dtype=torch.int64, device="cuda")
    decoded, at_once = (q4.token_logprobs(x, tokens, top=5) for x in (last, logits))
    off = max((a - b).abs().max().item() for a, b in zip(decoded[:3], at_once[:3]))
    if q4.device_error() != q4.OK:
        raise RuntimeError("a kernel reported an error")
    if verbose:
        print(f"decoded against all at once: log probabilities differ by at most {off:.4f}")
    return off


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--window", type=int, default=0)
    p.add_argument("--sinks", type=int, default=0)
    a = p.parse_args()
    main(a.steps, a.window, a.sinks)
