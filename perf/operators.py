"""Workloads of the operators that surround the matmuls of a served model:

  kv_append       rotate the queries and keys of a fused QKV row by position
                  and append keys and values to a paged cache;
  attention       causal attention over the paged cache, for single tokens,
                  drafts, chunks and whole prompts, optionally with a sliding
                  window and a few first tokens that stay visible;
  token_logprobs  log probability of a given token per row of logits, with
                  the row's entropy and its top alternatives.

listed() holds the fixed cases, draw() gives more of the same ranges,
prepare() makes what a program holds before the call, run() is one pass (the
plain form in torch operations, or the library's kernels when `own` is true),
work() counts the bytes and operations the operator cannot do without and
exact() evaluates its definition in 64 bits.

The head layout 40 / 8 x 128 is that of the QKV 7168 x 5120 and O 5120 x 5120
matrices this library's benchmark runs; the 256 + 16 row batch is its chunked
workload.
"""
import math
import random

import torch

own = False

ROPE_BASE = 10000.0


# --------------------------------------------------------------------- cases

def _batch(chunks, chunk_len, decodes, draft, context, ragged, q_heads=40, kv_heads=8, head_dim=128, page=16,
           head_major=True):
    """A batch of `chunks` sequences that bring up to chunk_len new tokens each
    and `decodes` sequences that bring `draft`, all with up to `context`
    tokens in the cache already (exactly as many when not ragged)."""
    return {"chunks": chunks, "chunk_len": chunk_len, "decodes": decodes, "draft": draft, "context": context,
            "ragged": ragged, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "head_major": head_major}


def _append(rot, interleaved, dtype, **batch):
    return {"op": "kv_append", "rot": rot, "interleaved": interleaved, "dtype": dtype, **batch}


def _attention(window, sinks, **batch):
    return {"op": "attention", "window": window, "sinks": sinks, **batch}


def _logprobs(rows, vocab, top, dtype, masked=0.0):
    return {"op": "token_logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype, "masked": masked}


def listed():
    return [
        # one decode step of 16 running requests: a few KB a row, all latency
        {"name": "append_decode_16", **_append(128, False, "float32", **_batch(0, 0, 16, 1, 700, True))},
        # a 256-token prompt chunk that shares its step with 16 decoding requests
        {"name": "append_chunk_272", **_append(128, False, "bfloat16", **_batch(1, 256, 16, 1, 500, True, page=32,
                                                                               head_major=False))},
        # a long prompt in one call, interleaved pairs on half of each head, odd length
        {"name": "append_prompt_8191", **_append(64, True, "float32", **_batch(1, 8191, 0, 1, 0, False, page=64))},
        # one user waiting for the next token of a short conversation: latency
        {"name": "attend_decode_1", **_attention(0, 0, **_batch(0, 0, 1, 1, 2047, False))},
        # 16 running requests of mixed lengths
        {"name": "attend_decode_16", **_attention(0, 0, **_batch(0, 0, 16, 1, 8192, True))},
        # 64 long requests under a sliding window with visible first tokens
        {"name": "attend_decode_64_window", **_attention(4096, 4, **_batch(0, 0, 64, 1, 32768, True, page=64,
                                                                          head_major=False))},
        # the chunked step: a 256-token chunk deep in a prompt and 16 decoding requests
        {"name": "attend_chunk_272", **_attention(0, 0, **_batch(1, 256, 16, 1, 8000, True, page=32))},
        # several prompts at once, narrow heads, a window shorter than the prompts
        {"name": "attend_prompts_window", **_attention(1000, 5, **_batch(4, 4096, 0, 1, 0, True, 24, 4, 64, 128))},
        # the second half of a long prompt, every earlier token visible
        {"name": "attend_prompt_8192", **_attention(0, 0, **_batch(1, 8192, 0, 1, 8192, False, page=64))},
        # the token just sampled and its five best alternatives
        {"name": "logprobs_1", **_logprobs(1, 32000, 5, "float32")},
        # a decode step that returns alternatives, odd vocabulary, most of it ruled out by a grammar
        {"name": "logprobs_16", **_logprobs(16, 128257, 20, "bfloat16", 0.9)},
        # scoring the tokens of a prompt
        {"name": "logprobs_2048", **_logprobs(2048, 131072, 20, "float32")},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        m = most.setdefault(c["op"], {"bytes": 0, "flops": 0})
        for k in m:
            m[k] = max(m[k], w[k])
    while True:
        c = _draw(rng)
        w, m = work(c), most[c["op"]]
        if w["bytes"] <= m["bytes"] and w["flops"] <= m["flops"] and _plain_scores(c) <= _plain_scores(_LARGEST):
            return c


def _draw(rng):
    op = rng.choice(["kv_append", "attention", "attention", "token_logprobs"])
    if op == "token_logprobs":
        return _logprobs(_log_int(rng, 1, 2048), _log_int(rng, 1000, 200000), rng.choice([0, 1, 5, 20, 32]),
                         rng.choice(["float32", "bfloat16"]), rng.choice([0.0, 0.0, 0.9]))
    q_heads, kv_heads, head_dim = rng.choice([(40, 8, 128), (32, 8, 128), (24, 4, 64), (28, 4, 128), (8, 8, 128),
                                              (16, 1, 64), (64, 8, 64), (6, 2, 128)])
    kind = rng.choice(["decode", "draft", "mixed", "prompt"])
    context = 0 if kind == "prompt" and rng.random() < 0.5 else _log_int(rng, 16, 1500 if op == "kv_append" else 33000)
    chunks, chunk_len, decodes, draft = 0, 0, 0, 1
    if kind in ("mixed", "prompt"):
        chunks, chunk_len = rng.randint(1, 4), _log_int(rng, 17, 8192)
    if kind != "prompt":
        decodes = _log_int(rng, 1, 128)
        draft = rng.randint(2, 7) if kind == "draft" else 1
    batch = _batch(chunks, chunk_len, decodes, draft, context, rng.random() < 0.8, q_heads, kv_heads, head_dim,
                   rng.choice([16, 32, 48, 64, 128, 256]), rng.random() < 0.5)
    if op == "kv_append":
        return _append(rng.choice([head_dim, head_dim // 2]), rng.random() < 0.5, rng.choice(["float32", "bfloat16"]),
                       **batch)
    window = 0 if rng.random() < 0.5 else _log_int(rng, 64, 8192)
    return _attention(window, rng.choice([0, 1, 4, 100]) if window else 0, **batch)


def _lengths(case):
    """(new tokens, tokens in the cache after them) of every sequence."""
    rng = random.Random("%(chunks)d %(chunk_len)d %(decodes)d %(draft)d %(context)d" % case)
    new, kv = [], []
    for i in range(case["chunks"] + case["decodes"]):
        n, before = (case["chunk_len"] if i < case["chunks"] else case["draft"]), case["context"]
        if case["ragged"]:
            before = rng.randint(before // 8, before)
            if i < case["chunks"] and case["chunks"] > 1:
                n = rng.randint(max(1, n // 4), n)
        new.append(n)
        kv.append(before + n)
    return new, kv


def _plain_scores(case):
    """Scores the plain form holds at once (it pads each group of a batch)."""
    if case["op"] != "attention":
        return 0
    new, kv = _lengths(case)
    c = case["chunks"]
    groups = [(n, k) for n, k in ((new[:c], kv[:c]), (new[c:], kv[c:])) if n]
    return case["q_heads"] * max(len(n) * max(n) * max(k) for n, k in groups)


_LARGEST = {"op": "attention", **_batch(1, 8192, 0, 1, 8192, False)}


def _visible(n, kv, window, sinks):
    """(query, key) pairs that see each other, and keys some query sees."""
    first = kv - n
    if not window:
        return sum(range(first + 1, kv + 1)), kv
    pairs = 0
    for p in range(first, kv):
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, first - window + 1)
    return pairs, kv - lo + min(sinks, lo)


def work(case):
    if case["op"] == "token_logprobs":
        size = 4 if case["dtype"] == "float32" else 2
        rows, vocab, top = case["rows"], case["vocab"], case["top"]
        # per logit: a compare, a difference, an exponential, its sum and the entropy's product and sum
        return {"bytes": rows * (vocab * size + 8 + 8 + top * 12), "flops": rows * vocab * 6}
    new, kv = _lengths(case)
    rows, hq, hk, d = sum(new), case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "kv_append":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": rows * ((hq + 2 * hk) * d * (size + 2) + case["rot"] * 4),
                "flops": rows * (hq + hk) * case["rot"] * 3}
    pairs, keys = map(sum, zip(*(_visible(n, k, case["window"], case["sinks"]) for n, k in zip(new, kv))))
    return {"bytes": rows * hq * d * 4 + keys * hk * d * 4, "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------------- inputs

def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "token_logprobs":
        rows, vocab = case["rows"], case["vocab"]
        # logits of a trained model: a broad bulk and a row temperature that makes some rows nearly sure
        logits = _normal(g, rows, vocab) * (1.0 + 2.0 * torch.rand(rows, 1, generator=g, device="cuda"))
        if case["masked"]:  # a grammar's mask: the ruled-out tokens are -inf, the given token is not
            logits[torch.rand(rows, vocab, generator=g, device="cuda") < case["masked"]] = -math.inf
        tokens = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        logits[torch.arange(rows, device="cuda"), tokens] = 2.0 + _normal(g, rows)
        return {"case": case, "logits": logits.to(getattr(torch, case["dtype"])), "tokens": tokens}
    new, kv = _lengths(case)
    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    pages = [-(-n // page) for n in kv]
    total = sum(pages) + 3
    used = torch.arange(max(pages))[None] < torch.tensor(pages)[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32)
    order = torch.randperm(total, generator=g, device="cuda").cpu().to(torch.int32)
    table[used] = order[:sum(pages)]
    # keys and values have channels with a mean of their own
    shape = (total, hk, page, d) if case["head_major"] else (total, page, hk, d)
    k_cache = (_normal(g, *shape, dtype=torch.bfloat16) + 0.5 * _normal(g, d).bfloat16())
    v_cache = (_normal(g, *shape, dtype=torch.bfloat16) + 0.5 * _normal(g, d).bfloat16())
    if not case["head_major"]:
        k_cache, v_cache = k_cache.transpose(1, 2), v_cache.transpose(1, 2)
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    state = {"case": case, "new": new, "kv": kv, "k_cache": k_cache, "v_cache": v_cache, "page_table": table.cuda(),
             "q_start": starts.cuda(), "kv_len": torch.tensor(kv, dtype=torch.int32).cuda()}
    rows = sum(new)
    if case["op"] == "kv_append":
        rot = case["rot"]
        freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        angle = torch.arange(max(kv), dtype=torch.float64)[:, None] * freq
        state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        state["qkv"] = _normal(g, rows, (hq + 2 * hk) * d).to(getattr(torch, case["dtype"]))
    else:
        # heads from nearly uniform to sharp
        state["q"] = (_normal(g, rows, hq, d) * torch.linspace(0.3, 2.0, hq, device="cuda")[:, None]).bfloat16()
    return state


# ---------------------------------------------------------------------- runs

def run(state):
    if own:
        return _run_own(state)
    return {"kv_append": _append_plain, "attention": _attention_plain,
            "token_logprobs": _logprobs_plain}[state["case"]["op"]](state)


def _run_own(s):
    import q4_weight_only_gb300 as q4
    c = s["case"]
    if c["op"] == "token_logprobs":
        return q4.token_logprobs(s["logits"], s["tokens"], top=c["top"])
    if c["op"] == "kv_append":
        q = q4.kv_append(s["qkv"], s["cos_sin"], s["k_cache"], s["v_cache"], s["page_table"], s["q_start"],
                         s["kv_len"], q_heads=c["q_heads"], interleaved=c["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    return q4.attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["q_start"], s["kv_len"],
                        max_q_len=max(s["new"]), window=c["window"], sinks=c["sinks"])


def _row_places(s, rows):
    """Position and cache slot (page, offset) of every row of the batch."""
    r = torch.arange(rows, dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(s["q_start"][1:], r, right=True)
    pos = (s["kv_len"][seq] - s["q_start"][seq + 1] + r).long()
    return pos, s["page_table"][seq, pos // s["case"]["page"]].long(), pos % s["case"]["page"]


def _rotate(x, cos, sin, interleaved):
    """x [rows, heads, rot], cos and sin [rows, 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _append_plain(s):
    c = s["case"]
    hq, hk, d, rot = c["q_heads"], c["kv_heads"], c["head_dim"], c["rot"]
    x = s["qkv"].float().view(-1, hq + 2 * hk, d)
    pos, page, offset = _row_places(s, x.shape[0])
    cos, sin = s["cos_sin"][pos][:, None].chunk(2, -1)
    qk = torch.cat([_rotate(x[:, :hq + hk, :rot], cos, sin, c["interleaved"]), x[:, :hq + hk, rot:]], -1).bfloat16()
    s["k_cache"][page, :, offset] = qk[:, hq:]
    s["v_cache"][page, :, offset] = x[:, hq + hk:].bfloat16()
    return qk[:, :hq].contiguous(), s["k_cache"], s["v_cache"]


def _attention_plain(s):
    new, c = s["new"], s["case"]["chunks"]
    parts = [_attend(s, lo, hi) for lo, hi in ((0, c), (c, len(new))) if hi > lo]
    return torch.cat(parts)


def _attend(s, lo, hi):
    """Sequences lo .. hi - 1, padded to the longest of them."""
    c, table = s["case"], s["page_table"][lo:hi]
    new, longest = max(s["new"][lo:hi]), max(s["kv"][lo:hi])
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    n, kv = (s["q_start"][lo + 1:hi + 1] - s["q_start"][lo:hi]).long(), s["kv_len"][lo:hi].long()
    i = torch.arange(new, device="cuda")
    real = i < n[:, None]
    pos = (kv - n)[:, None] + i
    rows = (s["q_start"][lo:hi].long()[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(hi - lo, new, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(hi - lo, hk, -1, d)
    j = torch.arange(longest, device="cuda")
    page = table[:, j // c["page"]].clamp(min=0).long()
    seen = (j <= pos[..., None]) & (j < kv[:, None, None])
    if c["window"]:
        seen &= (j > pos[..., None] - c["window"]) | (j < c["sinks"])
    k = s["k_cache"][page, :, j % c["page"]].float().transpose(1, 2)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5).view(hi - lo, hk, hq // hk, new, longest)
    w.masked_fill_(~seen[:, None, None], -math.inf)
    w.sub_(w.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = w.sum(-1, keepdim=True)
    v = s["v_cache"][page, :, j % c["page"]].float().transpose(1, 2)
    out = torch.matmul(w.view(hi - lo, hk, -1, longest), v).view(hi - lo, hk, hq // hk, new, d) / total
    return out.permute(0, 3, 1, 2, 4).reshape(hi - lo, new, hq, d)[real].bfloat16()


def _logprobs_plain(s):
    x, top = s["logits"].float(), s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(-1, keepdim=True)
    lse = m + total.log()
    logprob = x.gather(1, s["tokens"][:, None]) - lse
    p = e / total
    entropy = -(p * (x - lse).clamp(min=-3e38)).sum(-1)
    # a stable sort leaves the lowest id first among equal logits
    value, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    return logprob[:, 0], entropy, value[:, :top] - lse, ids[:, :top].clone()


# --------------------------------------------------------------------- exact

def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "token_logprobs":
        return _logprobs_exact(s)
    c = s["case"]
    hq, hk, d, page = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    table = s["page_table"].cpu().long()
    if case["op"] == "kv_append":
        x = s["qkv"].double().view(-1, hq + 2 * hk, d)
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        half = c["rot"] // 2
        first = torch.arange(half) * 2 if c["interleaved"] else torch.arange(half)
        second = first + (1 if c["interleaved"] else half)
        row = 0
        for b, (n, kv) in enumerate(zip(s["new"], s["kv"])):
            p = torch.arange(kv - n, kv)
            cs = s["cos_sin"][p.cuda()].double()
            turn = torch.complex(cs[:, None, :half].contiguous(), cs[:, None, half:].contiguous())
            part = x[row:row + n]
            z = torch.complex(part[:, :hq + hk, first.cuda()], part[:, :hq + hk, second.cuda()]) * turn
            part[:, :hq + hk, first.cuda()], part[:, :hq + hk, second.cuda()] = z.real, z.imag
            where, offset = table[b, p // page].cuda(), (p % page).cuda()
            k_cache[where, :, offset] = part[:, hq:hq + hk]
            v_cache[where, :, offset] = part[:, hq + hk:]
            row += n
        return x[:, :hq].contiguous(), k_cache, v_cache
    out, row = [], 0
    for b, (n, kv) in enumerate(zip(s["new"], s["kv"])):
        j = torch.arange(kv, device="cuda")
        where = table[b].cuda()[j // page]
        k = s["k_cache"][where, :, j % page].double().permute(1, 2, 0)
        v = s["v_cache"][where, :, j % page].double().permute(1, 0, 2)
        for i in range(0, n, 512):
            m = min(512, n - i)
            q = s["q"][row + i:row + i + m].double().view(m, hk, hq // hk, d)
            pos = (kv - n + i + torch.arange(m, device="cuda"))[:, None]
            hidden = j > pos
            if c["window"]:
                hidden |= (pos - j >= c["window"]) & (j >= c["sinks"])
            score = (q.permute(1, 2, 0, 3).reshape(hk, -1, d) @ k / math.sqrt(d)).view(hk, -1, m, kv)
            prob = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out.append((prob.view(hk, -1, kv) @ v).view(hk, -1, m, d).permute(2, 0, 1, 3).reshape(m, hq, d))
        row += n
    return torch.cat(out)


def _logprobs_exact(s):
    parts = []
    for lo in range(0, s["logits"].shape[0], 128):
        x, t = s["logits"][lo:lo + 128].double(), s["tokens"][lo:lo + 128]
        logp = torch.log_softmax(x, -1)
        entropy = -torch.where(logp > -math.inf, logp.exp() * logp, 0.0).sum(-1)
        value, ids = torch.sort(logp, dim=-1, descending=True, stable=True)
        top = s["case"]["top"]
        parts.append((logp.gather(1, t[:, None])[:, 0], entropy, value[:, :top].clone(), None))
    columns = list(zip(*parts))
    return tuple(torch.cat(c) for c in columns[:3]) + (None,)
