"""The 8-bit serving operators of the quantizer, as workloads for measurement.

Three operators, the parts of one attention layer that runs in 8 bits:

* ``linear``    y = (codes(x) @ w_codes^T) * scale(token) * scale(channel) + bias: a matrix
                product in 8-bit integers; the tokens are quantized inside the call.
* ``cache``     keys and values quantized as they are written into a paged cache, with one scale
                for each block of tokens and head, and the blocks that the write touched read back.
* ``attention`` attention over that cache, for single new tokens and for prompt chunks.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the framework's entry points.
Everything is a pure function of (case, seed).

Quantization, both sides: scale = amax / 127, inverse = 1 / scale, code = round-half-even(x *
inverse), every step rounded to 32 bits; where the scale would be below the smallest normal number
it is 0 and the codes are 0.  A cache block's scale never shrinks while its first token stays:
writing behind tokens already there takes the larger of the old and the new scale, and the old
codes c become round(c * (old / new)).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -126


# ------------------------------------------------------------------------------------- cases
def listed():
    lin = {"op": "linear"}
    cache = {"op": "cache"}
    att = {"op": "attention"}
    return [
        # one new token through a 4096 x 4096 projection: the decoding step's latency
        {"name": "linear_one_token", **lin, "tokens": 1, "in": 4096, "out": 4096, "dtype": "bf16",
         "bias": True},
        # a decoding batch through the 11008 -> 4096 down projection, odd token count
        {"name": "linear_batch_37", **lin, "tokens": 37, "in": 11008, "out": 4096,
         "dtype": "fp16", "bias": False},
        # ragged sizes in 32 bits: a small projection of an odd number of tokens
        {"name": "linear_ragged_fp32", **lin, "tokens": 1001, "in": 1032, "out": 520,
         "dtype": "fp32", "bias": True},
        # a prompt through the 28672 -> 8192 down projection: the largest product
        {"name": "linear_prompt", **lin, "tokens": 8192, "in": 28672, "out": 8192,
         "dtype": "bf16", "bias": False},
        # a decoding step of 64 sequences: one token each behind long prefixes
        {"name": "cache_step", **cache, "batch": 64, "new": 1, "before": 4096, "ragged": True,
         "kv_heads": 8, "head_dim": 128, "block": 64, "dtype": "bf16"},
        # four ragged prompts of up to 4096 tokens written into fresh blocks
        {"name": "cache_prompts", **cache, "batch": 4, "new": 4096, "before": 0, "ragged": True,
         "kv_heads": 8, "head_dim": 128, "block": 64, "dtype": "bf16"},
        # odd chunks behind odd prefixes, small blocks and heads, 32-bit keys and values
        {"name": "cache_chunks_fp32", **cache, "batch": 7, "new": 77, "before": 1001,
         "ragged": True, "kv_heads": 2, "head_dim": 64, "block": 16, "dtype": "fp32"},
        # a short chat turn: a few sequences, one token each, latency counts
        {"name": "attention_short", **att, "batch": 3, "new": 1, "len": 130, "ragged": True,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 16, "window": 0, "dtype": "bf16"},
        # a ragged decoding batch (one sequence of it empty), fp16, narrow heads
        {"name": "attention_batch_48", **att, "batch": 48, "new": 1, "len": 8192, "ragged": True,
         "heads": 32, "kv_heads": 8, "head_dim": 64, "block": 32, "window": 0, "dtype": "fp16"},
        # one long document, one new token
        {"name": "attention_long", **att, "batch": 1, "new": 1, "len": 131072, "ragged": False,
         "heads": 64, "kv_heads": 8, "head_dim": 128, "block": 64, "window": 0, "dtype": "bf16"},
        # a prompt chunk of 2048 tokens behind 2048 cached ones
        {"name": "attention_prompt", **att, "batch": 2, "new": 2048, "len": 4096, "ragged": False,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 64, "window": 0, "dtype": "bf16"},
        # odd chunks with a sliding window
        {"name": "attention_window", **att, "batch": 5, "new": 333, "len": 2500, "ragged": True,
         "heads": 16, "kv_heads": 4, "head_dim": 128, "block": 128, "window": 1000,
         "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "cache", "attention", "attention"])
    if op == "linear":
        return {"op": op, "tokens": _log(rng, 1, 8192), "in": 8 * _log(rng, 16, 3584),
                "out": _log(rng, 64, 8192), "dtype": rng.choice(["bf16", "fp16", "fp32"]),
                "bias": rng.random() < 0.5}
    case = {"op": op, "kv_heads": rng.choice([1, 2, 4, 8]), "head_dim": rng.choice([64, 128]),
            "block": rng.choice([16, 32, 64, 128]), "ragged": rng.random() < 0.7}
    if op == "cache":
        batch = _log(rng, 1, 64)
        return {**case, "batch": batch, "new": _log(rng, 1, 16384 // batch),
                "before": rng.choice([0, _log(rng, 1, 4096)]),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    case["dtype"] = rng.choice(["bf16", "fp16"])
    case["heads"] = case["kv_heads"] * rng.choice([1, 2, 4, 8])
    if rng.random() < 0.5:  # single new tokens, or a few guessed ones
        batch = _log(rng, 1, 64)
        length = _log(rng, 8, 131072 // batch)
        new = rng.choice([1, 1, 1, 2, 4])
    else:                   # prompt chunks
        batch = _log(rng, 1, 8)
        new = _log(rng, 5, 4096 // batch)
        length = new + rng.choice([0, _log(rng, 1, 4096)])
    return {**case, "batch": batch, "new": min(new, length), "len": length,
            "window": rng.choice([0, 0, 0, _log(rng, 1, length)])}


def _lengths(case):
    """(new tokens, tokens already cached) of each sequence, from the case alone."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    news, befores = [], []
    for b in range(case["batch"]):
        full = b == 0 or not case["ragged"]
        if case["op"] == "cache":
            n = case["new"] if full or case["new"] == 1 else rng.randint(1, case["new"])
            p = case["before"] if full else rng.randint(0, case["before"])
        else:
            n = case["new"] if full or case["new"] == 1 else rng.randint(1, case["new"])
            total = case["len"] if full else rng.randint(n, case["len"])
            if case["ragged"] and b == 2 and case["batch"] > 8:
                total = n = 0           # a slot of the batch without a request
            p = total - n
        news.append(n)
        befores.append(p)
    return news, befores


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _starts(counts):
    at = [0]
    for c in counts:
        at.append(at[-1] + c)
    return at


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _activations(g, shape, channels):
    """Normal values, with the few loud channels that activations of such layers have."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = torch.rand(channels, generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 20.0, 1.0)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "linear":
        m, k, n = case["tokens"], case["in"], case["out"]
        x = _activations(g, (m, k), k).to(DTYPES[case["dtype"]])
        ld = -(-k // 16) * 16
        w = torch.zeros(n, ld, dtype=torch.int8, device="cuda")
        w[:, :k] = torch.randn(n, k, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127)
        s = 0.02 / 32 * (0.5 + torch.rand(n, generator=g, device="cuda"))
        bias = torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        return {"op": "linear", "x": x, "w": w[:, :k], "w_scale": s, "bias": bias}

    news, befores = _lengths(case)
    totals = [n + p for n, p in zip(news, befores)]
    h, d, blk = case["kv_heads"], case["head_dim"], case["block"]
    width = max(1, -(-max(totals) // blk))
    pages = case["batch"] * width + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:case["batch"] * width]
    table = table.to(torch.int32).reshape(case["batch"], width)
    # the cache as earlier writes left it: every page full, its scale from its own values
    st = {"op": case["op"], "table": table}
    for name in ("k", "v"):
        x = torch.randn((pages, h, blk, d), generator=g, device="cuda")
        if name == "k":
            x *= torch.where(torch.rand((1, h, 1, d), generator=g, device="cuda") < 0.03, 6.0, 1.0)
        scale = x.abs().amax((2, 3)) / 127
        st[name + "_codes"] = x.div_(scale[:, :, None, None]).round_().to(torch.int8)
        st[name + "_scale"] = scale
        del x
    st["lens_before"] = _ints(befores)
    st["lens"] = _ints(totals)
    st["cu"] = _ints(_starts(news))
    st["tokens"] = sum(news)
    st["max_new"], st["max_len"] = max(news), max(totals)
    heads = case.get("heads", 0)
    qkv = _activations(g, (max(1, sum(news)), heads + 2 * h, d), d).to(DTYPES[case["dtype"]])
    qkv = qkv[:sum(news)]       # the projection's output; q, k and v are slices of it
    st["q"], st["k"], st["v"] = qkv[:, :heads], qkv[:, heads:heads + h], qkv[:, heads + h:]
    if case["op"] == "cache":   # read back: every block that the write touches, from its start
        first = [p // blk * blk for p in befores]
        st["read_start"] = _ints(first)
        st["read_cu"] = _ints(_starts([t - f for t, f in zip(totals, first)]))
        st["read_rows"] = sum(t - f for t, f in zip(totals, first))
    else:
        st["window"] = case["window"]
        st["softmax_scale"] = 1 / math.sqrt(d)
    return st


# ---------------------------------------------------------------------------------------- run
def run(st):
    if own:
        return _run_own(st)
    return {"linear": _linear, "cache": _write_read, "attention": _attention}[st["op"]](st)


def _run_own(st):
    import post_int4_weight_gptq_b200 as piq
    if st["op"] == "linear":
        return piq.int8_linear(st["x"], st["w"], st["w_scale"], st["bias"])
    cache = piq.KV8Cache(st["k_codes"], st["v_codes"], st["k_scale"], st["v_scale"])
    if st["op"] == "cache":
        piq.kv8_append(cache, st["k"], st["v"], st["cu"], st["lens_before"], st["table"])
        return piq.kv8_read(cache, st["read_cu"], st["read_start"], st["table"],
                            st["read_rows"], st["k"].dtype)
    return piq.kv8_attention(cache, st["q"], st["cu"], st["lens"], st["table"],
                             st["max_new"], st["max_len"], scale=st["softmax_scale"],
                             window=st["window"], return_lse=True)


def _scale_of(amax):
    # a divisor on the device: a Python number would become a product with its reciprocal
    s = amax / torch.full((), 127.0, device=amax.device)
    return torch.where(s < TINY, torch.zeros_like(s), s)


def _inverse(s):
    return torch.where(s > 0, torch.reciprocal(s), torch.zeros_like(s))


def _linear(st):
    x = st["x"].float()
    sx = _scale_of(x.abs().amax(1))
    codes = (x * _inverse(sx)[:, None]).round_().clamp_(-127, 127)
    y = (codes @ st["w"].float().t()) * sx[:, None] * st["w_scale"][None, :]
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(st["x"].dtype)


def _rows(cu, start, rows):
    """Sequence and position of each of `rows` ragged rows."""
    n = (cu[1:] - cu[:-1]).long()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=cu.device), n, output_size=rows)
    pos = torch.arange(rows, device=cu.device) - cu.long()[seq] + start.long()[seq]
    return seq, pos


def _write_read(st):
    out = []
    before, table = st["lens_before"].long(), st["table"].long()
    blk = st["k_codes"].shape[2]
    seq, pos = _rows(st["cu"], st["lens_before"], st["tokens"])
    page, off = table[seq, pos // blk], pos % blk
    fresh = page[torch.where(off == 0, torch.arange(pos.numel(), device=pos.device), 0)]
    tail = table.gather(1, (before // blk).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    rseq, rpos = _rows(st["read_cu"], st["read_start"], st["read_rows"])
    rpage, roff = table[rseq, rpos // blk], rpos % blk
    grows = (before % blk > 0) & (st["cu"][1:] > st["cu"][:-1])
    for name in ("k", "v"):
        x, codes, scale = st[name].float(), st[name + "_codes"], st[name + "_scale"]
        h = scale.shape[1]
        amax = torch.zeros_like(scale).scatter_reduce_(
            0, page[:, None].expand(-1, h), x.abs().amax(2), "amax")
        old = scale.clone()
        # blocks whose first token is written here start afresh (row 0 stands for "none": it is
        # fresh itself or restored below)
        first = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
        first[fresh] = True
        first[page[0]] = off[0] == 0
        old = torch.where(first[:, None], torch.zeros_like(old), old)
        new = torch.maximum(old, _scale_of(amax))
        # the codes already in a sequence's last block move to the larger scale
        ratio = torch.where(grows[:, None] & (new[tail] > old[tail]) & (new[tail] > 0),
                            old[tail] / new[tail], torch.ones_like(old[tail]))
        part = codes[tail]
        moved = (part.float() * ratio[:, :, None, None]).round_().to(torch.int8)
        codes[tail] = torch.where(grows[:, None, None, None], moved, part)
        scale[page] = new[page]
        codes[page, :, off] = (x * _inverse(new[page])[:, :, None]).round_().clamp_(
            -127, 127).to(torch.int8)
        out.append((codes[rpage, :, roff].float() * scale[rpage][:, :, None]).to(st[name].dtype))
    return out


def _attention(st):
    cu, lens, table = st["cu"].long(), st["lens"].long(), st["table"].long()
    q = st["q"]
    heads, d = q.shape[1], q.shape[2]
    h, blk = st["k_codes"].shape[1], st["k_codes"].shape[2]
    batch, m, length = lens.numel(), st["max_new"], st["max_len"]
    n = cu[1:] - cu[:-1]
    i = torch.arange(m, device=q.device)
    j = torch.arange(length, device=q.device)
    page, off = table[:, j // blk], j % blk                                   # [batch, length]
    k = st["k_codes"][page, :, off[None]].float() * st["k_scale"][page][..., None]
    v = st["v_codes"][page, :, off[None]].float() * st["v_scale"][page][..., None]
    k, v = k.transpose(1, 2), v.transpose(1, 2)                               # [batch, h, len, d]
    rows = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                      # [batch, m]
    qp = q[rows].float().reshape(batch, m, h, heads // h, d).permute(0, 2, 3, 1, 4)
    s = qp.reshape(batch, h, -1, d) @ k.transpose(2, 3) * st["softmax_scale"]
    s = s.reshape(batch, h, heads // h, m, length)
    at = (lens - n)[:, None] + i                                              # query positions
    see = (j <= at[..., None]) & (j < lens[:, None, None])
    if st["window"]:
        see = see & (j > at[..., None] - st["window"])
    s = s.masked_fill(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(batch, h, -1, length) @ v).reshape(batch, h, heads // h, m, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total))[..., 0]
    seq, pos = _rows(st["cu"], torch.zeros_like(st["lens"]), st["tokens"])
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, m, heads, d)[seq, pos]
    return o.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(batch, m, heads)[seq, pos]


# --------------------------------------------------------------------------------------- work
def _pairs(case):
    """(query, key) pairs that see each other, and keys that any query sees, over the batch."""
    pairs = keys = 0
    for n, p in zip(*_lengths(case)):
        w = case["window"] or n + p
        for_all = [min(p + i + 1, w) for i in range(n)]
        pairs += sum(for_all)
        if n:
            keys += n + p - max(0, p + 1 - w)
    return pairs, keys


def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "linear":
        m, k, n = case["tokens"], case["in"], case["out"]
        return {"bytes": m * k * size + n * k + m * n * size + 4 * n * (2 if case["bias"] else 1),
                "flops": 2.0 * m * n * k}
    news, befores = _lengths(case)
    h, d, blk = case["kv_heads"], case["head_dim"], case["block"]
    if case["op"] == "cache":
        back = sum(n + p - p // blk * blk for n, p in zip(news, befores))
        blocks = sum(-(-(n + p) // blk) - p // blk for n, p in zip(news, befores) if n)
        # tokens in, codes out; codes back in, tokens out; a scale each way per block and head
        return {"bytes": 2 * h * (d * (sum(news) * (size + 1) + back * (1 + size)) + 8 * blocks),
                "flops": 2 * h * d * (4.0 * sum(news) + 2.0 * back)}
    pairs, keys = _pairs(case)
    heads, rows = case["heads"], sum(news)
    return {"bytes": 2 * keys * h * d + 8 * keys * h / blk + rows * heads * (2 * d * size + 4),
            "flops": 4.0 * pairs * heads * d}


# -------------------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in 64 bits, one sequence and head at a time."""
    st = prepare(case, seed)
    if case["op"] == "linear":
        x = st["x"].double()
        unit = x.abs().max(dim=1, keepdim=True).values / 127
        codes = torch.where(unit > 0, torch.round(x / unit), 0.0)
        y = codes.mul_(unit) @ (st["w"].double() * st["w_scale"].double()[:, None]).T
        return y if st["bias"] is None else y + st["bias"].double()
    news, befores = _lengths(case)
    blk, table, cu = case["block"], st["table"].tolist(), st["cu"].tolist()
    if case["op"] == "cache":
        outs = []
        for name in ("k", "v"):
            x, codes = st[name].double(), st[name + "_codes"]
            parts = []
            for b, (n, p) in enumerate(zip(news, befores)):
                for first in range(p // blk * blk, n + p, blk):
                    page, lo, hi = table[b][first // blk], max(first, p), min(first + blk, n + p)
                    fresh = x[cu[b] + lo - p:cu[b] + hi - p].transpose(0, 1)      # [h, rows, d]
                    unit = fresh.abs().amax((1, 2), keepdim=True) / 127
                    kept = codes[page, :, :lo - first].double()
                    if lo > first:
                        was = st[name + "_scale"][page].double()[:, None, None]
                        both = torch.maximum(unit, was)
                        kept, unit = torch.round(kept * (was / both)), both
                    new = torch.round(fresh / torch.where(unit > 0, unit, 1.0))
                    parts.append((torch.cat([kept, new], 1) * unit).transpose(0, 1))
            outs.append(torch.cat(parts))
        return outs
    h, heads, d = case["kv_heads"], case["heads"], case["head_dim"]
    q = st["q"].double()
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b, (n, p) in enumerate(zip(news, befores)):
        if n == 0:
            continue
        page = st["table"][b, :-(-(n + p) // blk)].long()
        at = torch.arange(p, n + p, device=q.device)[:, None]
        key = torch.arange(n + p, device=q.device)[None, :]
        hide = key > at
        if case["window"]:
            hide = hide | (key <= at - case["window"])
        for kv in range(h):
            k = st["k_codes"][page, kv].double() * st["k_scale"][page, kv].double()[:, None, None]
            v = st["v_codes"][page, kv].double() * st["v_scale"][page, kv].double()[:, None, None]
            k, v = k.reshape(-1, d)[:n + p], v.reshape(-1, d)[:n + p]
            for head in range(kv * (heads // h), (kv + 1) * (heads // h)):
                s = (q[cu[b]:cu[b + 1], head] @ k.T / math.sqrt(d)).masked_fill(hide, -math.inf)
                z = torch.logsumexp(s, 1)
                o[cu[b]:cu[b + 1], head] = torch.exp(s - z[:, None]) @ v
                lse[cu[b]:cu[b + 1], head] = z
    return o, lse
