"""The 4-bit key/value cache: storing tokens, reading them back and attending over them.

A cache holds the keys and the values of its tokens in pages of `page` token
rows.  A page keeps, for each head, `page` rows of D codes (two 4-bit codes a
byte, the even element in the low half) and one bf16 scale for each run of 64
elements:

    codes  uint8 [pages, kv_heads, page, D / 2]
    scales bf16  [pages, kv_heads, page, D / 64]

once for the keys and once for the values.  Token `slot` is row slot % page of
page slot / page.

Storing a run x of 64 elements: the scale s is the run's largest magnitude
rounded to bf16 (to the largest finite bf16 at most; 0 where the magnitude is
below 2^-126, NaN where it is not finite), and each element's code is that of
the level next to fl(x fl(1 / s)) in 32 bits, the lower one on a tie (fl(0)
where s = 0).  An element stands for level[code] * s.

Attention: query i of the n_b queries of sequence b stands at position
p = length_b - n_b + i.  It sees key positions j <= p (causal; every j <
length_b otherwise) with j > p - window where a window is set, and its output
is sum_j softmax_j(scale q.k_j) v_j; zero where it sees none.
"""

import math
import random
from statistics import NormalDist

import numpy as np
import torch

own = False

BLOCK = 64
TABLES = {"nf4": 0, "uniform": 1, "fp4": 2}
TINY = 2.0 ** -126          # the smallest normal number in 32 bits
BF16_MAX = 3.3895313892515355e38


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token each of four sequences: a call's own cost
        dict(name="write_4_tokens", op="write", tokens=4, heads=8, dim=128, page=64, table="nf4", dtype="bf16",
             fused=True, padded=False),
        # one decode step of a batch of 64 on 32 heads of 128 (4096 wide)
        dict(name="write_64_tokens", op="write", tokens=64, heads=32, dim=128, page=64, table="nf4", dtype="bf16",
             fused=True, padded=False),
        # a padded batch of short prompts, every sixth token padding, 32-bit activations, narrow heads
        dict(name="write_1537_f32_d64", op="write", tokens=1537, heads=12, dim=64, page=16, table="uniform",
             dtype="f32", fused=False, padded=True),
        # a whole prompt of 4096 tokens on 32 heads of 128
        dict(name="write_4096_tokens", op="write", tokens=4096, heads=32, dim=128, page=64, table="nf4",
             dtype="bf16", fused=True, padded=False),
        # a few tokens moved out of a cache with wide heads, in 32 bits
        dict(name="read_131_f32_d256", op="read", tokens=131, heads=5, dim=256, page=32, table="fp4", dtype="f32",
             padded=True),
        # a long shared prefix read back for other use
        dict(name="read_32768_tokens", op="read", tokens=32768, heads=8, dim=128, page=64, table="nf4",
             dtype="bf16", padded=False),
        # single-token decode, one sequence, 32 heads with keys of their own
        dict(name="decode_1x700_mha", op="attention", seqs=1, queries=1, length=700, heads=32, kv_heads=32, dim=128,
             page=64, table="nf4", causal=True, window=0, ragged=False, fused=True),
        # single-token decode of a batch of 32 sequences of very different lengths, 64 heads on 8
        dict(name="decode_32x4096_gqa", op="attention", seqs=32, queries=1, length=4096, heads=64, kv_heads=8,
             dim=128, page=64, table="nf4", causal=True, window=0, ragged=True, fused=True),
        # two very long contexts
        dict(name="decode_2x131072_gqa", op="attention", seqs=2, queries=1, length=131072, heads=64, kv_heads=8,
             dim=128, page=128, table="nf4", causal=True, window=0, ragged=False, fused=True),
        # five proposed tokens a sequence checked at once, narrow heads, a window
        dict(name="verify_8x5x2900_d64", op="attention", seqs=8, queries=5, length=2900, heads=32, kv_heads=4, dim=64,
             page=16, table="uniform", causal=True, window=1024, ragged=False, fused=False),
        # the last 2048 tokens of an 8192-token prompt against all of it, 32 heads of 128
        dict(name="prompt_2048_of_8192", op="attention", seqs=1, queries=2048, length=8192, heads=32, kv_heads=32,
             dim=128, page=64, table="nf4", causal=True, window=0, ragged=False, fused=True),
        # a mixed batch of short prompts, wide heads
        dict(name="prompt_6x1500_d256", op="attention", seqs=6, queries=1500, length=1500, heads=16, kv_heads=4,
             dim=256, page=32, table="fp4", causal=True, window=0, ragged=True, fused=False),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    table = rng.choice(["nf4", "nf4", "uniform", "fp4"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    if op != "attention":
        most = 4096 * 32 * 128 if op == "write" else 32768 * 8 * 128
        heads = spread(rng, 1, 32)
        return dict(op=op, tokens=spread(rng, 1, most // (heads * dim)), heads=heads, dim=dim, page=page, table=table,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), padded=rng.random() < 0.3,
                    **({"fused": rng.random() < 0.5} if op == "write" else {}))
    kv_heads = spread(rng, 1, 32)
    heads = kv_heads * rng.choice([g for g in (1, 1, 2, 3, 4, 7, 8, 16) if g * kv_heads <= 128])
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "prompt":
        seqs = spread(rng, 1, 8)
        length = spread(rng, 32, 8192)
        queries = spread(rng, min(length, 32), min(length, 2048))
    else:
        seqs = spread(rng, 1, 64)
        length = spread(rng, 1, 131072)
        queries = 1 if kind == "decode" else min(length, rng.randint(2, 16))
    # no dearer than the largest listed cases
    length = max(1, min(length, 2 * 131072 * 8 * 128 // (seqs * kv_heads * dim)))
    queries = max(1, min(queries, length, 2048 * 8192 * 32 * 128 // (seqs * heads * dim * length)))
    return dict(op="attention", seqs=seqs, queries=queries, length=length, heads=heads, kv_heads=kv_heads, dim=dim,
                page=page, table=table, causal=rng.random() < 0.9, window=spread(rng, 16, 4096) if rng.random() < 0.2 else 0,
                ragged=rng.random() < 0.6, fused=rng.random() < 0.5)


def lengths_of(case):
    """(lengths, queries) of the sequences of an attention case."""
    n, most, q = case["seqs"], case["length"], case["queries"]
    if not case["ragged"]:
        return [most] * n, [q] * n
    lengths = [most] + [1 + int((most - 1) * (0.6180339887 * b % 1.0)) for b in range(1, n)]
    return lengths, [min(t, 1 + int((q - 1) * (1.0 if b == 0 else 0.3819660113 * (b + 1) % 1.0)))
                     for b, t in enumerate(lengths)]


def work(case):
    D, row = case["dim"], case["dim"] // 2 + 2 * (case["dim"] // BLOCK)
    if case["op"] != "attention":
        kept = len(kept_tokens(case))
        wide = 2 if case["dtype"] == "bf16" else 4
        n = 2 * case["heads"] * kept
        # write: the tokens in, the cache rows out, and these back again as values; read: rows in, values out
        return {"bytes": n * (D * wide * (2 if case["op"] == "write" else 1) + row), "flops": 0}
    rows = pairs = 0
    for length, queries in zip(*lengths_of(case)):
        first = length - queries
        low = np.maximum(first + np.arange(queries) - case["window"] + 1, 0) if case["window"] else np.zeros(queries, int)
        high = first + np.arange(queries) + 1 if case["causal"] else np.full(queries, length)
        pairs += int(np.sum(high - low))
        rows += int(high.max() - low.min())
    tokens = sum(lengths_of(case)[1])
    return {"bytes": 2 * rows * case["kv_heads"] * row + 2 * 2 * tokens * case["heads"] * D,
            "flops": 4 * pairs * case["heads"] * D}


# ------------------------------------------------------------------ inputs

def levels(table):
    """The 16 levels of a code table, in 32 bits: the normal distribution's quantiles, a uniform grid, 4-bit floats."""
    if table == "nf4":
        at = NormalDist().inv_cdf
        top = 0.9677083
        v = [at(0.5 + (top - 0.5) * i / 8) for i in range(1, 9)] + [-at(0.5 + (top - 0.5) * i / 7) for i in range(1, 8)]
        v = np.sort(np.array(v + [0.0]))
    elif table == "uniform":
        v = np.linspace(-1.0, 1.0, 16)
    else:
        half = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
        v = np.concatenate([-half[::-1], half]) + 0.0
    return (v / np.max(np.abs(v))).astype(np.float32)


def edges(table):
    """The largest numbers in 32 bits at or below the midpoints between the levels: a quotient above one has a higher code."""
    v = levels(table).astype(np.float64)
    mid = (v[1:] + v[:-1]) / 2
    e = mid.astype(np.float32)
    return np.where(e.astype(np.float64) > mid, np.nextafter(e, np.float32(-np.inf)), e)


def quantise(x, edge):
    """(codes, scales) of x [..., D] in 32 bits, by the rule at the top of this file."""
    runs = x.unflatten(-1, (-1, BLOCK))
    top = runs.abs().amax(-1)
    scale = torch.where(top < TINY, torch.zeros_like(top), top.clamp(max=BF16_MAX))
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(top, math.nan)).to(torch.bfloat16)
    s = scale.float()
    r = torch.where(s == 0, torch.zeros_like(s), 1.0 / s)
    code = torch.bucketize(runs * r.unsqueeze(-1), edge).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def values(codes, scales, level):
    """The numbers in 32 bits that packed codes [..., D / 2] and their scales [..., D / 64] stand for."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).int()
    return (level[c].unflatten(-1, (-1, BLOCK)) * scales.float().unsqueeze(-1)).flatten(-2)


def kept_tokens(case):
    return [t for t in range(case["tokens"]) if not (case["padded"] and t % 6 == 5)]


def tokens_like(g, tokens, heads, dim, dev):
    """Keys with a few strong channels, and values."""
    gain = torch.exp(0.5 * torch.randn((heads, dim), generator=g, device=dev))
    gain = gain / gain.square().mean(-1, keepdim=True).sqrt()
    return (torch.randn((tokens, heads, dim), generator=g, device=dev) * gain,
            torch.randn((tokens, heads, dim), generator=g, device=dev))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    host = random.Random(seed)
    D, page, table = case["dim"], case["page"], case["table"]
    s = dict(case)
    s["level"] = torch.from_numpy(levels(table)).to(dev)
    s["edge"] = torch.from_numpy(edges(table)).to(dev)
    if case["op"] == "attention":
        heads = case["kv_heads"]
        lengths, queries = lengths_of(case)
        need = [-(-t // page) for t in lengths]
    else:
        heads = case["heads"]
        need = [-(-case["tokens"] // page)]
    pages = sum(need) + 2
    # the pages hold tokens of other sequences before: the cache as a server has it
    parts = []
    step = max(1, (1 << 27) // (page * heads * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        parts.append([])
        for x in tokens_like(g, n * page, heads, D, dev):
            parts[-1] += quantise(x.unflatten(0, (n, page)).transpose(1, 2).contiguous(), s["edge"])
    s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"] = (torch.cat(p) for p in zip(*parts))
    order = list(range(pages))
    host.shuffle(order)
    if case["op"] != "attention":
        n = case["tokens"]
        row = torch.arange(n, device=dev)
        slots = torch.tensor(order, device=dev)[row // page] * page + row % page
        kept = torch.tensor(kept_tokens(case), device=dev)
        s["slots"] = torch.full((n,), -1, dtype=torch.int32, device=dev)
        s["slots"][kept] = slots[kept].int()
        s["kept"] = kept
        if case["op"] == "write":
            dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
            k, v = (x.to(dtype) for x in tokens_like(g, n, heads, D, dev))
            if case["fused"]:  # slices of one projection's output, queries first
                both = torch.cat([torch.zeros_like(k), k, v], 1)
                k, v = both[:, heads:2 * heads], both[:, 2 * heads:]
            s["k"], s["v"] = k, v
        return s
    table_of = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table_of[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    s["block_table"] = table_of.to(dev)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    starts = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
    s["q_starts"] = torch.from_numpy(starts).to(dev)
    s["max_q"], s["max_len"], tokens = max(queries), max(lengths), int(starts[-1])
    q = torch.randn((tokens, case["heads"], D), generator=g, device=dev).to(torch.bfloat16)
    if case["fused"]:
        q = torch.cat([q, torch.zeros((tokens, 2 * heads, D), dtype=q.dtype, device=dev)], 1)[:, :case["heads"]]
    s["q"] = q
    return s


# ------------------------------------------------------------------ one pass

def plain_write(s):
    page = s["page"]
    at = s["slots"][s["kept"]].long()
    for name in ("k", "v"):
        codes, scales = quantise(s[name].float(), s["edge"])
        s[name + "_codes"][at // page, :, at % page] = codes[s["kept"]]
        s[name + "_scales"][at // page, :, at % page] = scales[s["kept"]]


def plain_read(s):
    page, at = s["page"], s["slots"].long()
    there = (at >= 0).view(-1, 1, 1)
    at = at.clamp(min=0)
    dtype = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    return tuple(torch.where(there, values(s[n + "_codes"][at // page, :, at % page],
                                           s[n + "_scales"][at // page, :, at % page], s["level"]), 0.0).to(dtype)
                 for n in ("k", "v"))


def plain_attention(s):
    page, D, group = s["page"], s["dim"], s["heads"] // s["kv_heads"]
    n, most, width = s["seqs"], s["max_q"], s["max_len"]
    dev = s["q"].device
    starts, lengths = s["q_starts"].long(), s["lengths"].long()
    counts = starts[1:] - starts[:-1]
    key = torch.arange(width, device=dev)
    pages = s["block_table"][:, key // page].long().clamp(min=0)                     # [n, width]
    i = torch.arange(most, device=dev)
    token = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)                   # [n, most]
    pos = lengths[:, None] - counts[:, None] + i
    sees = key < lengths[:, None, None]
    if s["causal"]:
        sees = sees & (key <= pos[:, :, None])
    if s["window"]:
        sees = sees & (key > pos[:, :, None] - s["window"])
    sees = sees[:, None, None]                                                        # [n, 1, 1, most, width]
    k, v = (values(s[m + "_codes"][pages, :, key % page], s[m + "_scales"][pages, :, key % page], s["level"])
            .transpose(1, 2) for m in ("k", "v"))                                     # [n, kv_heads, width, D]
    q = s["q"][token].float().view(n, most, s["kv_heads"], group, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(n, s["kv_heads"], group * most, D) * D ** -0.5
    x = (q @ k.transpose(-1, -2)).view(n, s["kv_heads"], group, most, width)
    x = x.masked_fill_(~sees, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp_(x.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)))
    total = x.sum(-1, keepdim=True)
    x = x.view(n, s["kv_heads"], group * most, width) @ v.masked_fill((key >= lengths[:, None])[:, None, :, None], 0.0)
    x = x.view(n, s["kv_heads"], group, most, D) / torch.where(total == 0, torch.ones_like(total), total)
    x = x.permute(0, 3, 1, 2, 4).reshape(n, most, s["heads"], D)
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(starts, t, right=True) - 1
    return x[b, t - starts[b]].to(torch.bfloat16)


def run(state):
    s = state
    if not own:
        if s["op"] == "attention":
            return plain_attention(s)
        if s["op"] == "write":
            plain_write(s)
        return plain_read(s)
    import bit_nf4_quantized_quant_amd as qa
    cache = s.get("cache")
    if cache is None:
        cache = s["cache"] = qa.KVCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], TABLES[s["table"]])
    if s["op"] == "attention":
        out, _ = qa.kv_attention(s["q"], cache, s["block_table"], s["lengths"], s["q_starts"], s["max_q"], s["max_len"],
                                 causal=s["causal"], window=s["window"])
        return out
    dtype = torch.bfloat16 if s["dtype"] == "bf16" else torch.float32
    if s["op"] == "write":
        qa.kv_write(s["k"], s["v"], cache, s["slots"])
    return qa.kv_read(cache, s["slots"], dtype)


# ------------------------------------------------------------------ in 64 bits

def exact_rows(s, name, slots):
    """Rows [n, heads, D] of the cache in 64 bits, by a table of byte pairs, some tokens at a time."""
    if len(slots) > 16384:
        return torch.cat([exact_rows(s, name, part) for part in slots.split(16384)])
    lv = levels(s["table"]).astype(np.float64)
    pair = torch.from_numpy(np.stack([np.tile(lv, 16), np.repeat(lv, 16)], -1)).to(slots.device)   # [256, 2]
    P, H, page, half = s[name + "_codes"].shape
    rows = (slots // page * H)[:, None] * page + torch.arange(H, device=slots.device) * page + (slots % page)[:, None]
    x = pair[s[name + "_codes"].view(-1, half)[rows].int()].reshape(*rows.shape, half // 32, BLOCK)
    return (x * s[name + "_scales"].view(-1, half // 32)[rows].double()[..., None]).reshape(*rows.shape, 2 * half)


def exact_stored(x, table):
    """What the values of x [tokens, heads, D] stand for once stored, in 64 bits (the two roundings of the quotient and
    the scale's are part of the rule)."""
    lv = torch.from_numpy(levels(table).astype(np.float64)).to(x.device)
    mid = (lv[1:] + lv[:-1]) / 2
    runs = x.double().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = torch.linalg.vector_norm(runs, ord=math.inf, dim=-1, keepdim=True)
    s = top.float().bfloat16().double()
    r = (1.0 / s).float().double()
    q = (runs * r).float().double()
    code = torch.zeros_like(q, dtype=torch.int64)
    for m in mid:
        code += q > m
    return torch.where(s > 0, lv[code] * s, torch.zeros_like(q)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] != "attention":
        out = []
        for name in ("k", "v"):
            got = torch.zeros((case["tokens"], case["heads"], case["dim"]), dtype=torch.float64, device="cuda")
            kept = s["kept"]
            got[kept] = (exact_stored(s[name], case["table"])[kept] if case["op"] == "write"
                         else exact_rows(s, name, s["slots"][kept].long()))
            out.append(got)
        return tuple(out)
    D, group, page = case["dim"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (length, queries) in enumerate(zip(*lengths_of(case))):
        j = torch.arange(length, device="cuda")
        slots = s["block_table"][b].long()[j // page] * page + j % page
        k, v = exact_rows(s, "k", slots), exact_rows(s, "v", slots)
        p = length - queries + torch.arange(queries, device="cuda")[:, None]
        hidden = j[None] > p if case["causal"] else torch.zeros((queries, length), dtype=torch.bool, device="cuda")
        if case["window"]:
            hidden = hidden | (j[None] + case["window"] <= p)
        for h in range(case["kv_heads"]):
            parts = [(k[c:c + 16384, h].T.contiguous(), v[c:c + 16384, h].contiguous()) for c in range(0, length, 16384)]
            for q0 in range(h * group, (h + 1) * group):
                q = s["q"][at:at + queries, q0].double()
                score = torch.cat([q @ kt for kt, _ in parts], -1) / math.sqrt(D)
                weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0)
                out[at:at + queries, q0] = sum(w @ vh for w, (_, vh) in zip(weight.split(16384, -1), parts))
        at += queries
    return out
