"""Cases for measuring the serving operators of the library: the rotation of queries and keys at
given positions, the append of keys and values to a paged 8-bit cache, the attention over that
cache, and the causal attention over packed prompts.

`run` computes an operator in its plain form (elementary torch operations in 32 bits) or, where
`own` is true, through the library. Formulas, with s = 1/sqrt(d):

  rope_at       y = R(position) x on the first `rot` columns of each head, pairs (2i, 2i+1) or
                (i, i + rot/2); the transpose is R^T (the gradient with respect to x).
  cache_append  a page of `page` tokens and one head holds e4m3 codes and one scale, a power of two,
                the smallest with |x| <= 448 scale over the page's tokens; a page that gets new
                tokens keeps the larger of its old and its new scale.
  cache_attn    O = softmax(s Q K^T) V over a sequence's cached keys, K and V being code * scale;
                causal: query i of n sees keys < len - n + i + 1; else all keys < len.
  prompt_attn   O = softmax(s Q K^T) V inside each packed sequence, key position <= query position.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
TOP = 448.0  # largest e4m3 value, 0.875 * 2^9
LOW_EXP, HIGH_EXP = -32, 32  # a page scale lies between 2^-32 and 2^32


def listed():
    return [
        # The rotation of one decode step of a batch: launch latency. Half layout, grouped heads.
        {"name": "rope decode step", "op": "rope", "tokens": 64, "heads": 32, "kv_heads": 8, "d": 128, "rot": 128,
         "layout": "half", "type": "bf16", "transpose": False, "positions": 32768},
        # Training: the gradients of q and k of the 21 frames of 1560 tokens, 12 heads, of the benchmark.
        {"name": "rope gradient 21 frames", "op": "rope", "tokens": 32760, "heads": 12, "kv_heads": 12, "d": 128, "rot": 128,
         "layout": "interleaved", "type": "bf16", "transpose": True, "positions": 32760},
        # One token of each of 64 sequences appended: decode.
        {"name": "append decode step", "op": "append", "seqs": 64, "new_low": 1, "new_high": 1, "old_low": 100, "old_high": 8000,
         "kv_heads": 8, "d": 128, "page": 64, "rot": 128, "layout": "half", "type": "bf16"},
        # A frame of 1560 tokens appended behind ten frames: the key-value cache of the frame-wise model.
        {"name": "append one frame", "op": "append", "seqs": 1, "new_low": 1560, "new_high": 1560, "old_low": 15600, "old_high": 15600,
         "kv_heads": 12, "d": 128, "page": 64, "rot": 128, "layout": "interleaved", "type": "bf16"},
        # Packed prompts of different lengths appended, pages of 16 tokens.
        {"name": "append packed prompts", "op": "append", "seqs": 16, "new_low": 17, "new_high": 4000, "old_low": 0, "old_high": 500,
         "kv_heads": 8, "d": 128, "page": 16, "rot": 64, "layout": "half", "type": "bf16"},
        # One sequence decoding at a short length: latency.
        {"name": "decode one short sequence", "op": "cache", "seqs": 1, "new": 1, "len_low": 777, "len_high": 777, "heads": 32,
         "kv_heads": 8, "d": 128, "page": 16, "causal": True, "type": "bf16"},
        # A batch decoding at lengths up to 8192.
        {"name": "decode batch of 64", "op": "cache", "seqs": 64, "new": 1, "len_low": 500, "len_high": 8192, "heads": 32,
         "kv_heads": 8, "d": 128, "page": 64, "causal": True, "type": "bf16"},
        # Four proposed tokens checked for each of three long sequences.
        {"name": "verify 4 tokens, long", "op": "cache", "seqs": 3, "new": 4, "len_low": 40001, "len_high": 131072, "heads": 32,
         "kv_heads": 8, "d": 128, "page": 64, "causal": True, "type": "fp16"},
        # One frame of 1560 tokens attending to itself and 20 cached frames: full attention inside the chunk.
        {"name": "one frame over 21 cached", "op": "cache", "seqs": 1, "new": 1560, "len_low": 32760, "len_high": 32760, "heads": 12,
         "kv_heads": 12, "d": 128, "page": 64, "causal": False, "type": "bf16"},
        # One prompt of odd length.
        {"name": "prompt of 1333 tokens", "op": "prompt", "seqs": 1, "len_low": 1333, "len_high": 1333, "heads": 16, "kv_heads": 4,
         "d": 64, "type": "fp16"},
        # Prompts of different lengths packed into one row of tokens.
        {"name": "packed prompts", "op": "prompt", "seqs": 5, "len_low": 61, "len_high": 8192, "heads": 16, "kv_heads": 4,
         "d": 128, "type": "bf16"},
        # One prompt as long as the 21 frames of the benchmark.
        {"name": "prompt of 32760 tokens", "op": "prompt", "seqs": 1, "len_low": 32760, "len_high": 32760, "heads": 8, "kv_heads": 2,
         "d": 128, "type": "bf16"},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] < 5e8 and w["flops"] < 1e12:  # no more than the largest listed ones
            return c


def _draw(rng):
    op = rng.choice(["rope", "append", "cache", "cache", "prompt"])
    d = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 12])
    if op == "rope":
        return {"op": op, "tokens": _log_int(rng, 1, 16000), "heads": kv * rng.choice([1, 2, 4]), "kv_heads": kv, "d": d,
                "rot": rng.choice([d, d // 2, 32]), "layout": rng.choice(["half", "interleaved"]),
                "type": rng.choice(["bf16", "fp16", "fp32"]), "transpose": rng.random() < 0.4, "positions": _log_int(rng, 16000, 131072)}
    if op == "append":
        seqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 1, 30000 // seqs)
        old = _log_int(rng, 1, 20000 // seqs + 1)
        return {"op": op, "seqs": seqs, "new_low": rng.randint(0, high) if seqs > 1 else high, "new_high": high, "old_low": rng.randint(0, old),
                "old_high": old, "kv_heads": kv, "d": d, "page": rng.choice([16, 32, 64, 128]), "rot": rng.choice([d, d // 2, 32]),
                "layout": rng.choice(["half", "interleaved"]), "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "cache":
        seqs = _log_int(rng, 1, 64)
        high = _log_int(rng, 16, 260000 // max(seqs, 2))
        new = _log_int(rng, 1, max(1, min(1600 // seqs, high)))
        return {"op": op, "seqs": seqs, "new": new, "len_low": rng.randint(new, high) if seqs > 1 else high, "len_high": high,
                "heads": kv * rng.choice([1, 2, 3, 4, 8] if kv <= 4 else [1]), "kv_heads": kv, "d": d, "page": rng.choice([16, 32, 64, 128]),
                "causal": rng.random() < 0.7, "type": rng.choice(["bf16", "fp16"])}
    seqs = _log_int(rng, 1, 40)
    high = _log_int(rng, 1, 16000 // max(seqs, 2))
    return {"op": op, "seqs": seqs, "len_low": rng.randint(0, high) if seqs > 1 else high, "len_high": high,
            "heads": kv * rng.choice([1, 2, 4] if kv <= 4 else [1]), "kv_heads": kv, "d": d, "type": rng.choice(["bf16", "fp16"])}


def _spread(low, high, n):
    """n whole numbers between low and high, `high` first, the others by the golden ratio's multiples."""
    return [high if i == 0 else low + int((high - low) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _tables(rot, positions, device):
    """Cosines and sines of positions * frequencies in 64 bits; base 10000, frequencies stretched by 4 beyond 32768 positions."""
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if positions > 32768:
        freq = freq / 4
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


def _quantise_pages(x):
    """Codes and scales of pages of values [..., page, d]: how a filled cache is laid down for the attention's cases."""
    amax = x.abs().amax(dim=(-1, -2)).double()
    scale = torch.exp2(torch.ceil(torch.log2(amax / TOP)).clamp(LOW_EXP, HIGH_EXP)).float()
    return (x / scale[..., None, None]).clamp(-TOP, TOP).to(F8), scale


def _filled(pages, kv_heads, page, d, g, spread):
    """A pool of pages of random values, each head's columns of their own size."""
    size = torch.exp(spread * torch.randn(kv_heads, 1, d, generator=g, device="cuda"))
    codes, scales = [], []
    for first in range(0, pages, 512):
        n = min(512, pages - first)
        c, s = _quantise_pages(torch.randn(n, kv_heads, page, d, generator=g, device="cuda") * size)
        codes.append(c.view(torch.uint8))
        scales.append(s)
    return torch.cat(codes).view(F8), torch.cat(scales).contiguous()


def _page_table(lens, page, g):
    """Pages for sequences of these lengths in a shuffled pool: (table [seqs, most], pages in the pool)."""
    need = [max(1, -(-n // page)) for n in lens]
    most, total = max(need), sum(need) + 3
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), most, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[c["type"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(t)

    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c}
    if c["op"] == "rope":
        # q and k are views of one projection's output, as a model has them
        qkv = randn(c["tokens"], c["heads"] + 2 * c["kv_heads"], c["d"])
        s["q"], s["k"] = qkv[:, :c["heads"]], qkv[:, c["heads"]:c["heads"] + c["kv_heads"]]
        s["positions"] = torch.randint(0, c["positions"], (c["tokens"],), generator=g, device="cuda", dtype=torch.int32)
        if c["tokens"] > 1000:
            s["positions"] = s["positions"].sort().values.contiguous()
        s["cos"], s["sin"] = _tables(c["rot"], c["positions"], "cuda")
    elif c["op"] == "append":
        new, old = _spread(c["new_low"], c["new_high"], c["seqs"]), _spread(c["old_low"], c["old_high"], c["seqs"])
        lens = [a + b for a, b in zip(new, old)]
        s["table"], pages = _page_table(lens, c["page"], g)
        s["k_codes"], s["k_scale"] = _filled(pages, c["kv_heads"], c["page"], c["d"], g, 0.5)
        s["v_codes"], s["v_scale"] = _filled(pages, c["kv_heads"], c["page"], c["d"], g, 0.5)
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        s["starts"], s["old"] = ints(starts), ints(old)
        qkv = randn(starts[-1], 2 * c["kv_heads"], c["d"])
        s["k"], s["v"] = qkv[:, :c["kv_heads"]], qkv[:, c["kv_heads"]:]
        s["cos"], s["sin"] = _tables(c["rot"], max(lens), "cuda")
    elif c["op"] == "cache":
        lens = _spread(c["len_low"], c["len_high"], c["seqs"])
        s["table"], pages = _page_table(lens, c["page"], g)
        s["k_codes"], s["k_scale"] = _filled(pages, c["kv_heads"], c["page"], c["d"], g, 0.5)
        s["v_codes"], s["v_scale"] = _filled(pages, c["kv_heads"], c["page"], c["d"], g, 0.2)
        s["lens"] = ints(lens)
        s["q"] = randn(c["seqs"], c["new"], c["heads"], c["d"])
    else:
        starts = [0]
        for n in _spread(c["len_low"], c["len_high"], c["seqs"]):
            starts.append(starts[-1] + n)
        s["starts"] = ints(starts)
        qkv = randn(starts[-1], c["heads"] + 2 * c["kv_heads"], c["d"])
        s["q"], s["k"], s["v"] = qkv.split([c["heads"], c["kv_heads"], c["kv_heads"]], dim=1)
    return s


def run(s):
    c = s["case"]
    if own:
        import attention_jvp_attn_b200 as lib
        if c["op"] == "rope":
            return lib.rope_at(s["q"], s["k"], s["positions"], s["cos"], s["sin"], layout=c["layout"], transpose=c["transpose"])
        if c["op"] == "append":
            cache = lib.PagedCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
            lib.cache_append(cache, s["k"], s["v"], s["starts"], s["old"], s["table"], s["cos"], s["sin"], layout=c["layout"])
            return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]
        if c["op"] == "cache":
            cache = lib.PagedCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
            return lib.cache_attn(s["q"], cache, s["lens"], s["table"], causal=c["causal"])
        return lib.prompt_attn(s["q"], s["k"], s["v"], s["starts"])
    if c["op"] == "rope":
        cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
        sin = -sin if c["transpose"] else sin
        return tuple(_rotate(x.float(), cos, sin, c["layout"]).to(x.dtype) for x in (s["q"], s["k"]))
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "cache":
        return _cache_attn(s)
    return _prompt_attn(s)


def _rotate(x, cos, sin, layout):
    """Rows [tokens, heads, d] of 32-bit values rotated by cos, sin [tokens, rot/2]."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        a, b = turned[..., :half], turned[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b = turned[..., 0::2], turned[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _needed_exp(amax):
    """The smallest e with amax <= 448 * 2^e, between the limits."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (m > 0.875).int(), LOW_EXP).clamp(LOW_EXP, HIGH_EXP)


def _append(s):
    c = s["case"]
    page, starts, old, table = c["page"], s["starts"].long(), s["old"].long(), s["table"].long()
    tokens = s["k"].shape[0]
    at = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(starts, at, right=True) - 1
    place = old[seq] + at - starts[seq]
    pages, rows = table[seq, place // page], place % page
    new = starts[1:] - starts[:-1]
    seqs = torch.arange(len(old), device="cuda")
    first = table[seqs, torch.where(new > 0, old // page, 0)]
    kept = torch.where(new > 0, old % page, 0)  # rows of the first page that stay
    for x, codes, scale in ((_rotate(s["k"].float(), s["cos"][place], s["sin"][place], c["layout"]), s["k_codes"], s["k_scale"]),
                            (s["v"].float(), s["v_codes"], s["v_scale"])):
        amax = torch.zeros_like(scale).scatter_reduce_(0, pages[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        fresh = torch.exp2(_needed_exp(amax).float())
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, pages, True)
        before = torch.zeros_like(scale).index_put_((first,), torch.where(kept[:, None] > 0, scale[first], 0.0), accumulate=True)
        after = torch.where(touched[:, None], torch.maximum(fresh, before), scale)
        held = codes[first].float() * (scale[first] / after[first])[..., None, None]
        stay = (torch.arange(page, device="cuda")[None] < kept[:, None])[:, None, :, None]
        held = torch.where(stay, held.clamp(-TOP, TOP), codes[first].float()).to(F8)
        raw = codes.view(torch.uint8)
        # sequences without new tokens write what is there
        raw[first] = torch.where((kept > 0)[:, None, None, None], held.view(torch.uint8), raw[first])
        raw[pages, :, rows] = (x / after[pages][..., None]).clamp(-TOP, TOP).to(F8).view(torch.uint8)
        scale.copy_(after)
    return s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"]


def _held(codes, scale, table):
    """The values of each sequence's pages, [seqs, kv_heads, tokens, d] in 32 bits."""
    x = codes.view(torch.uint8)[table].view(F8).float() * scale[table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _cache_attn(s):
    c = s["case"]
    table, lens = s["table"].long(), s["lens"].long()
    k, v = _held(s["k_codes"], s["k_scale"], table), _held(s["v_codes"], s["v_scale"], table)
    b, n, h, d = s["q"].shape
    q = s["q"].float().view(b, n, c["kv_heads"], h // c["kv_heads"], d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = q @ k.transpose(-1, -2)
    score *= d ** -0.5
    seen = lens[:, None] - (n - 1 - torch.arange(n, device="cuda") if c["causal"] else torch.zeros(n, device="cuda", dtype=torch.long))
    hidden = torch.arange(k.shape[2], device="cuda") >= seen[:, :, None]
    score = score.view(b, c["kv_heads"], -1, n, k.shape[2]).masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).view(*total.shape[:-1], d) / total
    lse = (top + total.log()).squeeze(-1).flatten(1, 2)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["q"].dtype), lse


def _prompt_attn(s):
    c = s["case"]
    starts = s["starts"].long()
    tokens, h, d = s["q"].shape
    at = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(starts, at, right=True)
    hidden = (seq[:, None] != seq[None]) | (at[None] > at[:, None])
    group = h // c["kv_heads"]
    q = s["q"].float().transpose(0, 1).reshape(c["kv_heads"], group * tokens, d)
    k, v = s["k"].float().transpose(0, 1), s["v"].float().transpose(0, 1)
    score = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).view(h, tokens, tokens).masked_fill_(hidden, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(c["kv_heads"], group * tokens, tokens) @ v).view(h, tokens, d) / total
    return o.transpose(0, 1).contiguous().to(s["q"].dtype), (top + total.log()).squeeze(-1)


def work(case):
    c = case
    size, d = BYTES[c["type"]], c["d"]
    if c["op"] == "rope":
        heads = c["heads"] + c["kv_heads"]
        rows = min(c["tokens"], c["positions"])
        return {"bytes": 2 * size * c["tokens"] * heads * d + 4 * c["tokens"] + rows * c["rot"] * 4, "flops": 3 * c["tokens"] * heads * c["rot"]}
    if c["op"] == "append":
        tokens = sum(_spread(c["new_low"], c["new_high"], c["seqs"]))
        values = 2 * tokens * c["kv_heads"] * d
        pages = sum(-(-n // c["page"]) for n in _spread(c["new_low"], c["new_high"], c["seqs"]))
        return {"bytes": values * (size + 1) + tokens * c["rot"] * 4 + pages * c["kv_heads"] * 8 + 12 * c["seqs"], "flops": values * 4}
    if c["op"] == "cache":
        lens, n = _spread(c["len_low"], c["len_high"], c["seqs"]), c["new"]
        pairs = sum(n * m - (n * (n - 1) // 2 if c["causal"] else 0) for m in lens)
        pages = sum(-(-m // c["page"]) for m in lens)
        return {"bytes": sum(lens) * c["kv_heads"] * d * 2 + pages * (8 * c["kv_heads"] + 4) + c["seqs"] * n * c["heads"] * (2 * d * size + 4),
                "flops": 4 * d * c["heads"] * pairs}
    lens = _spread(c["len_low"], c["len_high"], c["seqs"])
    return {"bytes": sum(lens) * (2 * (c["heads"] + c["kv_heads"]) * d * size + 4 * c["heads"]),
            "flops": 4 * d * c["heads"] * sum(m * (m + 1) // 2 for m in lens)}


def exact(case, seed):
    """The operators in 64 bits, sequence by sequence, from their definitions."""
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "rope":
        return [_turn_exact(x, s["positions"].long(), s["cos"], s["sin"], c["layout"], c["transpose"]) for x in (s["q"], s["k"])]
    if c["op"] == "append":
        return _append_exact(s)
    if c["op"] == "cache":
        outs, logs = [], []
        for b, m in enumerate(s["lens"].tolist()):
            pages = s["table"][b, :-(-m // c["page"])].long()
            k, v = ((codes.view(torch.uint8)[pages].view(F8).double() * scale[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :m]
                    for codes, scale in ((s["k_codes"], s["k_scale"]), (s["v_codes"], s["v_scale"])))
            o, l = _softmax_exact(s["q"][b], k, v, c["causal"])
            outs.append(o)
            logs.append(l)
        return torch.stack(outs), torch.stack(logs)
    outs, logs = [], []
    starts = s["starts"].tolist()
    for a, b in zip(starts, starts[1:]):
        o, l = _softmax_exact(s["q"][a:b], s["k"][a:b].double().transpose(0, 1), s["v"][a:b].double().transpose(0, 1), True)
        outs.append(o)
        logs.append(l)
    return torch.cat(outs), torch.cat(logs, 1)


def _softmax_exact(q, k, v, causal):
    """Rows [n, heads, d] over keys [kv_heads, m, d], head by head."""
    n, heads, d = q.shape
    m = k.shape[1]
    o, lse = torch.empty(n, heads, d, dtype=torch.float64, device="cuda"), torch.empty(heads, n, dtype=torch.float64, device="cuda")
    for h in range(heads):
        at = h // (heads // k.shape[0])
        score = q[:, h].double() @ k[at].T / math.sqrt(d)
        if causal:
            score += torch.full((n, m), -math.inf, dtype=torch.float64, device="cuda").triu(m - n + 1)
        lse[h] = torch.logsumexp(score, -1)
        o[:, h] = torch.softmax(score, -1) @ v[at]
    return o, lse


def _turn_exact(x, positions, cos, sin, layout, transpose):
    """Each pair as a complex number times cos +- i sin."""
    half = cos.shape[1]
    turn = torch.complex(cos[positions].double(), sin[positions].double())[:, None]
    turn = turn.conj() if transpose else turn
    y = x.double().clone()
    first, second = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    z = torch.complex(y[..., first].clone(), y[..., second].clone()) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _append_exact(s):
    """Token by token's definition, one sequence's page after the other, on the host."""
    c = s["case"]
    page, starts, old, table = c["page"], s["starts"].tolist(), s["old"].tolist(), s["table"].tolist()
    at = torch.cat([torch.arange(n, n + b - a) for n, a, b in zip(old, starts, starts[1:])]).to("cuda")
    out = []
    for x, codes, scale in ((_turn_exact(s["k"], at, s["cos"], s["sin"], c["layout"], False), s["k_codes"], s["k_scale"]),
                            (s["v"].double(), s["v_codes"], s["v_scale"])):
        values, scales = codes.double(), scale.double()
        for b, (n, a, e) in enumerate(zip(old, starts, starts[1:])):
            done = a
            while done < e:
                p = n + done - a
                first, take = p % page, min(page - p % page, e - done)
                at_page = table[b][p // page]
                rows = x[done:done + take]
                need = torch.ceil(torch.log2(rows.abs().amax((0, 2)) / TOP)).clamp(LOW_EXP, HIGH_EXP).exp2()
                if first:
                    need = torch.maximum(need, scales[at_page])
                    kept = values[at_page, :, :first] * (scales[at_page] / need)[:, None, None]
                    values[at_page, :, :first] = kept.float().to(F8).double()
                values[at_page, :, first:first + take] = (rows.transpose(0, 1) / need[:, None, None]).clamp(-TOP, TOP).float().to(F8).double()
                scales[at_page] = need
                done += take
        out.append((values, scales))
    return out[0][0], out[1][0], out[0][1], out[1][1]
