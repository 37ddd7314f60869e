"""Attention beside the compressed linears: the cases its operators are timed
and compared on, their plain form and their definition in 64 bits.

Four operators share one paged key-value cache:

  prompt   attention of packed prompts (causal or not, grouped heads, keys
           that may begin before the queries), on dense q, k and v
  decode   attention of one new token per sequence over the paged cache
  append   new tokens' keys and values written into the cache, kept as bf16,
           8-bit or 4-bit codes with one scale per token and head
  read     cached tokens read back as dense keys and values

A case names its operator in "op". Cache cases time append followed by read of
the same tokens ("cache"), or read alone ("read").

The cache holds pages [num_pages][kv_heads][page][row]: rows of head_dim bf16
values, of head_dim int8 codes, or of head_dim / 2 bytes with two 4-bit codes
each (code + 8; the even dimension in the low half); scales are float32
[num_pages][kv_heads][page]. With a = max |x| over a head's row and Q = 127
(8 bits) or 7 (4 bits): code = round_half_even(Q x / a), scale = a / Q.
"""
import math

import torch

own = False

QMAX = {"int8": 127, "int4": 7}


def _glq():
    from dequant_e8_codebook_amd import glq
    return glq


# ------------------------------------------------------------------- cases

def _prompt(name, batch, longest, heads, kv_heads, dim, causal=True, prefix=0, dtype="bf16"):
    return {"name": name, "op": "prompt", "batch": batch, "longest": longest, "prefix": prefix, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "causal": causal, "dtype": dtype}


def _decode(name, batch, longest, heads, kv_heads, dim, fmt, page, dtype="bf16"):
    return {"name": name, "op": "decode", "batch": batch, "longest": longest, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "format": fmt, "page": page, "dtype": dtype}


def _cache(name, op, tokens, kv_heads, dim, fmt, page):
    return {"name": name, "op": op, "tokens": tokens, "kv_heads": kv_heads, "dim": dim, "format": fmt, "page": page,
            "dtype": "bf16"}


def listed():
    return [
        # a short question to a 4096-wide model (32 heads of 128, 8 kept): one launch, latency counts
        _prompt("prompt.short", 1, 17, 32, 8, 128),
        # a serving step's packed prompts of very different lengths, an empty one and a single token among them
        _prompt("prompt.packed", 12, 2048, 32, 8, 128),
        # one long document
        _prompt("prompt.long", 1, 8192, 32, 8, 128),
        # the image block of the benchmark: 4096 tokens, 24 heads of 128, every token sees every other
        _prompt("prompt.image", 1, 4096, 24, 24, 128, causal=False),
        # chunks of prompts on top of cached prefixes, float32 as in the float32 path of the linears
        _prompt("prompt.chunk.f32", 3, 333, 16, 2, 64, prefix=1000, dtype="f32"),
        # one user: the next token of a chat of 1000 tokens, cache not quantised
        _decode("decode.one", 1, 1000, 32, 8, 128, "bf16", 64),
        # a serving step: 32 users with chats of up to 4096 tokens, 8-bit cache in small pages
        _decode("decode.batch", 32, 4096, 32, 8, 128, "int8", 16),
        # two users with book-length contexts, 4-bit cache
        _decode("decode.long", 2, 131072, 32, 8, 128, "int4", 64),
        # one kept head of 256 for all query heads, float32 activations
        _decode("decode.mqa.f32", 8, 3000, 8, 1, 256, "bf16", 32, dtype="f32"),
        # the new tokens of a serving step into the 8-bit cache: latency
        _cache("cache.token", "cache", 32, 8, 128, "int8", 16),
        # a long prompt into the 4-bit cache, and back for its next chunk
        _cache("cache.prompt", "cache", 8192, 8, 128, "int4", 64),
        # a shared 8-bit prefix read back for the chunks that follow it
        _cache("cache.prefix", "read", 50001, 8, 128, "int8", 32),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "decode", "decode", "cache", "read"])
    heads, kv_heads = rng.choice([(32, 8), (24, 24), (16, 2), (8, 1), (12, 4), (40, 8), (7, 7)])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "int8", "int4"])
    if op == "prompt":
        top = {c["dtype"]: work(c)["flops"] for c in listed() if c["op"] == op and c["name"] in ("prompt.long", "prompt.chunk.f32")}
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        case = _prompt("", rng.randint(1, 12), _between(rng, 1, 8192), heads, kv_heads, dim, rng.random() < 0.75,
                       rng.choice([0, 0, _between(rng, 1, 2000)]), dtype)
        while work(case)["flops"] > top[dtype] or _padded(case) > 2 ** 31:
            case["batch"], case["longest"] = max(1, case["batch"] - 1), max(1, case["longest"] * 4 // 5)
            case["prefix"] = case["prefix"] * 4 // 5
    elif op == "decode":
        top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
        case = _decode("", _between(rng, 1, 48), _between(rng, 1, 131072), heads, kv_heads, dim, fmt, page,
                       rng.choice(["bf16", "bf16", "bf16", "f32"]))
        while work(case)["bytes"] > top or case["batch"] * case["longest"] * kv_heads * dim > 2 ** 28:
            case["longest"] = max(1, case["longest"] * 3 // 4)
    else:
        top = max(work(c)["bytes"] for c in listed() if c["op"] == op)
        case = _cache("", op, _between(rng, 1, 50000), kv_heads, dim, fmt, page)
        while work(case)["bytes"] > top:
            case["tokens"] = max(1, case["tokens"] * 3 // 4)
    del case["name"]
    return case


def _lens(batch, longest):
    """Lengths from 0 to `longest`, spread evenly; the first is the longest, one of three or more is 1, one of four or more 0."""
    out = [longest] + [1 + int((longest - 1) * (i * 0.6180339887498949 % 1.0)) for i in range(1, batch)]
    if batch >= 3:
        out[2] = 1
    if batch >= 4:
        out[3] = 0
    return out


def _padded(case):
    return case["batch"] * case["heads"] * case["longest"] * (case["longest"] + case["prefix"])


def _row_bytes(case):
    """Bytes of one cached head of one token, its scale among them."""
    return {"bf16": 2 * case["dim"], "int8": case["dim"] + 4, "int4": case["dim"] // 2 + 4}[case["format"]]


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    d, kvh = case["dim"], case["kv_heads"]
    if case["op"] == "prompt":
        pairs = queries = keys = 0
        for n in _lens(case["batch"], case["longest"]):
            p = case["prefix"] if n else 0
            queries, keys = queries + n, keys + n + p
            pairs += n * p + (n * (n + 1) // 2 if case["causal"] else n * n)
        return {"bytes": size * d * (2 * queries * case["heads"] + 2 * keys * kvh), "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "decode":
        tokens = sum(_lens(case["batch"], case["longest"]))
        return {"bytes": 2 * tokens * kvh * _row_bytes(case) + 2 * size * d * case["heads"] * case["batch"],
                "flops": 4 * d * case["heads"] * tokens}
    n = case["tokens"] * kvh
    dense, held = 2 * n * d * size, 2 * n * _row_bytes(case)
    if case["op"] == "read":
        return {"bytes": dense + held + 4 * case["tokens"], "flops": 2 * n * d}
    return {"bytes": 2 * dense + 2 * held + 4 * case["tokens"], "flops": 8 * n * d}


# ------------------------------------------------------------------ inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _quantise(x, fmt):
    """Codes of the cache's format and their scales, for x [..., dim]."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    x = x.to(torch.float32)
    top = x.abs().amax(-1, keepdim=True)
    code = torch.where(top > 0, torch.round(x * QMAX[fmt] / top), torch.zeros_like(x))
    scale = (top / QMAX[fmt]).squeeze(-1)
    if fmt == "int8":
        return code.to(torch.int8), scale
    code = (code + 8).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _values(codes, scale, fmt):
    """float32 values of gathered cache rows."""
    if fmt == "bf16":
        return codes.to(torch.float32)
    if fmt == "int4":
        codes = torch.stack(((codes & 15).to(torch.float32) - 8, (codes >> 4).to(torch.float32) - 8), -1).flatten(-2)
    return codes.to(torch.float32) * scale.unsqueeze(-1)


def _pages_for(lens, page, gen, dev):
    """A page table [batch, most pages] of pages in no order, and the number of pages."""
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(len(lens), max(1, max(need)), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _offsets(lens, dev):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    d, kvh, dt = case["dim"], case["kv_heads"], _dtype(case)
    s = {"case": dict(case), "seed": seed}
    if case["op"] == "prompt":
        lens = _lens(case["batch"], case["longest"])
        keys = [n + case["prefix"] if n else 0 for n in lens]
        s.update(q=(1.5 * normal(sum(lens), case["heads"], d)).to(dt), k=normal(sum(keys), kvh, d).to(dt),
                 v=normal(sum(keys), kvh, d).to(dt), cu_q=_offsets(lens, dev), cu_k=_offsets(keys, dev))
        s["out"] = torch.empty_like(s["q"])
        return s
    fmt, page = case["format"], case["page"]
    if case["op"] == "decode":
        lens = _lens(case["batch"], case["longest"])
        s["table"], pages = _pages_for(lens, page, gen, dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q"] = (1.5 * normal(case["batch"], case["heads"], d)).to(dt)
        s["out"] = torch.empty_like(s["q"])
        s["cache"] = _quantise(normal(pages, kvh, page, d), fmt) + _quantise(normal(pages, kvh, page, d), fmt)
    else:
        n = case["tokens"]
        table, pages = _pages_for([n], page, gen, dev)
        at = torch.arange(n, device=dev)
        s["slots"] = (table[0, at // page] * page + at % page).to(torch.int32)
        few = torch.where(torch.rand(kvh, d, generator=gen, device=dev) < 0.02, 8.0, 1.0)     # channels that stand out
        s["k_out"], s["v_out"] = (torch.empty(n, kvh, d, dtype=dt, device=dev) for _ in range(2))
        if case["op"] == "read":
            s["cache"] = _quantise(normal(pages, kvh, page, d), fmt) + _quantise(normal(pages, kvh, page, d), fmt)
        else:
            s["k"], s["v"] = (normal(n, kvh, d) * few).to(dt), normal(n, kvh, d).to(dt)
            s["cache"] = tuple(None if t is None else torch.zeros_like(t)
                               for _ in range(2) for t in _quantise(torch.zeros(pages, kvh, page, d, device=dev), fmt))
    if own:
        glq = _glq()
        k, ks, v, vs = s["cache"]
        s["handle"] = glq.KvCache(k, v, ks, vs)
        if case["op"] == "decode":
            s["workspace"] = torch.zeros(glq.attn_decode_workspace_bytes(s["handle"], case["batch"], case["heads"],
                                                                         case["longest"]),
                                         dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    if own:
        glq = _glq()
        if case["op"] == "prompt":
            return glq.attn_prompt(s["q"], s["k"], s["v"], s["out"], s["cu_q"], s["cu_k"], max_q=case["longest"],
                                   causal=case["causal"])
        if case["op"] == "decode":
            return glq.attn_decode(s["handle"], s["q"], s["table"], s["lens"], s["out"], s["workspace"],
                                   max_len=case["longest"])
        if case["op"] == "cache":
            glq.kv_append(s["handle"], s["k"], s["v"], s["slots"])
        glq.kv_read(s["handle"], s["slots"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    if case["op"] == "prompt":
        return _plain_prompt(s, case)
    if case["op"] == "decode":
        return _plain_decode(s, case)
    return _plain_cache(s, case)


def _softmax(scores, seen):
    """Rows of weights; a row that sees nothing is all zero."""
    scores = scores.masked_fill_(~seen, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    weight = torch.exp(scores - torch.where(torch.isfinite(top), top, 0.0))
    total = weight.sum(-1, keepdim=True)
    return weight / torch.where(total > 0, total, 1.0)


def _plain_prompt(s, case):
    """Sequences padded to the longest, one product for all of them."""
    batch, most, d, kvh = case["batch"], case["longest"], case["dim"], case["kv_heads"]
    group, most_k, dev = case["heads"] // kvh, most + case["prefix"], s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(most, device=dev), torch.arange(most_k, device=dev)
    row = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    col = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[row].reshape(batch, most, kvh, group, d).permute(0, 2, 3, 1, 4).reshape(batch, kvh, group * most, d)
    k, v = s["k"].float()[col].permute(0, 2, 3, 1), s["v"].float()[col].transpose(1, 2)
    seen = (i < lq[:, None])[:, :, None] & (j < lk[:, None])[:, None, :]
    if case["causal"]:
        seen = seen & (j[None, None, :] <= (i[None, :] + (lk - lq)[:, None])[:, :, None])
    scores = torch.matmul(q, k.contiguous()).mul_(d ** -0.5).view(batch, kvh, group, most, most_k)
    weight = _softmax(scores, seen[:, None, None]).view(batch, kvh, group * most, most_k)
    o = torch.matmul(weight, v.contiguous()).view(batch, kvh, group, most, d).permute(0, 3, 1, 2, 4)
    return o.reshape(batch, most, case["heads"], d)[i < lq[:, None]].to(s["q"].dtype)


def _plain_decode(s, case):
    batch, most, d, kvh, page = case["batch"], case["longest"], case["dim"], case["kv_heads"], case["page"]
    table = s["table"].long()

    def gathered(codes, scale):                     # [batch, kv_heads, tokens, dim]
        x = _values(codes[table], None if scale is None else scale[table], case["format"])
        return x.transpose(1, 2).reshape(batch, kvh, table.shape[1] * page, d)

    k, v = gathered(*s["cache"][:2]), gathered(*s["cache"][2:])
    q = s["q"].float().view(batch, kvh, case["heads"] // kvh, d)
    seen = torch.arange(k.shape[2], device=k.device) < s["lens"][:, None]
    weight = _softmax(torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5), seen[:, None, None])
    return torch.matmul(weight, v).view(batch, case["heads"], d).to(s["q"].dtype)


def _plain_cache(s, case):
    k, ks, v, vs = s["cache"]
    page, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]

    def put(cache, scales, x):
        codes, scale = _quantise(x, case["format"])
        cache[page, :, off] = codes
        if scale is not None:
            scales[page, :, off] = scale

    def get(cache, scales):
        return _values(cache[page, :, off], None if scales is None else scales[page, :, off], case["format"])

    if case["op"] == "cache":
        put(k, ks, s["k"])
        put(v, vs, s["v"])
    return get(k, ks).to(s["k_out"].dtype), get(v, vs).to(s["v_out"].dtype)


# ---------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(s, case)
    if case["op"] == "decode":
        return _exact_decode(s, case)
    if case["op"] == "read":
        return tuple(_exact_rows(s["cache"][i], s["cache"][i + 1], s["slots"], case) for i in (0, 2))
    return tuple(_exact_round_trip(s[n].double(), case["format"]) for n in ("k", "v"))


def _exact_attend(q, k, v, last):
    """q [queries, dim], k and v [keys, dim]; query i sees keys 0 .. last[i]."""
    out = torch.zeros_like(q)
    rows = torch.nonzero(last >= 0).flatten()
    for r in rows.split(2048):
        e = q[r] @ k.T / math.sqrt(q.shape[1])
        e[torch.arange(k.shape[0], device=q.device)[None] > last[r, None]] = -math.inf
        e = torch.exp(e - e.max(1, keepdim=True).values)
        out[r] = (e @ v) / e.sum(1, keepdim=True)
    return out


def _exact_prompt(s, case):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["batch"]):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if not n:
            continue
        last = torch.arange(n, device=out.device) + (m - n) if case["causal"] else torch.full((n,), m - 1, device=out.device)
        for h in range(case["heads"]):
            g = h * case["kv_heads"] // case["heads"]
            k, v = (s[x][ck[b]:ck[b + 1], g].double() for x in "kv")
            out[cq[b]:cq[b + 1], h] = _exact_attend(s["q"][cq[b]:cq[b + 1], h].double(), k, v, last)
    return out


def _exact_codes(codes, fmt):
    if fmt != "int4":
        return codes.double()
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = codes % 16, codes // 16
    return out - 8


def _exact_rows(codes, scale, slots, case):
    """Cached rows [tokens, kv_heads, dim] at the slots."""
    slots = slots.long()
    pick = (torch.div(slots, case["page"], rounding_mode="floor"), slice(None), slots % case["page"])
    x = _exact_codes(codes[pick], case["format"])
    return x if scale is None else x * scale[pick].double()[..., None]


def _exact_decode(s, case):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    group = case["heads"] // case["kv_heads"]
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        at = torch.arange(n, device=out.device)
        slots = s["table"][b].long()[at // case["page"]] * case["page"] + at % case["page"]
        k, v = (_exact_rows(s["cache"][i], s["cache"][i + 1], slots, case) for i in (0, 2))
        for h in range(case["heads"]):
            out[b, h] = _exact_attend(s["q"][b, h:h + 1].double(), k[:, h // group], v[:, h // group],
                                      torch.tensor([n - 1], device=out.device))[0]
    return out


def _exact_round_trip(x, fmt):
    if fmt == "bf16":
        return x
    top, levels = x.abs().max(-1, keepdim=True).values, QMAX[fmt]
    safe = torch.where(top == 0, 1.0, top)
    return torch.round(x * levels / safe) * top / levels
