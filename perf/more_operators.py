"""A serving step around the compressed linears and the paged cache: the cases
its operators are timed and compared on, their plain form and their definition
in 64 bits.

Four operators, in the order in which a step of a model whose feed-forward layers
are compressed experts runs them:

  plan     from the requests' lengths: pages taken from the free ones, slots and
           positions of the new tokens, offsets, and the slots of all cached tokens
  rope     norms of the queries and keys of every head with the rotation by their
           positions, and the write of keys and values into the paged cache
  route    each token's experts and their weights from the router's scores, and
           the tokens in the experts' order
  experts  the compressed linear of each row's own expert over ragged groups of
           rows, gathered from the tokens and, on the way back, summed into them

A case names its operator in "op".

The cache is the paged one of the attention calls: pages [num_pages][kv_heads]
[page][row], rows of head_dim bf16 values or of int8 codes with float32 scales
[num_pages][kv_heads][page]; a = max |x| over a head's row, code =
round_half_even(127 x / a), scale = a / 127. A compressed expert is y = U^T (s W)
(V x): W holds, for every 8 inputs, the E8 codebook's entry i1 plus 2^-k times the
entry i2 (none at 2 bits a weight; k = 1 with 8-bit i2 at 3, k = 2 with 16-bit i2 at
4); U and V are sign flips followed by a block Walsh-Hadamard transform over the
largest power of two that divides the length.
"""
import functools
import itertools
import math

import numpy as np
import torch

own = False


def _glq():
    from dequant_e8_codebook_amd import glq
    return glq


# ------------------------------------------------------------------- cases

def _plan(name, batch, longest, new, page, read=False, short=0):
    return {"name": name, "op": "plan", "batch": batch, "longest": longest, "new": new, "page": page, "read": read,
            "short": short}


def _rope(name, tokens, heads, kv_heads, dim, rot, pairs=False, norm=True, format="none", dense=True, dtype="bf16"):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "pairs": pairs, "norm": norm, "format": format, "dense": dense, "page": 16, "dtype": dtype}


def _route(name, tokens, experts, top, dtype="f32", normalize=True, padded=0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "top": top, "normalize": normalize,
            "padded": padded, "dtype": dtype}


def _experts(name, tokens, experts, top, n, k, bpw, gather=True, combine=True, row_scale=False, dtype="bf16"):
    return {"name": name, "op": "experts", "tokens": tokens, "experts": experts, "top": top, "n": n, "k": k, "bpw": bpw,
            "gather": gather, "combine": combine, "row_scale": row_scale, "dtype": dtype}


def listed():
    return [
        # one token for each of 32 users with chats of up to 4096 tokens, small pages: latency
        _plan("plan.step", 32, 4096, 1, 16),
        # chunks of prompts of 300 users, the pages short by a few, and everything cached listed to be read back
        _plan("plan.chunks", 300, 8192, 2048, 64, read=True, short=5),
        # one user's next token, 32 heads on 8 of 128: latency
        _rope("rope.token", 1, 32, 8, 128, 128),
        # a serving step's tokens, straight into the 8-bit cache
        _rope("rope.step", 32, 32, 8, 128, 128, format="int8", dense=False),
        # a long prompt: keys stay at hand for its own attention and go into the cache
        _rope("rope.prompt", 8192, 32, 8, 128, 128, format="bf16"),
        # float32 path, half of each head rotated in neighbouring pairs
        _rope("rope.pairs.f32", 999, 16, 2, 64, 32, pairs=True, dtype="f32"),
        # a serving step: 32 tokens to 8 of 64 experts
        _route("route.step", 32, 64, 8),
        # a long prompt in bf16 scores (ties are common), the batch padded at its end
        _route("route.prompt", 8192, 128, 8, dtype="bf16", padded=77),
        # one user's token through 2 of 8 experts of 4096 x 4096, 4 bits: latency and the indices
        _experts("experts.one", 1, 8, 2, 4096, 4096, 4),
        # a serving step on many small experts: a few rows each, none for some
        _experts("experts.step", 32, 64, 8, 1024, 2048, 2),
        # a prompt of 4096 tokens, two experts of eight each: matrix cores
        _experts("experts.prompt", 4096, 8, 2, 4096, 4096, 3),
        # float32 path, odd sizes, a scale for each output row, rows in the experts' order in and out
        _experts("experts.f32", 70, 5, 2, 1000, 328, 4, gather=False, combine=False, row_scale=True, dtype="f32"),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "route", "experts", "experts", "experts"])
    if op == "plan":
        case = _plan("", _between(rng, 1, 600), _between(rng, 1, 8192), _between(rng, 1, 2048),
                     rng.choice([16, 32, 64, 128]), rng.random() < 0.5, rng.choice([0, 0, 3]))
    elif op == "rope":
        heads, kv_heads = rng.choice([(32, 8), (24, 24), (16, 2), (8, 1), (12, 4), (40, 8), (7, 7)])
        dim, dtype = rng.choice([64, 128, 128, 256]), rng.choice(["bf16", "bf16", "bf16", "f32"])
        form = rng.choice(["none", "bf16", "int8"])
        case = _rope("", _between(rng, 1, 8192), heads, kv_heads, dim, rng.choice([dim, dim, dim // 2]), rng.random() < 0.4,
                     rng.random() < 0.8, form, form == "none" or rng.random() < 0.5, dtype)
    elif op == "route":
        experts = rng.choice([4, 8, 8, 16, 60, 64, 128, 160, 256])
        case = _route("", _between(rng, 1, 8192), experts, min(experts, rng.choice([1, 2, 4, 6, 8])),
                      rng.choice(["f32", "bf16"]), rng.random() < 0.6, rng.choice([0, 0, 1, 30]))
        case["padded"] = min(case["padded"], case["tokens"] // 2)
    else:
        experts = rng.choice([2, 4, 8, 8, 16, 60, 64])
        top, dtype = min(experts, rng.choice([1, 2, 2, 4, 8])), rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        sides = [256, 512, 1000, 1024, 1416, 2048, 2048, 4096, 4096]
        case = _experts("", _between(rng, 1, 4096), experts, top, rng.choice(sides), rng.choice(sides + [328]),
                        rng.choice([2, 3, 4]), rng.random() < 0.7, rng.random() < 0.7, rng.random() < 0.2, dtype)
        while experts * case["n"] * case["k"] > 2 ** 27:
            case["n"], case["k"] = min(case["n"], 2048 if experts < 60 else 1024), min(case["k"], 2048)
    top = {k: max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")}
    if case["dtype" if op != "plan" else "op"] == "f32" and op == "experts":
        top["flops"] /= 16
    size = "new" if op == "plan" else "tokens"
    while any(work(case)[k] > top[k] for k in top) and case[size] > 1:
        case[size] = case[size] * 3 // 4
        if op == "plan":
            case["longest"] = max(1, case["longest"] * 3 // 4)
        if op == "route":
            case["padded"] = min(case["padded"], case["tokens"] // 2)
    del case["name"]
    return case


def _spread(batch, longest):
    """Lengths from 0 to `longest`, spread evenly; the first is the longest, one of three or more is 1, one of four or more 0."""
    out = [longest] + [int((longest + 0.999) * (i * 0.6180339887498949 % 1.0)) for i in range(1, batch)]
    if batch >= 3:
        out[2] = min(1, longest)
    if batch >= 4:
        out[3] = 0
    return out


def _plan_lens(case):
    """Cached tokens and new ones of every request."""
    held = _spread(case["batch"], case["longest"])
    return held, _spread(case["batch"], case["new"])[::-1] if case["new"] > 1 else [1] * case["batch"]


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    op = case["op"]
    if op == "plan":
        held, new = _plan_lens(case)
        p = case["page"]
        before, after = (sum(-(-n // p) for n in x) for x in (held, [a + b for a, b in zip(held, new)]))
        words = 5 * case["batch"] + 2 * sum(new) + 2 * (after - before)
        if case["read"]:
            words += before + sum(held) + sum(new) + case["batch"]
        return {"bytes": 4 * words, "flops": 0}
    if op == "rope":
        t, d, size = case["tokens"], case["dim"], _size(case)
        rows, kv = t * (case["heads"] + case["kv_heads"]), t * case["kv_heads"]
        wrote = t * case["heads"] + (kv if case["dense"] else 0)
        held = 0 if case["format"] == "none" else 2 * kv * (2 * d if case["format"] == "bf16" else d + 4)
        back = held + 2 * kv * d * size if case["format"] == "int8" else 0
        return {"bytes": size * d * (rows + wrote) + (size * kv * d if held else 0) + held + back
                + t * (4 + 4 * case["rot"]), "flops": 0}
    if op == "route":
        t, picks = case["tokens"], case["tokens"] * case["top"]
        return {"bytes": t * case["experts"] * _size(case) + 16 * picks + 4 * case["experts"], "flops": 0}
    rows, n, k = case["tokens"] * case["top"], case["n"], case["k"]
    used = case["experts"] * (1.0 - (1.0 - case["top"] / case["experts"]) ** case["tokens"])
    ins = case["tokens"] if case["gather"] else rows
    outs = case["tokens"] if case["combine"] else rows
    return {"bytes": used * n * k * case["bpw"] / 8 + used * (n + k) + _size(case) * (ins * k + outs * n),
            "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs

def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


@functools.lru_cache(maxsize=2)
def _codebook(device):
    """The 65,536 E8 points in the format's order, float32 [65536, 8]. Points are
    y = 2x with all of them even or all odd and a sum divisible by 4, of squared norm
    up to 12, sorted by (|x|^2, -orbit size, max |x_i|, |x|, sign counter)."""
    both = []
    for vals in (range(-6, 7, 2), range(-5, 6, 2)):
        half = np.array(list(itertools.product(vals, repeat=4)), np.int16)
        half = half[(half ** 2).sum(1) <= 48]
        a, b = (g.ravel() for g in np.meshgrid(np.arange(len(half)), np.arange(len(half)), indexing="ij"))
        near = (half ** 2).sum(1)[a] + (half ** 2).sum(1)[b] <= 48
        both.append(np.concatenate((half[a[near]], half[b[near]]), 1))
    y = np.concatenate(both).astype(np.int64)
    y = y[y.sum(1) % 4 == 0]
    mag, neg, odd = np.abs(y), y < 0, y[:, :1] % 2 == 1
    bit = np.where(odd, np.array([0, 1, 2, 62, 3, 4, 5, 6]), np.cumsum(mag > 0, 1) - 1)      # (62: fixed by the parity)
    counter = np.where(neg & (bit < 62), 1 << np.clip(bit, 0, 8), 0).sum(1)
    orbit = np.where(odd[:, 0], 128, 1 << (mag > 0).sum(1))
    order = np.lexsort([counter] + [mag[:, c] for c in range(7, -1, -1)] + [mag.max(1), -orbit, (y ** 2).sum(1)])
    return torch.from_numpy(y[order[:65536]].astype(np.float32) / 2).to(device)


def _signs(gen, *shape):
    return (torch.randint(0, 2, shape, generator=gen, device=gen.device) * 2 - 1).to(torch.int8)


def _grouped(ids, experts):
    """Choices [tokens, top] of experts (or -1) in the experts' order: offsets, tokens of the rows, rows of the choices."""
    flat = ids.flatten().long()
    order = torch.sort(torch.where(flat < 0, experts, flat), stable=True)
    bounds = torch.searchsorted(order.values, torch.arange(experts + 1, device=ids.device))
    at = torch.empty_like(flat)
    at[order.indices] = torch.arange(len(flat), device=ids.device)
    rows = torch.arange(len(flat), device=ids.device) < bounds[-1]
    src = torch.where(rows, order.indices // ids.shape[1], -1)
    pos = torch.where(flat < 0, -1, at).view(ids.shape)
    return bounds.to(torch.int32), src.to(torch.int32), pos.to(torch.int32)


def prepare(case, seed):
    dev = torch.device(_device(), 0) if _device() == "cuda" else torch.device("cpu")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case), "seed": seed}
    {"plan": _prepare_plan, "rope": _prepare_rope, "route": _prepare_route, "experts": _prepare_experts}[case["op"]](
        case, s, gen, dev)
    return s


def _prepare_plan(case, s, gen, dev):
    held, new = _plan_lens(case)
    page = case["page"]
    mix = torch.randperm(case["batch"], generator=gen, device=dev).cpu().tolist()       # which request has which length
    held, new = [held[i] for i in mix], [new[i] for i in mix]
    pages = [-(-n // page) for n in held]
    wanted = sum(-(-(a + b) // page) for a, b in zip(held, new)) - sum(pages)
    s["num_pages"] = sum(pages) + wanted + 9
    s["most"] = sum(new) + 7                                   # a batch padded at its end
    s["most_read"] = sum(held) + sum(new) if case["read"] else 0
    order = torch.randperm(s["num_pages"], generator=gen, device=dev).to(torch.int32)
    s["table"] = torch.full((case["batch"], -(-(case["longest"] + case["new"]) // page)), -1, dtype=torch.int32, device=dev)
    at = torch.arange(s["table"].shape[1], device=dev)
    count = torch.tensor(pages, device=dev)
    s["table"][at < count[:, None]] = order[:sum(pages)]
    s["free"] = order[sum(pages):sum(pages) + max(0, wanted + 4 - 4 * bool(case["short"]) - case["short"])].contiguous()
    s["lens"], s["added"] = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (held, new))
    if own:
        s["plan"] = _glq().KvPlan(s["table"], page, s["num_pages"], s["most"], s["most_read"])


def _prepare_rope(case, s, gen, dev):
    t, h, kvh, d, page = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["page"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    few = torch.where(torch.rand(h + 2 * kvh, d, generator=gen, device=dev) < 0.02, 8.0, 1.0)    # channels that stand out
    qkv = (normal(t, h + 2 * kvh, d) * few).to(_dtype(case))                  # one projection's output
    s["q"], s["k"], s["v"] = qkv.split((h, kvh, kvh), 1)
    s["w"] = [None, None] if not case["norm"] else [1.0 + 0.3 * normal(d) for _ in range(2)]
    most = 32768
    turn = torch.arange(case["rot"] // 2, dtype=torch.float64, device=dev) * (-2.0 / case["rot"])
    angle = torch.arange(most, dtype=torch.float64, device=dev)[:, None] * torch.exp(turn * math.log(500000.0))
    s["rotary"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    begins = torch.randint(0, most - t, (1,), generator=gen, device=dev)
    s["positions"] = ((torch.arange(t, device=dev) + begins) % most).to(torch.int32)
    s["q_out"] = torch.empty(t, h, d, dtype=_dtype(case), device=dev)
    s["k_out"] = torch.empty(t, kvh, d, dtype=_dtype(case), device=dev) if case["dense"] else None
    s["cache"] = s["slots"] = None
    if case["format"] == "none":
        return
    pages = -(-t // page) + 3
    order = torch.randperm(pages, generator=gen, device=dev)
    at = torch.arange(t, device=dev)
    s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
    code = torch.int8 if case["format"] == "int8" else torch.bfloat16
    k, v = (torch.zeros(pages, kvh, page, d, dtype=code, device=dev) for _ in range(2))
    scales = [torch.zeros(pages, kvh, page, device=dev) if case["format"] == "int8" else None for _ in range(2)]
    s["cache"] = (k, scales[0], v, scales[1])
    s["back"] = [torch.empty(t, kvh, d, dtype=_dtype(case), device=dev) for _ in range(2)]
    if own:
        s["handle"] = _glq().KvCache(k, v, *scales)


def _scores(gen, tokens, experts):
    """Router scores: some experts are asked for far more often than others."""
    lean = torch.randn(experts, generator=gen, device=gen.device)
    return torch.randn(tokens, experts, generator=gen, device=gen.device) + 0.7 * lean


def _prepare_route(case, s, gen, dev):
    t, e, top = case["tokens"], case["experts"], case["top"]
    logits = 2.0 * _scores(gen, t, e)
    logits[t - case["padded"]:] = -math.inf                       # rows behind the last token
    s["logits"] = logits.to(_dtype(case))
    if own:
        s["weights"] = torch.empty(t, top, device=dev)
        s["ids"], s["pos"] = (torch.empty(t, top, dtype=torch.int32, device=dev) for _ in range(2))
        s["src"], s["offsets"] = (torch.empty(m, dtype=torch.int32, device=dev) for m in (t * top, e + 1))
        s["workspace"] = torch.zeros(_glq().route_workspace_bytes(t, e, top), dtype=torch.uint8, device=dev)


def _prepare_experts(case, s, gen, dev):
    t, e, top, n, k, bpw = (case[x] for x in ("tokens", "experts", "top", "n", "k", "bpw"))
    ids = torch.topk(_scores(gen, t, e), top).indices
    s["offsets"], src, pos = _grouped(ids, e)
    s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max().item())      # rows of the busiest expert
    rows = t * top
    few = torch.where(torch.rand(k, generator=gen, device=dev) < 0.01, 8.0, 1.0)        # channels that stand out
    s["x"] = (torch.randn(t if case["gather"] else rows, k, generator=gen, device=dev) * few).to(_dtype(case))
    s["src"] = src if case["gather"] else None
    s["pos"] = pos if case["combine"] else None
    s["weights"] = torch.softmax(torch.randn(t, top, generator=gen, device=dev), 1) if case["combine"] else None
    g = k // 8
    s["idx1"] = torch.randint(0, 65536, (e, n, g), generator=gen, device=dev, dtype=torch.int32).to(torch.int16)
    s["idx2"] = None
    if bpw > 2:
        s["idx2"] = torch.randint(0, 256 if bpw == 3 else 65536, (e, n, g), generator=gen, device=dev,
                                  dtype=torch.int32).to(torch.uint8 if bpw == 3 else torch.int16)
    s["sign_k"], s["sign_n"] = _signs(gen, e, k), _signs(gen, e, n)
    s["scale"] = (0.5 + torch.rand(e, generator=gen, device=dev)) * (0.4 / math.sqrt(k))
    s["row_scale"] = 0.5 + torch.rand(e, n, generator=gen, device=dev) if case["row_scale"] else None
    s["codebook"] = _codebook(str(dev))
    s["y"] = torch.empty(t if case["combine"] else rows, n, dtype=_dtype(case), device=dev)
    if own:
        glq = _glq()
        s["experts"] = glq.Experts(e, n, k, bpw, s["scale"], s["idx1"], s["idx2"], s["sign_k"], s["sign_n"],
                                   _device_tables(str(dev)), s["row_scale"])
        s["workspace"] = torch.zeros(glq.expert_linear_workspace_bytes(s["experts"], rows), dtype=torch.uint8, device=dev)


@functools.lru_cache(maxsize=2)
def _device_tables(device):
    return _glq().device_codebook(device)


# --------------------------------------------------------------- one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"plan": _plain_plan, "rope": _plain_rope, "route": _plain_route, "experts": _plain_experts}[op](s, case)
    glq = _glq()
    if op == "plan":
        p = glq.kv_plan(s["plan"], s["lens"], s["added"], s["free"])
        out = (p.new_lens, p.cu_q, p.slots, p.positions, p.used, s["table"])
        return out + (p.cu_k, p.read_slots) if case["read"] else out
    if op == "rope":
        glq.qk_norm_rope(s["q"], s["k"], s["positions"], s["rotary"], s["q_out"], s["k_out"], s["w"][0], s["w"][1],
                         pairs=case["pairs"], cache=s.get("handle"), v=s["v"] if s["cache"] else None, slots=s["slots"])
        if case["format"] == "int8":
            glq.kv_read(s["handle"], s["slots"], *s["back"])
        return _rope_outputs(s, case, s["back"] if case["format"] == "int8" else None)
    if op == "route":
        glq.route(s["logits"], case["top"], s["weights"], s["ids"], s["pos"], s["src"], s["offsets"], s["workspace"],
                  normalize=case["normalize"])
        return s["weights"], s["ids"], s["pos"], s["src"], s["offsets"]
    return glq.expert_linear(s["experts"], s["x"], s["y"], s["offsets"], s["workspace"], src=s["src"], pos=s["pos"],
                             weights=s["weights"])


def _rope_outputs(s, case, back):
    out = (s["q_out"],) + ((s["k_out"],) if case["dense"] else ())
    if case["format"] == "bf16":
        return out + (s["cache"][0], s["cache"][2])
    return out + tuple(back or ())


def _plain_plan(s, case):
    lens, added, page, table = s["lens"].long(), s["added"].long(), case["page"], s["table"]
    held, total = (lens + page - 1) // page, (lens + added + page - 1) // page
    take = total - held
    first = torch.cumsum(take, 0) - take
    at = torch.arange(table.shape[1], device=table.device)
    which = first[:, None] + at - held[:, None]
    fresh = (at >= held[:, None]) & (at < total[:, None])
    free = torch.cat((s["free"], s["free"].new_full((1,), -1)))
    got = free[which.clamp(0, len(s["free"]))]
    table = torch.where(fresh, got, table)

    def lists(count, begin, most):
        """Offsets, and of every token in a row of `most` its request (batch: none) and number."""
        cu = torch.cat((count.new_zeros(1), torch.cumsum(count, 0)))
        i = torch.arange(most, device=cu.device)
        b = torch.searchsorted(cu[1:].contiguous(), i, right=True)
        safe = b.clamp(max=len(count) - 1)
        t = i - cu[safe] + begin[safe]
        pg = table[safe, (t // page).clamp(0, table.shape[1] - 1)].long()
        slot = torch.where((b < len(count)) & (pg >= 0), pg * page + t % page, -1)
        return cu.to(torch.int32), slot.to(torch.int32), torch.where(b < len(count), t, 0).to(torch.int32)

    cu_q, slots, positions = lists(added, lens, s["most"])
    out = ((lens + added).to(torch.int32), cu_q, slots, positions, take.sum().to(torch.int32).view(1), table)
    if not case["read"]:
        return out
    cu_k, read_slots, _ = lists(lens + added, torch.zeros_like(lens), s["most_read"])
    return out + (cu_k, read_slots)


def _turned(x, w, s, case):
    """float32 rows [tokens, heads, dim], normalised where there are weights, and rotated."""
    x = x.float()
    if w is not None:
        x = x * (w / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6))
    rot = case["rot"]
    cos, sin = s["rotary"][s["positions"].long()][:, None].chunk(2, -1)
    y = x.clone()
    if case["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(s, case):
    s["q_out"].copy_(_turned(s["q"], s["w"][0], s, case))
    k = _turned(s["k"], s["w"][1], s, case).to(s["q"].dtype)
    if case["dense"]:
        s["k_out"].copy_(k)
    if case["format"] == "none":
        return _rope_outputs(s, case, None)
    ck, ks, cv, vs = s["cache"]
    page, off = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
    if case["format"] == "bf16":
        ck[page, :, off], cv[page, :, off] = k.to(ck.dtype), s["v"].to(cv.dtype)
        return _rope_outputs(s, case, None)

    def through(cache, scales, x):
        x = x.float()
        top = x.abs().amax(-1, keepdim=True)
        cache[page, :, off] = torch.where(top > 0, torch.round(x * 127.0 / top), 0.0).to(torch.int8)
        scales[page, :, off] = (top / 127.0).squeeze(-1)
        return (cache[page, :, off].float() * scales[page, :, off].unsqueeze(-1)).to(s["q"].dtype)

    return _rope_outputs(s, case, (through(ck, ks, k), through(cv, vs, s["v"])))


def _plain_route(s, case):
    logits = s["logits"].float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    value, ids = order.values[:, :case["top"]], order.indices[:, :case["top"]]
    ok = value > -math.inf
    among = value if case["normalize"] else logits
    peak = torch.where(ok[:, :1], value[:, :1], 0.0)
    total = torch.exp(among - peak).sum(1, keepdim=True)
    weights = torch.where(ok, torch.exp(value - peak) / torch.where(total > 0, total, 1.0), 0.0)
    ids = torch.where(ok, ids, -1)
    offsets, src, pos = _grouped(ids, case["experts"])
    return weights, ids.to(torch.int32), pos, src, offsets


def _hadamard(x):
    """Block Walsh-Hadamard transform of the last axis, over 1 / sqrt(block)."""
    length = x.shape[-1]
    block = length & -length
    wide = 1 << (block.bit_length() // 2)
    tall = block // wide

    def matrix(b):
        i = torch.arange(b, device=x.device)
        bits = (i[:, None] & i)[..., None] >> torch.arange(15, device=x.device) & 1
        return (1.0 - 2.0 * (bits.sum(-1) % 2)).to(x.dtype)

    y = x.reshape(-1, length // block, tall, wide)
    return (torch.matmul(torch.matmul(matrix(tall), y), matrix(wide)) * block ** -0.5).view(x.shape)


def _plain_experts(s, case):
    e, n, k, rows = case["experts"], case["n"], case["k"], case["tokens"] * case["top"]
    dev = s["x"].device
    r = torch.arange(rows, device=dev)
    of = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    x = (s["x"] if s["src"] is None else s["x"][s["src"].long()]).float()
    x = _hadamard(x * s["sign_k"][of])
    if rows < e:                                              # few rows: each with its own expert's weights
        chosen, group, inside, most = of, r, torch.zeros_like(r), 1
    else:                                                     # rows padded to the busiest expert's
        chosen, group, inside, most = slice(None), of, r - s["offsets"].long()[of], s["most"]
    w = s["codebook"][s["idx1"][chosen].int() & 0xFFFF]
    if s["idx2"] is not None:
        shift = {3: 0.5, 4: 0.25}[case["bpw"]]
        w = w.add_(s["codebook"][s["idx2"][chosen].int() & 0xFFFF], alpha=shift)
    scale = s["scale"][chosen, None]
    if s["row_scale"] is not None:
        scale = scale * s["row_scale"][chosen]
    w = w.view(w.shape[0], n, k).mul_(scale[..., None])
    padded = x.new_zeros(w.shape[0], most, k)
    padded[group, inside] = x
    z = torch.matmul(padded, w.transpose(1, 2))[group, inside]
    y = _hadamard(z) * s["sign_n"][of]
    if s["pos"] is not None:
        y = (y[s["pos"].long()] * s["weights"][..., None]).sum(1)
    return y.to(s["y"].dtype)


# ---------------------------------------------------- the definition, 64 bits

def exact(case, seed):
    if case["op"] == "plan":
        return None                                           # whole numbers alone
    s = prepare(case, seed)
    return {"rope": _exact_rope, "route": _exact_route, "experts": _exact_experts}[case["op"]](s, case)


def _exact_rope(s, case):
    d, rot = case["dim"], case["rot"]
    c, sn = (t.double()[s["positions"].long()] for t in s["rotary"].tensor_split(2, 1))
    turn = torch.complex(c, sn).unsqueeze(1)
    if case["pairs"]:
        first = torch.arange(0, rot, 2, device=c.device)
        second = first + 1
    else:
        first = torch.arange(rot // 2, device=c.device)
        second = first + rot // 2

    def rows(x, w):
        x = x.double()
        if w is not None:
            x = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        out = x.clone()
        out[..., first], out[..., second] = z.real, z.imag
        return out

    q, k = rows(s["q"], s["w"][0]), rows(s["k"], s["w"][1])
    out = (q,) + ((k,) if case["dense"] else ())
    if case["format"] == "none":
        return out
    kept = [k.to(s["k"].dtype).double(), s["v"].double()]
    if case["format"] == "int8":
        tops = [x.abs().max(-1, keepdim=True).values for x in kept]
        return out + tuple(torch.round(x * 127.0 / torch.where(a == 0, 1.0, a)) * a / 127.0 for x, a in zip(kept, tops))
    p, off = torch.div(s["slots"].long(), case["page"], rounding_mode="floor"), s["slots"].long() % case["page"]
    held = [torch.zeros(s["cache"][0].shape, dtype=torch.float64, device=q.device) for _ in range(2)]
    for h, x in zip(held, kept):
        h[p, :, off] = x
    return out + tuple(held)


def _exact_route(s, case):
    e = torch.exp(s["logits"].double())
    e = torch.where(e.isnan(), 0.0, e)
    top = torch.topk(e, case["top"], 1).values
    total = (top if case["normalize"] else e).sum(1, keepdim=True)
    return torch.where(total > 0, top / total, 0.0), None, None, None, None


def _exact_matrix(length, dev):
    """H / sqrt(b), one block, by its recursion."""
    block = 1
    while length % (2 * block) == 0:
        block *= 2
    h = torch.ones(1, 1, dtype=torch.float64, device=dev)
    while h.shape[0] < block:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return h / math.sqrt(block)


def _exact_experts(s, case):
    n, k, top, dev = case["n"], case["k"], case["top"], s["x"].device
    hk, hn = _exact_matrix(k, dev), _exact_matrix(n, dev)
    rows, book = case["tokens"] * top, s["codebook"].double()
    y = torch.zeros(rows, n, dtype=torch.float64, device=dev)
    ends = s["offsets"].tolist()
    for e in range(case["experts"]):
        at = torch.arange(ends[e], ends[e + 1], device=dev)
        if not len(at):
            continue
        x = s["x"][at if s["src"] is None else s["src"].long()[at]].double() * s["sign_k"][e].double()
        x = (x.view(len(at), -1, len(hk)) @ hk).reshape(len(at), k)
        w = book[s["idx1"][e].long() % 65536]
        if case["bpw"] > 2:
            w = w + book[s["idx2"][e].long() % 65536] / (2.0 if case["bpw"] == 3 else 4.0)
        z = x @ w.reshape(n, k).T * s["scale"][e].double()
        if case["row_scale"]:
            z = z * s["row_scale"][e].double()
        y[at] = (z.view(len(at), -1, len(hn)) @ hn).reshape(len(at), n) * s["sign_n"][e].double()
    if s["pos"] is None:
        return y
    out = torch.zeros(case["tokens"], n, dtype=torch.float64, device=dev)
    for j in range(top):
        out += y[s["pos"][:, j].long()] * s["weights"][:, j, None].double()
    return out
