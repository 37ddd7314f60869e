"""A serving step's plan, head norms with rotation, and routing: GPU results against plain
formulas in whole numbers or 64 bits, the refusals of the C ABI and of the binding on the CPU.

Tolerances. u = 2^-24, a float32 rounding.
  norms and rotation   the mean of squares is at most 8 products summed in turn and 5 sums of
           lanes, 13 u; eps, root, quotient, the weight's and x's products 1 u each, the mean's half
           by the root: 11 u; the rotation's product and sum 2 u more, relative to |y_i cos| + |y_j
           sin|: held to 16 u of that, and for bf16 to half a step of the output, 2^-8 of it, on top.
  weights  exp's argument is a rounded difference d, |d| u, and exp itself 2 u, above and below the
           line; sums of positive terms at most 24 u; the quotient 1 u: 2 (|d| + 2) u + 25 u relative
           with |d| the row's range of scores above -inf, and the smallest normal number (2^-126).
Whole numbers, and what the cache holds against glq_kv_append's, are held to equality.
"""
import ctypes
import math

import pytest
import torch

glq = pytest.importorskip("dequant_e8_codebook_amd.glq")

U = 2.0 ** -24
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture
def gen():
    return torch.Generator().manual_seed(5)


# ------------------------------------------------------------------- the plan

def _plan_reference(lens, added, table, free, page, num_pages, max_tokens, max_read):
    """By the words: lists of what glq_kv_plan writes, and the table."""
    table, free, want = [list(r) for r in table], list(free), 0
    slots, positions, read, cu_q, cu_k, new_lens = [], [], [], [0], [0], []
    for b, (n, a) in enumerate(zip(lens, added)):
        n, a = max(n, 0), max(a, 0)
        for e in range(-(-n // page), min(-(-(n + a) // page), len(table[b]))):
            table[b][e] = free[want] if want < len(free) else -1
            want += 1

        def slot(t):
            if t // page >= len(table[b]) or not 0 <= table[b][t // page] < num_pages:
                return -1
            return table[b][t // page] * page + t % page

        slots += [slot(t) for t in range(n, n + a)]
        positions += list(range(n, n + a))
        read += [slot(t) for t in range(n + a)]
        new_lens.append(n + a)
        cu_q.append(min(len(slots), max_tokens))
        cu_k.append(min(len(read), max_read))

    def cut(x, most, fill):
        return x[:most] + [fill] * (most - len(x))

    return {"new_lens": new_lens, "cu_q": cu_q, "slots": cut(slots, max_tokens, -1),
            "positions": cut(positions, max_tokens, 0), "used": [want], "cu_k": cu_k, "read_slots": cut(read, max_read, -1)}, table


def _plan_case(gen, lens, added, page=16, max_pages=None, spare=3, short=0, max_tokens=None, max_read=None):
    held = [-(-max(n, 0) // page) for n in lens]
    total = [-(-(max(n, 0) + max(a, 0)) // page) for n, a in zip(lens, added)]
    max_pages = max(max(total, default=0), 1) if max_pages is None else max_pages
    num = sum(total) + spare
    order = torch.randperm(num, generator=gen).tolist()
    table = torch.full((len(lens), max_pages), -7, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        h = min(h, max_pages)
        table[b, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
        at += h
    free = order[at:len(order) - spare - short]
    max_tokens = sum(max(a, 0) for a in added) + 5 if max_tokens is None else max_tokens
    max_read = sum(max(n, 0) + max(a, 0) for n, a in zip(lens, added)) + 3 if max_read is None else max_read
    return table, torch.tensor(free, dtype=torch.int32), num, max_tokens, max_read


def _check_plan(plan, lens, added, before, free, page, num, after=None):
    ref, table = _plan_reference(lens, added, before.tolist(), free.tolist(), page, num, len(plan.slots),
                                 0 if plan.read_slots is None else len(plan.read_slots))
    for name, want in ref.items():
        got = getattr(plan, name)
        if got is not None:
            assert got.tolist() == want, name
    assert plan.page_table.tolist() == table


def _run_plan(gen, lens, added, page=16, read=True, **how):
    table, free, num, max_tokens, max_read = _plan_case(gen, lens, added, page, **how)
    plan = glq.KvPlan(table.cuda(), page, num, max_tokens, max_read if read else 0)
    glq.kv_plan(plan, *(torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, added)), free.cuda())
    _check_plan(plan, lens, added, table, free, page, num)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64, 1024])
@pytest.mark.parametrize("lens,added", [
    ([0], [1]), ([5], [0]), ([0], [0]), ([15, 16, 17, 0, 31], [1, 1, 1, 1, 1]), ([100, 0, 33, 1], [0, 70, 16, 15]),
    ([-3, 20], [4, -2]), ([4095, 2048, 1], [3, 2049, 4000])])
def test_plan(gen, page, lens, added):
    _run_plan(gen, lens, added, page)
    _run_plan(gen, lens, added, page, read=False)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [63, 64, 257, 1024, 1025, 3000])
def test_plan_many_requests(gen, batch):
    lens = torch.randint(0, 200, (batch,), generator=gen)
    added = torch.randint(0, 40, (batch,), generator=gen) * (torch.rand(batch, generator=gen) < 0.7)
    _run_plan(gen, lens.tolist(), added.tolist())
    _run_plan(gen, lens.tolist(), [1] * batch, short=7)


@pytest.mark.gpu
def test_plan_limits(gen):
    lens, added = [40, 0, 90, 10], [30, 50, 0, 60]
    _run_plan(gen, lens, added, short=4)                               # pages missing
    _run_plan(gen, lens, added, short=10 ** 6, max_tokens=11, max_read=7)      # none, and lists cut
    _run_plan(gen, lens, added, max_pages=3)                           # rows of the table full
    _run_plan(gen, [0] * 40, [500] * 40, max_tokens=1)                 # pages taken whatever the lists hold
    _run_plan(gen, [3] * 1100, [2000] * 1100, max_tokens=64, read=False)
    _run_plan(gen, [100000], [5000])


@pytest.mark.gpu
def test_plan_pages_outside_the_cache():
    table = torch.tensor([[4, 99, -1, 0]], dtype=torch.int32)
    free = torch.tensor([50, 2], dtype=torch.int32)
    plan = glq.KvPlan(table.cuda(), 16, 5, 40, 90)
    lens, added = [48], [32]
    glq.kv_plan(plan, *(torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, added)), free.cuda())
    _check_plan(plan, lens, added, table, free, 16, 5)


@pytest.mark.gpu
def test_plan_nothing():
    plan = glq.KvPlan(torch.zeros(0, 3, dtype=torch.int32).cuda(), 16, 4, 6, 2)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    plan.used.fill_(9)
    glq.kv_plan(plan, none, none, none)
    assert plan.cu_q.tolist() == [0] and plan.cu_k.tolist() == [0] and plan.used.tolist() == [0]
    assert plan.slots.tolist() == [-1] * 6 and plan.positions.tolist() == [0] * 6 and plan.read_slots.tolist() == [-1] * 2


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 1024])
@pytest.mark.parametrize("max_tokens", [0, 15, 16, 17, 1024, 4096, 100000])
@pytest.mark.parametrize("max_read", [0, 40])
def test_plan_no_requests(page, max_tokens, max_read):
    """Every output is written for a batch of none, whatever the lists hold."""
    plan = glq.KvPlan(torch.zeros(0, 3, dtype=torch.int32).cuda(), page, 4, max_tokens, max_read)
    none = torch.zeros(0, dtype=torch.int32).cuda()
    for t in (plan.used, plan.cu_q, plan.slots, plan.positions, plan.cu_k, plan.read_slots):
        if t is not None:
            t.fill_(9)
    glq.kv_plan(plan, none, none, none)
    assert plan.used.tolist() == [0] and plan.cu_q.tolist() == [0]
    assert (plan.slots == -1).all() and (plan.positions == 0).all()
    if max_read:
        assert plan.cu_k.tolist() == [0] and (plan.read_slots == -1).all()


# ------------------------------------------------------ norms and rotation

def _turn_reference(x, weight, eps, cos, sin, pairs):
    """y in float64 and |y_i cos| + |y_j sin| of x [tokens, heads, d] (float64)."""
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    rot = 2 * cos.shape[1]
    if rot == 0:
        return x, x.abs()
    cos, sin = cos.double()[:, None], sin.double()[:, None]
    i = torch.arange(0, rot, 2) if pairs else torch.arange(rot // 2)
    j = i + 1 if pairs else i + rot // 2
    y, mag = x.clone(), x.abs()
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * cos - b * sin, b * cos + a * sin
    mag[..., i], mag[..., j] = (a * cos).abs() + (b * sin).abs(), (b * cos).abs() + (a * sin).abs()
    return y, mag


def _held_turn(got, ref, mag, dtype):
    tol = 16 * U * mag + 1e-38 + (2.0 ** -8 * (ref.abs() + 16 * U * mag) if dtype == "bf16" else 0.0)
    err = (got.double().cpu() - ref).abs()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} of the tolerance"


def _qkv(gen, tokens, heads, kv_heads, dim, dtype):
    """q, k, v as parts of one projection's rows."""
    x = torch.randn(tokens, heads + 2 * kv_heads, dim, generator=gen) * 3
    return x.to(DTYPES[dtype]).cuda().split((heads, kv_heads, kv_heads), 1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (128, 0), (256, 256), (256, 48)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope(gen, dtype, dim, rot, pairs, norm):
    for tokens, heads, kv_heads in [(1, 1, 1), (3, 8, 1), (37, 5, 3), (130, 32, 8)]:
        q, k, _ = _qkv(gen, tokens, heads, kv_heads, dim, dtype)
        positions = torch.randint(0, 500, (tokens,), generator=gen).to(torch.int32)
        table = glq.rotary_table(500, rot, 10000.0, "cpu") if rot else torch.zeros(500, 0)
        w = [1 + 0.5 * torch.randn(dim, generator=gen) for _ in range(2)] if norm else [None, None]
        outs = [torch.full((tokens + 1, h, dim), 7.0, dtype=DTYPES[dtype], device="cuda") for h in (heads, kv_heads)]
        glq.qk_norm_rope(q, k, positions.cuda() if rot else None, table.cuda() if rot else None, outs[0][:tokens], outs[1][:tokens],
                         *(None if t is None else t.cuda() for t in w), eps=1e-5, pairs=pairs)
        cos, sin = table[positions.long()].chunk(2, 1) if rot else (torch.zeros(tokens, 0),) * 2
        for x, out, weight in zip((q, k), outs, w):
            ref, mag = _turn_reference(x.double().cpu(), weight, 1e-5, cos, sin, pairs)
            _held_turn(out[:tokens], ref, mag, dtype)
            assert (out[tokens] == 7).all()
        # in place, on strided rows: the same bits
        before = [t.clone() for t in (q, k)]
        glq.qk_norm_rope(q, k, positions.cuda() if rot else None, table.cuda() if rot else None, q, k,
                         *(None if t is None else t.cuda() for t in w), eps=1e-5, pairs=pairs)
        assert torch.equal(q, outs[0][:tokens]) and torch.equal(k, outs[1][:tokens])
        q.copy_(before[0]), k.copy_(before[1])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("pairs", [False, True])
def test_norm_rope_into_the_cache(gen, fmt, dtype, dim, pairs):
    """The cache holds what glq_kv_append of the outputs writes, bit for bit."""
    form = {"bf16": glq.KV_BF16, "int8": glq.KV_INT8, "int4": glq.KV_INT4}[fmt]
    for tokens, heads, kv_heads, page in [(1, 8, 2, 16), (45, 6, 3, 32), (300, 7, 7, 64)]:
        pages = -(-tokens // page) + 2
        q, k, v = _qkv(gen, tokens, heads, kv_heads, dim, dtype)
        v[tokens // 2] = 0
        slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32)
        if tokens > 3:
            slots[1], slots[3] = -1, pages * page                      # dropped
        slots = slots.cuda()
        positions = torch.arange(tokens, dtype=torch.int32).cuda()
        table, w = glq.rotary_table(tokens, dim), [torch.rand(dim, generator=gen).cuda() + 0.5 for _ in range(2)]
        caches = [glq.KvCache.empty(pages, page, kv_heads, dim, form) for _ in range(3)]
        outs = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k, q)]
        glq.qk_norm_rope(q, k, positions, table, outs[0], outs[1], *w, pairs=pairs)
        glq.kv_append(caches[0], outs[1], v, slots)
        k2 = torch.empty_like(outs[1])
        glq.qk_norm_rope(q, k, positions, table, outs[2], k2, *w, pairs=pairs, cache=caches[1], v=v, slots=slots)
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], k2)
        glq.qk_norm_rope(q, k, positions, table, outs[2], None, *w, pairs=pairs, cache=caches[2], v=v, slots=slots)
        for c in caches[1:]:
            assert torch.equal(caches[0].k, c.k) and torch.equal(caches[0].v, c.v)
            if form != glq.KV_BF16:
                assert torch.equal(caches[0].k_scale, c.k_scale) and torch.equal(caches[0].v_scale, c.v_scale)


def _tokens_of_a_prompt(heads, dim):
    """The fewest tokens of so many heads that are a prompt to the kernel, whose lanes then take several heads each."""
    return -(-2 ** 19 // (heads * dim // 8))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 48)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("heads,kv_heads", [(7, 7), (6, 3), (5, 1), (32, 8)])
def test_norm_rope_of_prompts(gen, dtype, dim, rot, pairs, heads, kv_heads):
    """On both sides of the number of tokens from which lanes take several heads, of counts that four does and does not divide."""
    most = _tokens_of_a_prompt(heads + kv_heads, dim)
    table, w = glq.rotary_table(500, rot, 10000.0, "cpu"), [1 + 0.5 * torch.randn(dim, generator=gen) for _ in range(2)]
    for tokens in (most - 1, most):
        q, k, _ = _qkv(gen, tokens, heads, kv_heads, dim, dtype)
        positions = torch.randint(0, 500, (tokens,), generator=gen).to(torch.int32)
        outs = [torch.full((tokens + 1, h, dim), 7.0, dtype=DTYPES[dtype], device="cuda") for h in (heads, kv_heads)]
        args = (positions.cuda(), table.cuda())
        ws = [t.cuda() for t in w]
        glq.qk_norm_rope(q, k, *args, outs[0][:tokens], outs[1][:tokens], *ws, eps=1e-5, pairs=pairs)
        cos, sin = table[positions.long()].chunk(2, 1)
        for x, out, weight in zip((q, k), outs, w):
            ref, mag = _turn_reference(x.double().cpu(), weight, 1e-5, cos, sin, pairs)
            _held_turn(out[:tokens], ref, mag, dtype)
            assert (out[tokens] == 7).all()
        glq.qk_norm_rope(q, k, *args, q, k, *ws, eps=1e-5, pairs=pairs)
        assert torch.equal(q, outs[0][:tokens]) and torch.equal(k, outs[1][:tokens])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 96), (256, 256)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("heads,kv_heads", [(7, 7), (6, 3), (5, 1), (32, 8)])
def test_norm_rope_of_prompts_into_the_cache(gen, fmt, dtype, dim, rot, pairs, heads, kv_heads):
    """The cache holds what glq_kv_append of the outputs writes, bit for bit, and nothing else of it changes."""
    form, page = {"bf16": glq.KV_BF16, "int8": glq.KV_INT8, "int4": glq.KV_INT4}[fmt], 32
    most = _tokens_of_a_prompt(heads + 2 * kv_heads, dim)
    table, w = glq.rotary_table(most, rot), [torch.rand(dim, generator=gen).cuda() + 0.5 for _ in range(2)]
    for tokens in (most - 1, most):
        pages = -(-tokens // page) + 2
        q, k, v = _qkv(gen, tokens, heads, kv_heads, dim, dtype)
        slots = torch.randperm(pages * page, generator=gen)[:tokens].to(torch.int32)
        slots[1], slots[3], slots[-1] = -1, pages * page, 2 ** 31 - 1
        slots, positions = slots.cuda(), torch.arange(tokens, dtype=torch.int32).cuda()
        caches = [glq.KvCache.empty(pages, page, kv_heads, dim, form) for _ in range(3)]
        outs = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k, q, k)]
        glq.qk_norm_rope(q, k, positions, table, outs[0], outs[1], *w, pairs=pairs, cache=caches[0], v=v, slots=slots)
        glq.kv_append(caches[1], outs[1], v, slots)
        ref, mag = _turn_reference(k.double().cpu(), w[1].cpu(), 1e-6, *table[:tokens].cpu().chunk(2, 1), pairs)
        _held_turn(outs[1], ref, mag, dtype)
        glq.qk_norm_rope(q, k, positions, table, outs[2], None, *w, pairs=pairs, cache=caches[2], v=v, slots=slots)
        assert torch.equal(outs[0], outs[2])
        glq.qk_norm_rope(q, k, positions, table, q, k, *w, pairs=pairs, cache=caches[0], v=v, slots=slots)      # in place
        assert torch.equal(q, outs[0]) and torch.equal(k, outs[1])
        for c in (caches[0], caches[2]):
            assert torch.equal(caches[1].k, c.k) and torch.equal(caches[1].v, c.v)
            if form != glq.KV_BF16:
                assert torch.equal(caches[1].k_scale, c.k_scale) and torch.equal(caches[1].v_scale, c.v_scale)


@pytest.mark.gpu
def test_norm_rope_positions_and_special_values(gen):
    """Positions outside the table are the nearest inside; what is not finite stays in its head."""
    tokens, dim = 6, 64
    q, k, v = _qkv(gen, tokens, 3, 2, dim, "f32")
    q[2, 1, 5], q[3, 0, 9], k[4, 1, 0] = math.nan, math.inf, -math.inf
    q[5, 2], k[0, 0] = 0, 0
    table, w = glq.rotary_table(10, dim), torch.ones(dim, device="cuda")
    outs = [[torch.empty(t.shape, device="cuda") for t in (q, k)] for _ in range(2)]
    for positions, (qo, ko) in zip(([-5, 0, 9, 400, 2 ** 31 - 1, 3], [0, 0, 9, 9, 9, 3]), outs):
        glq.qk_norm_rope(q, k, torch.tensor(positions, dtype=torch.int32).cuda(), table, qo, ko, w, w)
    for a, b in zip(*outs):
        assert torch.equal(a.nan_to_num(7.5), b.nan_to_num(7.5))
    bad_q, bad_k = ~torch.isfinite(outs[0][0]).all(-1).cpu(), ~torch.isfinite(outs[0][1]).all(-1).cpu()
    assert bad_q.nonzero().tolist() == [[2, 1], [3, 0]] and bad_k.nonzero().tolist() == [[4, 1]]
    assert (outs[0][0][5, 2] == 0).all() and (outs[0][1][0, 0] == 0).all()


# ------------------------------------------------------------------- routing

def _route_reference(logits, top, normalize):
    """By the words, token by token, on float64 scores."""
    tokens, experts = logits.shape
    x = logits.double()
    weights, ids = torch.zeros(tokens, top, dtype=torch.float64), torch.full((tokens, top), -1)
    reach = torch.zeros(tokens, 1, dtype=torch.float64)
    rows = [[] for _ in range(experts)]
    for t in range(tokens):
        ok = [e for e in range(experts) if x[t, e] > -math.inf]
        pick = sorted(ok, key=lambda e: (-x[t, e].item(), e))[:top]
        if not pick:
            continue
        among = torch.tensor(pick if normalize else ok)
        peak = x[t, pick[0]]
        total = torch.exp(x[t, among] - peak).sum()
        reach[t] = peak - x[t, torch.tensor(ok)].min()
        for j, e in enumerate(pick):
            ids[t, j], weights[t, j] = e, torch.exp(x[t, e] - peak) / total
            rows[e].append((t, j))
    pos, src, offsets = torch.full((tokens, top), -1), [], [0]
    for r in rows:
        for t, j in r:
            pos[t, j] = len(src)
            src.append(t)
        offsets.append(len(src))
    return weights, reach, ids, pos, src + [-1] * (tokens * top - len(src)), offsets


def _route_buffers(tokens, experts, top, fill=77):
    return (torch.full((tokens, top), 7.0, device="cuda"), *(torch.full(s, fill, dtype=torch.int32, device="cuda")
            for s in ((tokens, top), (tokens, top), (tokens * top,), (experts + 1,))),
            torch.randint(0, 255, (glq.route_workspace_bytes(tokens, experts, top),), dtype=torch.uint8, device="cuda"))


def _check_route(logits, top, normalize, outs):
    weights, reach, ids, pos, src, offsets = _route_reference(logits, top, normalize)
    assert outs[1].tolist() == ids.tolist() and outs[2].tolist() == pos.tolist()
    assert outs[3].tolist() == src and outs[4].tolist() == offsets
    tol = (2 * (reach + 2) + 25) * U * weights + 2.0 ** -126
    assert ((outs[0].double().cpu() - weights).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [0, 1, 5, 64, 65, 333])
@pytest.mark.parametrize("experts,top", [(1, 1), (8, 2), (60, 4), (64, 64), (65, 1), (160, 6), (257, 8), (600, 3), (1024, 10)])
@pytest.mark.parametrize("dtype,normalize", [("f32", True), ("bf16", False)])
def test_route(gen, tokens, experts, top, dtype, normalize):
    logits = (2 * torch.randn(tokens, experts, generator=gen)).to(DTYPES[dtype])
    if tokens > 4:
        logits[0, ::2] = -math.inf                                     # fewer than top_k are left
        logits[1] = -math.inf
        logits[2] = math.nan
        logits[3] = torch.finfo(logits.dtype).min                      # a mask of the lowest value: scores like others
        logits[4] = 0.0
        logits[4, 1::3] = -0.0                                         # equal: the lowest index
        logits[-1, experts // 2] = math.nan
    outs = _route_buffers(tokens, experts, top)
    glq.route(logits.cuda(), top, *outs, normalize=normalize)
    _check_route(logits, top, normalize, outs)


@pytest.mark.gpu
def test_route_many_tokens(gen):
    logits = torch.randn(5000, 40, generator=gen).round()              # equal scores everywhere
    logits[4000:4100] = -math.inf
    outs = _route_buffers(5000, 40, 6)
    glq.route(logits.cuda(), 6, *outs)
    _check_route(logits, 6, True, outs)
    logits = torch.full((130, 4), 0.0)
    logits[:, 2] = 90.0                                                # all to one expert
    outs = _route_buffers(130, 4, 1)
    glq.route(logits.cuda(), 1, *outs, normalize=False)
    _check_route(logits, 1, False, outs)


@pytest.mark.gpu
def test_route_infinite_score():
    logits = torch.tensor([[0.0, math.inf, 1.0], [1.0, 2.0, 3.0]])
    outs = _route_buffers(2, 3, 2)
    glq.route(logits.cuda(), 2, *outs)
    assert outs[1].tolist() == [[1, 2], [2, 1]] and outs[0][0].isnan().any() and not outs[0][1].isnan().any()


# ------------------------------------------------- refusals (nothing is launched)

def _plan_struct(**change):
    """A struct that would be taken, its pointers never followed on the host."""
    p = 4096
    st = glq.PlanStruct(2, 4, 100, 16, p, p + 64, p + 128, 5, p + 256, p + 512, p + 576, 7, p + 640, p + 768, 9, p + 896,
                        p + 960, p + 1024)
    for name, value in change.items():
        setattr(st, name, value)
    return ctypes.byref(st)


@pytest.mark.parametrize("change,status", [
    ({"batch": -1}, -1), ({"max_pages": 0}, -1), ({"num_pages": 0}, -1), ({"page_size": 24}, -1), ({"page_size": 8}, -1),
    ({"page_size": 2048}, -1), ({"num_free": -1}, -1), ({"max_tokens": -1}, -1), ({"max_read": -1}, -1), ({"lens": 0}, -1),
    ({"added": 0}, -1), ({"free_pages": 0}, -1), ({"page_table": 0}, -1), ({"new_lens": 0}, -1), ({"cu_q": 0}, -1),
    ({"slots": 0}, -1), ({"positions": 0}, -1), ({"cu_k": 0}, -1), ({"read_slots": 0}, -1), ({"used": 0}, -1),
    ({"lens": 4098}, -1), ({"new_lens": 4096}, -1), ({"num_pages": 2 ** 40}, -2), ({"max_pages": 2 ** 40}, -2),
    ({"max_tokens": 2 ** 31}, -2), ({"max_read": 2 ** 31}, -2), ({"batch": 2 ** 40}, -2)])
def test_plan_refusals(change, status):
    assert glq.raw().glq_kv_plan(_plan_struct(**change), None) == status


def test_plan_refuses_no_struct():
    assert glq.raw().glq_kv_plan(None, None) == -1


def _qk_struct(**change):
    p = 4096
    st = glq.QkStruct(p, p, p, p, 1, 4, 2, 64, 256, 128, 256, 128, 3, p, p, 1e-6, 64, p, p, 10, p, 128, p)
    for name, value in change.items():
        setattr(st, name, value)
    return ctypes.byref(st)


def _cache_struct(**change):
    st = glq.KvCacheStruct(0, 2, 64, 16, 4, 4096, 4096, 0, 0)
    for name, value in change.items():
        setattr(st, name, value)
    return ctypes.byref(st)


@pytest.mark.parametrize("change,status", [
    ({"dt": 2}, -1), ({"q_heads": 0}, -1), ({"kv_heads": 0}, -1), ({"head_dim": 96}, -2), ({"rotary_dim": 24}, -2),
    ({"rotary_dim": 80}, -1), ({"rotary_dim": -16}, -1), ({"tokens": -1}, -1), ({"eps": -1.0}, -1), ({"eps": math.nan}, -1),
    ({"eps": math.inf}, -1), ({"q": 0}, -1), ({"k": 0}, -1), ({"q_out": 0}, -1), ({"q": 4104}, -1), ({"q_stride": 248}, -1),
    ({"k_stride": 129}, -1), ({"q_out_stride": 0}, -1), ({"q_weight": 4100}, -1), ({"positions": 0}, -1),
    ({"rotary": 0}, -1), ({"rotary": 4100}, -1), ({"max_positions": 0}, -1), ({"v": 0}, -1), ({"slots": 0}, -1),
    ({"slots": 4097}, -1), ({"tokens": 2 ** 45}, -2), ({"tokens": 2 ** 31}, -2)])
def test_norm_rope_refusals(change, status):
    assert glq.raw().glq_qk_norm_rope(_qk_struct(**change), _cache_struct(), 0, None) == status


def test_norm_rope_refuses_caches_and_flags():
    call = glq.raw().glq_qk_norm_rope
    assert call(None, None, 0, None) == -1
    assert call(_qk_struct(), _cache_struct(), 2, None) == -1
    assert call(_qk_struct(), _cache_struct(kv_heads=4), 0, None) == -1
    assert call(_qk_struct(), _cache_struct(head_dim=128), 0, None) == -1
    assert call(_qk_struct(), _cache_struct(format=1), 0, None) == -1
    assert call(_qk_struct(k_out=0), None, 0, None) == -1
    assert call(_qk_struct(tokens=0), None, 0, None) == 0


def _route_args(**change):
    p = 4096
    a = dict(logits=p, dt=0, tokens=100, experts=8, top=2, flags=1, weights=p, ids=p, pos=p, src=p, offsets=p, ws=p,
             ws_bytes=1 << 20)
    a.update(change)
    return tuple(a.values()) + (None,)


@pytest.mark.parametrize("change,status", [
    ({"dt": 5}, -1), ({"flags": 2}, -1), ({"tokens": -1}, -1), ({"experts": 0}, -1), ({"top": 0}, -1), ({"top": 9}, -1),
    ({"experts": 1025}, -2), ({"experts": 100, "top": 65}, -2), ({"tokens": 2 ** 26}, -2), ({"logits": 0}, -1),
    ({"logits": 4098}, -1), ({"weights": 0}, -1), ({"ids": 0}, -1), ({"pos": 0}, -1), ({"src": 0}, -1), ({"offsets": 0}, -1),
    ({"offsets": 4097}, -1), ({"src": 4098}, -1), ({"ws": 0}, -4), ({"ws": 4100}, -4), ({"ws_bytes": 256}, -4)])
def test_route_refusals(change, status):
    assert glq.raw().glq_route(*_route_args(**change)) == status
    if status == -2:
        assert glq.route_workspace_bytes(change.get("tokens", 100), change.get("experts", 8), change.get("top", 2)) == 0


def test_binding_refuses_host_tensors():
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        glq.KvPlan(torch.zeros(2, 3, dtype=torch.int32), 16, 4, 5)
    with pytest.raises(ValueError):
        glq.qk_norm_rope(torch.zeros(2, 1, 64), torch.zeros(2, 1, 64), ints, torch.zeros(4, 64), torch.zeros(2, 1, 64),
                         torch.zeros(2, 1, 64))
    with pytest.raises(ValueError):
        glq.route(torch.zeros(2, 3), 1, torch.zeros(2, 1), ints, ints, ints, ints, torch.zeros(4))
