"""The paged key-value cache and the attention over it: GPU results against
plain 64-bit formulas, the refusals of the C ABI and of the binding on the CPU.

Tolerances. With A = sum_j p_j |v_j| (the same weights, absolute values):
  float32  1e-5 A: a score's error is a few float32 roundings of |s| <= ~30 (at
           most ~100 units of 2^-24 = 6e-6), and it is the weight's relative error;
  bf16     2^-9 (A + |o|) for the output's own rounding (at most 2^-8 |o|, and A >=
           |o|), 1e-5 A for the rest: the weights keep 16 bits or more;
  prompts in bf16   2^-8 A on top: each weight is rounded to bf16, 2^-8 relative
           (1 + 2^-8 rounds to 1), while their sum is not.
Codes, scales and values read back are held to equality: for bf16 inputs Q x is
exact in float32 and Q x / a is a quotient of 8-bit numbers times Q, further than
a float32 rounding from every half unless it is one.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

glq = pytest.importorskip("dequant_e8_codebook_amd.glq")

FORMATS = {"bf16": glq.KV_BF16, "int8": glq.KV_INT8, "int4": glq.KV_INT4}
LEVELS = {"int8": 127, "int4": 7}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture
def gen():
    return torch.Generator().manual_seed(11)


def _normal(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen).to(dtype)


# ------------------------------------------------------------- 64-bit formulas

def _ref_codes(x, fmt):
    """Codes (float64) and scales (float32) of x [..., d] (float64)."""
    top = x.abs().amax(-1, keepdim=True)
    q = LEVELS[fmt]
    code = torch.where(top > 0, torch.round(x * q / torch.where(top > 0, top, 1.0)), torch.zeros_like(x))
    return code, (top / q).squeeze(-1).to(torch.float32)


def _ref_values(x, fmt):
    """float32 values that the cache stands for."""
    if fmt == "bf16":
        return x.to(torch.bfloat16).to(torch.float32)
    code, scale = _ref_codes(x.double(), fmt)
    return code.to(torch.float32) * scale[..., None]


def _ref_attend(q, k, v, scale, seen):
    """float64 attention of q [n, d] over k, v [m, d], seen [n, m] bool: the result
    and A = sum p |v|; rows that see nothing are zero."""
    q, k, v = q.double(), k.double(), v.double()
    out, mag = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64), torch.zeros(q.shape[0], v.shape[1],
                                                                                      dtype=torch.float64)
    rows = seen.any(1)
    if rows.any():
        s = (q[rows] @ k.T) * scale
        s = s.masked_fill(~seen[rows], -math.inf)
        p = torch.softmax(s, 1)
        out[rows] = p @ v
        mag[rows] = p @ v.abs()
    return out, mag


def _held(got, ref, mag, dtype, rounded_weights=False):
    tol = 1e-5 * mag + (0 if dtype == "f32" else 2.0 ** -9 * 1.01 * (mag + ref.abs())) + 1e-30
    if rounded_weights and dtype == "bf16":
        tol = tol + 2.0 ** -8 * mag
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3g} of the tolerance"


# -------------------------------------------------------------- write and read

def _slots(gen, tokens, capacity):
    return torch.randperm(capacity, generator=gen)[:tokens].to(torch.int32)


def _unpack(cache):
    """Codes of a quantised cache as float64 [pages, heads, page, d]."""
    out = []
    for t in (cache.k, cache.v):
        t = t.cpu()
        if cache.format == glq.KV_INT4:
            t = torch.stack(((t & 15).to(torch.int32) - 8, (t >> 4).to(torch.int32) - 8), -1).flatten(-2)
        out.append(t.double())
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("tokens,heads,dim,page,dtype", [(1, 1, 64, 16, "bf16"), (37, 3, 128, 16, "bf16"),
                                                         (130, 8, 64, 64, "f32"), (77, 5, 256, 32, "bf16"),
                                                         (1000, 2, 128, 1024, "bf16")])
def test_append_and_read(gen, fmt, tokens, heads, dim, page, dtype):
    pages = -(-tokens // page) + 2
    cache = glq.KvCache.empty(pages, page, heads, dim, FORMATS[fmt])
    slots = _slots(gen, tokens, pages * page)
    # k and v as halves of one projection's rows: strided
    kv = _normal(gen, tokens, 2 * heads, dim, dtype=torch.bfloat16) * 3
    kv[tokens // 2, 0] = 0
    kv = kv.to(DTYPES[dtype]).cuda()
    k, v = kv[:, :heads], kv[:, heads:]
    dropped = torch.full_like(slots, -1)
    dropped[0] = pages * page
    glq.kv_append(cache, k, v, dropped.cuda())
    assert not cache.k.any() and not cache.v.any()
    glq.kv_append(cache, k, v, slots.cuda())
    for fill, dt in ((7.0, torch.bfloat16), (7.0, torch.float32)):
        ko, vo = (torch.full((tokens + 1, heads, dim), fill, dtype=dt, device="cuda") for _ in range(2))
        where = torch.cat((slots, torch.tensor([-5], dtype=torch.int32))).cuda()
        glq.kv_read(cache, where, ko, vo)
        for x, o in ((k, ko), (v, vo)):
            want = _ref_values(x.cpu().float(), fmt)
            assert torch.equal(o[:tokens].cpu(), want.to(dt))
            assert not o[tokens].any()               # a slot outside the cache
    if fmt != "bf16":
        at = slots.long()
        for x, codes, scale in ((k, _unpack(cache)[0], cache.k_scale), (v, _unpack(cache)[1], cache.v_scale)):
            code, s = _ref_codes(x.cpu().double(), fmt)
            assert torch.equal(codes[at // page, :, at % page], code)
            assert torch.equal(scale.cpu()[at // page, :, at % page], s)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "int4"])
def test_append_special_values(fmt):
    big = 3e38
    rows = [[math.nan, 1.0], [math.inf, 1.0], [-math.inf, math.nan], [big, -big / 2], [1e-30, -1e-30], [0.0, -0.0],
            [big, 1e-30]]
    x = torch.zeros(len(rows), 1, 64)
    for i, r in enumerate(rows):
        x[i, 0, 5], x[i, 0, 40] = r
    cache = glq.KvCache.empty(1, 16, 1, 64, FORMATS[fmt])
    slots = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    glq.kv_append(cache, x.cuda(), x.cuda(), slots)
    ko, vo = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    glq.kv_read(cache, slots, ko, vo)
    ko = ko.cpu()
    assert torch.equal(torch.nan_to_num(ko, 7.0), torch.nan_to_num(vo.cpu(), 7.0))
    assert torch.isnan(ko[:3]).all()
    q = LEVELS[fmt]
    for i in (3, 4, 6):
        assert ko[i, 0, 5].item() == pytest.approx(rows[i][0], rel=1e-6)
        assert abs(ko[i, 0, 40].item() - rows[i][1]) <= abs(rows[i][0]) / (2 * q) * 1.0001
    assert not ko[5].any()


# ------------------------------------------------------------------ one new token

def _decode_case(gen, fmt, lens, q_heads, kv_heads, dim, page, dtype, spread=1.5, stride=0):
    """A cache filled through shuffled pages, garbage wherever no token is."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    if fmt == "bf16":
        k, v = (_normal(gen, pages, kv_heads, page, dim, dtype=torch.bfloat16) for _ in range(2))
        parts = [k, v, None, None]
        dense = (k.float(), v.float())
    else:
        parts, dense = [], []
        for _ in range(2):
            code, scale = _ref_codes(_normal(gen, pages, kv_heads, page, dim).double(), fmt)
            dense.append(code.to(torch.float32) * scale[..., None])
            c = code.to(torch.int8) if fmt == "int8" else ((code[..., 0::2] + 8).to(torch.uint8)
                                                           | (code[..., 1::2] + 8).to(torch.uint8) << 4)
            parts += [c, scale]
        parts = [parts[0], parts[2], parts[1], parts[3]]
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    most = max(1, max(need)) + 1
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    table[:, -1] = 2 ** 31 - 1
    used = torch.zeros(pages, page, dtype=torch.bool)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        for i in range(n):
            used[order[at + i].item(), :min(page, lens[b] - i * page)] = True
        at += n
    free = ~used[:, None, :].expand(pages, kv_heads, page)
    for t in parts[2:] if fmt != "bf16" else parts[:2]:
        t[free] = math.nan
    q = _normal(gen, len(lens), q_heads + stride, dim, dtype=DTYPES[dtype]) * spread
    q = q.cuda()[:, :q_heads]
    cache = glq.KvCache(*[None if t is None else t.contiguous().cuda() for t in parts])
    ref = torch.zeros(len(lens), q_heads, dim, dtype=torch.float64)
    mag = torch.zeros_like(ref)
    for b, n in enumerate(lens):
        if not n:
            continue
        pg, off = table[b].long()[torch.arange(n) // page], torch.arange(n) % page
        for h in range(kv_heads):
            kk, vv = dense[0][pg, h, off], dense[1][pg, h, off]
            r = slice(h * (q_heads // kv_heads), (h + 1) * (q_heads // kv_heads))
            ref[b, r], mag[b, r] = _ref_attend(q[b, r].cpu(), kk, vv, dim ** -0.5,
                                               torch.ones(q_heads // kv_heads, n, dtype=torch.bool))
    return cache, q, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), ref, mag


def _decode(cache, q, table, lens, max_len, workspace=None, **kw):
    if workspace is None:
        workspace = torch.zeros(glq.attn_decode_workspace_bytes(cache, q.shape[0], q.shape[1], max_len),
                                dtype=torch.uint8, device="cuda")
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), 7.0, dtype=q.dtype, device="cuda")
    glq.attn_decode(cache, q, table, lens, out, workspace, max_len, **kw)
    return out, workspace


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_decode_lengths(gen, fmt, dim, dtype):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 65, 127, 128, 129, 300]
    cache, q, table, ln, ref, mag = _decode_case(gen, fmt, lens, 6, 2, dim, 16, dtype, stride=1)
    out, ws = _decode(cache, q, table, ln, 300)
    _held(out, ref, mag, dtype)
    assert not out[0].any()                          # no tokens: zeros
    assert not ws[:65536].any()                      # control words left as they were


@pytest.mark.gpu
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (16, 1), (17, 1), (40, 2), (24, 3), (7, 7)])
@pytest.mark.parametrize("fmt,page", [("bf16", 32), ("int8", 64), ("int4", 128)])
def test_decode_groups_and_pages(gen, q_heads, kv_heads, fmt, page):
    lens = [200, 0, 77, 1]
    cache, q, table, ln, ref, mag = _decode_case(gen, fmt, lens, q_heads, kv_heads, 128, page, "bf16")
    out, _ = _decode(cache, q, table, ln, 200)
    _held(out, ref, mag, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("int8", "f32"), ("int4", "bf16"), ("int4", "f32")])
@pytest.mark.parametrize("spread", [1.5, 0.0])
def test_decode_long(gen, fmt, dtype, spread):
    # long enough that the work is split over the length; spread 0: every token
    # has the same weight, the largest cancellation of the sums
    lens = [20011, 9000, 3]
    cache, q, table, ln, ref, mag = _decode_case(gen, fmt, lens, 4, 1, 128, 64, dtype, spread=spread)
    out, ws = _decode(cache, q, table, ln, 20011)
    _held(out, ref, mag, dtype)
    again, ws = _decode(cache, q, table, ln, 20011, ws)
    assert torch.equal(out, again)                   # and the order of the workgroups does not show
    # lens are read as at most max_len
    few, _ = _decode(cache, q, table, torch.full_like(ln, 2 ** 30), 3, ws)
    assert torch.equal(few[2], out[2])


@pytest.mark.gpu
def test_decode_peaked_and_extreme_scores(gen):
    # one token far ahead of the rest (early, or in the last tile), and scores of
    # +-1e4, whose differences leave the range of exp
    for at in (3, 498):
        cache, q, table, ln, _, _ = _decode_case(gen, "bf16", [500], 2, 1, 64, 16, "bf16")
        pg = table[0, at // 16].item()
        cache.k[pg, 0, at % 16] = (q[0, 0].float() * 100).to(torch.bfloat16)
        out, _ = _decode(cache, q, table, ln, 500)
        assert torch.equal(out[0, 0], cache.v[pg, 0, at % 16])
        assert torch.isfinite(out).all()


@pytest.mark.gpu
def test_decode_scale_stream_and_graph(gen):
    lens = [1500, 20]
    cache, q, table, ln, ref, mag = _decode_case(gen, "int8", lens, 8, 2, 128, 32, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, ws = _decode(cache, q, table, ln, 1500)
        also, ws = _decode(cache, (q.float() * 2).to(torch.bfloat16), table, ln, 1500, ws, scale=0.5 * 128 ** -0.5)
    side.synchronize()
    _held(out, ref, mag, "bf16")
    assert torch.equal(out, also)                    # twice the query at half the scale
    res = torch.zeros_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        glq.attn_decode(cache, q, table, ln, res, ws, 1500)
    for _ in range(3):
        res.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, out)
        ln.copy_(ln)                                 # eager work in between
        torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("batch,fmt,dtype", [(70, "int8", "bf16"), (130, "int4", "bf16"), (65, "bf16", "f32")])
def test_decode_many_sequences(gen, batch, fmt, dtype):
    # more than 64 sequences: the parts are found in another way; one sequence far
    # longer than the rest, and empty ones
    lens = [int(x) for x in torch.randint(0, 200, (batch,), generator=gen)]
    lens[0], lens[5], lens[batch - 1] = 0, 3000, 17
    cache, q, table, ln, ref, mag = _decode_case(gen, fmt, lens, 4, 2, 64, 16, dtype)
    out, ws = _decode(cache, q, table, ln, 3000)
    _held(out, ref, mag, dtype)
    assert not ws[:65536].any()


@pytest.mark.gpu
def test_decode_one_workspace_for_many_calls(gen):
    # one workspace, large enough for all, under batches and lengths that change
    cases = [_decode_case(gen, "int8", lens, 8, 2, 128, 32, "bf16")
             for lens in ([5000], [40] * 9, [1, 700, 0], [3000, 2999, 12, 1024])]
    size = max(glq.attn_decode_workspace_bytes(c[0], c[1].shape[0], 8, 5000) for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for cache, q, table, ln, ref, mag in cases:
            out, _ = _decode(cache, q, table, ln, int(ln.max()), ws)
            _held(out, ref, mag, "bf16")
            assert not ws[:65536].any()


@pytest.mark.gpu
def test_decode_nothing_cached(gen):
    cache, q, table, ln, _, _ = _decode_case(gen, "bf16", [0, 0, 0], 2, 1, 64, 16, "bf16")
    out, _ = _decode(cache, q, table, ln, 0)
    assert not out.any()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_cache_beyond_32_bits(gen, fmt):
    # pages whose rows lie past 2^32 bytes (and 2^31 elements) into the cache
    heads, dim, page = 8, 128, 64
    pages = 2 ** 32 // (heads * page * dim) + 40
    dt = torch.int8 if fmt == "int8" else torch.bfloat16
    k, v = (torch.empty(pages, heads, page, dim, dtype=dt, device="cuda") for _ in range(2))
    scales = [torch.empty(pages, heads, page, device="cuda") for _ in range(2)] if fmt == "int8" else [None, None]
    cache = glq.KvCache(k, v, *scales)
    n = 150
    x, y = (_normal(gen, n, heads, dim, dtype=torch.bfloat16).cuda() for _ in range(2))
    table = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    slots = (table[0].long()[at // page] * page + at % page).to(torch.int32)
    glq.kv_append(cache, x, y, slots)
    xo, yo = torch.empty_like(x), torch.empty_like(y)
    glq.kv_read(cache, slots, xo, yo)
    assert torch.equal(xo.cpu(), _ref_values(x.cpu().float(), fmt).to(torch.bfloat16))
    assert torch.equal(yo.cpu(), _ref_values(y.cpu().float(), fmt).to(torch.bfloat16))
    q = _normal(gen, 1, 16, dim, dtype=torch.bfloat16).cuda()
    out, _ = _decode(cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    kk, vv = (_ref_values(z.cpu().float(), fmt) for z in (x, y))
    for h in range(16):
        ref, mag = _ref_attend(q[0, h:h + 1].cpu(), kk[:, h // 2], vv[:, h // 2], dim ** -0.5, torch.ones(1, n, dtype=torch.bool))
        _held(out[0, h:h + 1], ref, mag, "bf16")
    del cache, k, v, scales
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------ prompts

def _prompt_case(gen, lens_q, lens_k, q_heads, kv_heads, dim, dtype, causal, scale=None, fused=False):
    dt = DTYPES[dtype]
    tq, tk = sum(lens_q), sum(lens_k)
    if fused:                                        # q, k and v as parts of one projection's rows
        qkv = _normal(gen, tq, q_heads + 2 * kv_heads, dim, dtype=dt).cuda()
        q, k, v = qkv[:, :q_heads], qkv[:, q_heads:q_heads + kv_heads], qkv[:, q_heads + kv_heads:]
    else:
        q = (_normal(gen, tq, q_heads, dim, dtype=dt) * 1.5).cuda()
        k, v = (_normal(gen, tk, kv_heads, dim, dtype=dt).cuda() for _ in range(2))
    cu_q, cu_k = (torch.tensor(np.concatenate(([0], np.cumsum(x))), dtype=torch.int32) for x in (lens_q, lens_k))
    ref, mag = torch.zeros(tq, q_heads, dim, dtype=torch.float64), torch.zeros(tq, q_heads, dim, dtype=torch.float64)
    qc, kc, vc = q.cpu(), k.cpu(), v.cpu()
    for b, (n, m) in enumerate(zip(lens_q, lens_k)):
        a, c = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
        seen = torch.ones(n, m, dtype=torch.bool)
        if causal:
            seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
        for h in range(q_heads):
            g = h // (q_heads // kv_heads)
            ref[a, h], mag[a, h] = _ref_attend(qc[a, h], kc[c, g], vc[c, g], scale or dim ** -0.5, seen)
    return q, k, v, cu_q.cuda(), cu_k.cuda(), ref, mag


def _prompt(q, k, v, cu_q, cu_k, **kw):
    out = torch.full((q.shape[0], q.shape[1], q.shape[2]), 7.0, dtype=q.dtype, device="cuda")
    return glq.attn_prompt(q, k, v, out, cu_q, cu_k, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths(gen, dtype, dim, causal):
    lens = [1, 0, 2, 31, 32, 33, 64, 0, 65, 127, 129, 200]
    q, k, v, cu, _, ref, mag = _prompt_case(gen, lens, lens, 4, 2, dim, dtype, causal, fused=True)
    _held(_prompt(q, k, v, cu, None, max_q=200, causal=causal), ref, mag, dtype, True)
    _held(_prompt(q, k, v, cu, None, causal=causal), ref, mag, dtype, True)     # max_q left at the total


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (12, 4), (7, 7), (9, 1)])
def test_prompt_prefixes_and_empty_rows(gen, dtype, causal, q_heads, kv_heads):
    # keys before the queries (a cached prefix), one token on a prefix, fewer
    # keys than queries (causal: the first rows see nothing), no keys at all
    lens_q, lens_k = [40, 1, 70, 5, 3], [300, 257, 30, 0, 3]
    q, k, v, cu_q, cu_k, ref, mag = _prompt_case(gen, lens_q, lens_k, q_heads, kv_heads, 64, dtype, causal)
    out = _prompt(q, k, v, cu_q, cu_k, max_q=70, causal=causal)
    _held(out, ref, mag, dtype, True)
    if causal:
        assert not out[41:41 + 40].any()
    assert not out[111:116].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dim,causal", [("bf16", 128, True), ("bf16", 128, False), ("f32", 64, True)])
def test_prompt_long(gen, dtype, dim, causal):
    lens = [1111, 700]
    q, k, v, cu, _, ref, mag = _prompt_case(gen, lens, lens, 4, 1, dim, dtype, causal)
    _held(_prompt(q, k, v, cu, None, max_q=1111, causal=causal), ref, mag, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_few_rows_on_many_keys(gen, dim, causal):
    # rows enough for a part of the card only: keys up to several tiles of each wave,
    # tiles that only some waves have, sequences without keys or queries
    lens_q, lens_k = [3, 1, 40, 0, 5, 70], [700, 64, 1030, 300, 0, 65]
    q, k, v, cu_q, cu_k, ref, mag = _prompt_case(gen, lens_q, lens_k, 6, 2, dim, "bf16", causal)
    out = _prompt(q, k, v, cu_q, cu_k, max_q=70, causal=causal)
    _held(out, ref, mag, "bf16", True)
    assert torch.equal(out, _prompt(q, k, v, cu_q, cu_k, max_q=70, causal=causal))
    if causal:                                       # keys that only the last of 40 queries sees
        at = 64 + 700 + 1029
        k[at, 1, 0], v[at, 1, 7], v[at, 1, dim - 2] = 0.5, math.nan, math.inf
        got = _prompt(q, k, v, cu_q, cu_k, max_q=70, causal=causal)
        assert torch.isnan(got[43, 3:, 7]).all() and not torch.isfinite(got[43, 3:, dim - 2]).any()
        got[43], out[43] = 0, 0
        assert torch.isfinite(got).all()
        _held(got[:43], ref[:43], mag[:43], "bf16", True)
        assert torch.equal(got[44:], out[44:])


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_many_float32_rows(gen, causal):
    lens_q, lens_k = [520, 505, 33], [520, 515, 33]
    q, k, v, cu_q, cu_k, ref, mag = _prompt_case(gen, lens_q, lens_k, 64, 64, 64, "f32", causal)
    at = 520 + 514                                   # a value that the last of 505 queries sees alone
    got = _prompt(q, k, v, cu_q, cu_k, max_q=520, causal=causal)
    _held(got, ref, mag, "f32", True)
    if causal:
        v[at, 5, 9] = math.nan
        nan = torch.isnan(_prompt(q, k, v, cu_q, cu_k, max_q=520))
        assert nan[1024, 5, 9] and nan.sum() == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_heads,kv_heads,lens", [(300, 2, [3, 40, 1]), (131, 1, [130, 7]), (129, 3, [64, 129])])
def test_prompt_large_groups(gen, dtype, q_heads, kv_heads, lens):
    # a query's heads over several tiles of rows, tiles that begin within a query
    q, k, v, cu, _, ref, mag = _prompt_case(gen, lens, lens, q_heads, kv_heads, 64, dtype, True)
    _held(_prompt(q, k, v, cu, None, max_q=max(lens)), ref, mag, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_rows_for_the_whole_card(gen, dim, causal):
    lens_q, lens_k = [400, 90, 33, 301], [430, 90, 600, 301]
    q, k, v, cu_q, cu_k, ref, mag = _prompt_case(gen, lens_q, lens_k, 24, 3, dim, "bf16", causal)
    _held(_prompt(q, k, v, cu_q, cu_k, max_q=400, causal=causal), ref, mag, "bf16", True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_unseen_values_do_not_reach(gen, dtype, dim):
    # NaN and infinities in keys and values that only later queries see
    n = 150
    for where in (0, 17, 70, 149):
        q, k, v, cu, _, ref, mag = _prompt_case(gen, [n, 40], [n, 40], 2, 1, dim, dtype, True)
        k[where, 0, 3], v[where, 0, 5], v[where, 0, dim - 1] = math.inf, math.nan, -math.inf
        out = _prompt(q, k, v, cu, None, max_q=n)
        _held(out[:where], ref[:where], mag[:where], dtype, True)
        _held(out[n:], ref[n:], mag[n:], dtype, True)
        # value dimension 5 of a query that sees the NaN with a finite weight
        k[where, 0, 3] = 0.5
        out = _prompt(q, k, v, cu, None, max_q=n)
        assert torch.isnan(out[where:n, :, 5]).all()
        assert not torch.isfinite(out[where:n, :, dim - 1]).any()
        assert torch.isfinite(out[where:n, :, 6]).all() and torch.isfinite(out[:where]).all()
        assert torch.isfinite(out[n:]).all()


@pytest.mark.gpu
def test_prompt_rows_outside_sequences_and_wide_offsets(gen):
    # offsets that do not start at 0 or end at the total: other rows stay as
    # they are; offsets past the rows are read as the nearest
    q, k, v, cu, _, ref, mag = _prompt_case(gen, [20, 30], [20, 30], 2, 2, 64, "bf16", True)
    cu2 = torch.tensor([20, 50], dtype=torch.int32, device="cuda")
    out = _prompt(q, k, v, cu2, None, max_q=30)
    assert (out[:20] == 7).all()
    _held(out[20:], ref[20:], mag[20:], "bf16", True)
    cu3 = torch.tensor([-4, 20, 2 ** 30], dtype=torch.int32, device="cuda")
    _held(_prompt(q, k, v, cu3, None, max_q=2 ** 30), ref, mag, "bf16", True)


@pytest.mark.gpu
def test_prompt_scale_and_extreme_scores(gen):
    q, k, v, cu, _, ref, mag = _prompt_case(gen, [90], [90], 2, 1, 128, "bf16", True, scale=0.02)
    _held(_prompt(q, k, v, cu, None, scale=0.02), ref, mag, "bf16", True)
    # every score -inf (finite products that overflow): no weight anywhere, zeros
    big = torch.full_like(q, -3e38)
    out = _prompt(big, torch.full_like(k, 3e38), v, cu, None)
    assert not out.any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_many_sequences(gen, dtype, causal):
    # more than 64 sequences: the workgroups find theirs in another way
    lens = [int(x) for x in torch.randint(0, 90, (67,), generator=gen)]
    lens[0], lens[3], lens[66] = 0, 400, 1
    q, k, v, cu, _, ref, mag = _prompt_case(gen, lens, lens, 4, 2, 64, dtype, causal)
    _held(_prompt(q, k, v, cu, None, max_q=400, causal=causal), ref, mag, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_prompt_row_strides(gen, dim):
    # rows 16 bytes further apart than their heads need, out among them
    n, heads, kvh = 200, 4, 2
    q, k, v, cu, _, ref, mag = _prompt_case(gen, [n], [n], heads, kvh, dim, "bf16", True)

    def wide(t, by):
        w = torch.full((t.shape[0], t.shape[1] * dim + by), math.nan, dtype=t.dtype, device="cuda")
        w[:, :t.shape[1] * dim] = t.flatten(1)
        return w[:, :t.shape[1] * dim].unflatten(1, (t.shape[1], dim))
    q, k, v, out = wide(q, 8), wide(k, 8), wide(v, 24), wide(torch.zeros_like(q), 40)
    _held(glq.attn_prompt(q, k, v, out, cu), ref, mag, "bf16", True)
    assert torch.isnan(out.as_strided((n, 40), (out.stride(0), 1), heads * dim)).all()      # between the rows: as it was


@pytest.mark.gpu
def test_prompt_keys_beyond_32_bits(gen):
    # a sequence whose keys lie past 2^31 elements into k and v
    n, heads, dim, stride = 100, 2, 64, 32768
    rows = 2 ** 31 // stride + 200
    k, v = (torch.empty(rows, stride, dtype=torch.bfloat16, device="cuda")[:, :heads * dim].unflatten(1, (heads, dim))
            for _ in range(2))
    q, kd, vd, _, _, ref, mag = _prompt_case(gen, [n], [n], heads, heads, dim, "bf16", True)
    k[rows - n:], v[rows - n:] = kd, vd
    cu_q = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([rows - n, rows], dtype=torch.int32, device="cuda")
    _held(_prompt(q, k, v, cu_q, cu_k), ref, mag, "bf16", True)
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.gpu
def test_prompt_agrees_with_decode(gen):
    # the last row of a causal prompt is what one new token sees
    n, heads, kvh, dim = 333, 8, 2, 128
    q, k, v, cu, _, ref, mag = _prompt_case(gen, [n], [n], heads, kvh, dim, "f32", True)
    cache = glq.KvCache.empty(12, 32, kvh, dim, glq.KV_INT8)
    table = torch.randperm(12, generator=gen).to(torch.int32)[None].cuda()
    at = torch.arange(n, device="cuda")
    slots = (table[0].long()[at // 32] * 32 + at % 32).to(torch.int32)
    glq.kv_append(cache, k, v, slots)
    k8, v8 = torch.empty_like(k), torch.empty_like(v)
    glq.kv_read(cache, slots, k8, v8)
    out = _prompt(q, k8, v8, cu, None)
    one, _ = _decode(cache, q[n - 1:], table, torch.tensor([n], dtype=torch.int32, device="cuda"), n)
    assert (one[0] - out[n - 1]).abs().max() <= 2e-5 * out[n - 1].abs().max()


# --------------------------------------------------------------- refusals (CPU)

def _cache_struct(**kw):
    c = dict(format=1, kv_heads=2, head_dim=128, page_size=32, num_pages=4, k=256, v=256, k_scale=256, v_scale=256)
    c.update(kw)
    return glq.KvCacheStruct(*[c[f[0]] for f in glq.KvCacheStruct._fields_])


BAD_CACHES = [(dict(format=3), "ARG"), (dict(format=-1), "ARG"), (dict(kv_heads=0), "ARG"), (dict(num_pages=0), "ARG"),
              (dict(page_size=8), "ARG"), (dict(page_size=48), "ARG"), (dict(page_size=2048), "ARG"),
              (dict(k=0), "ARG"), (dict(v=0), "ARG"), (dict(k=264), "ARG"), (dict(k_scale=0), "ARG"),
              (dict(v_scale=260), "ARG"), (dict(head_dim=96), "UNSUPPORTED"), (dict(head_dim=0), "UNSUPPORTED"),
              (dict(num_pages=1 << 40), "UNSUPPORTED"), (dict(kv_heads=1 << 20), "UNSUPPORTED")]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_refusals(bad, status):
    lib, c, want = glq.raw(), _cache_struct(**bad), getattr(glq, "GLQ_ERR_" + status)
    r = ctypes.byref(c)
    assert lib.glq_kv_append(r, 256, 256, 1, 256, 256, 256, 1, None) == want
    assert lib.glq_kv_read(r, 256, 1, 256, 256, 1, 256, 256, None) == want
    assert lib.glq_attn_decode_workspace(r, 1, 2, 10) == 0
    assert lib.glq_attn_decode(r, 256, 1, 256, 1, 2, 256, 1, 256, 10, 0.1, 256, 256, 256, 1 << 20, None) == want


def test_cache_io_refusals():
    lib, c = glq.raw(), _cache_struct()
    good = dict(k=256, v=256, dt=1, ks=256, vs=256, slots=256, tokens=1)
    for bad in (dict(k=0), dict(v=0), dict(k=258), dict(dt=2), dict(dt=-1), dict(ks=255), dict(ks=128), dict(vs=260),
                dict(slots=0), dict(slots=258), dict(tokens=-1)):
        a = dict(good, **bad)
        assert lib.glq_kv_append(ctypes.byref(c), a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["slots"], a["tokens"],
                                 None) == glq.GLQ_ERR_ARG, bad
        assert lib.glq_kv_read(ctypes.byref(c), a["slots"], a["tokens"], a["k"], a["v"], a["dt"], a["ks"], a["vs"],
                               None) == glq.GLQ_ERR_ARG, bad
    assert lib.glq_kv_append(None, 256, 256, 1, 256, 256, 256, 1, None) == glq.GLQ_ERR_ARG
    assert lib.glq_kv_append(ctypes.byref(c), 0, 0, 1, 0, 0, 0, 0, None) == glq.GLQ_OK
    assert lib.glq_kv_append(ctypes.byref(c), 256, 256, 1, 256, 256, 256, 1 << 40, None) == glq.GLQ_ERR_UNSUPPORTED


def test_decode_refusals():
    lib, c = glq.raw(), _cache_struct()

    def call(**kw):
        a = dict(q=256, dt=1, qs=512, batch=2, heads=4, table=256, pages=3, lens=256, most=96, scale=0.1, out=256,
                 os=512, ws=256, bytes=1 << 30)
        a.update(kw)
        return lib.glq_attn_decode(ctypes.byref(c), a["q"], a["dt"], a["qs"], a["batch"], a["heads"], a["table"],
                                   a["pages"], a["lens"], a["most"], a["scale"], a["out"], a["os"], a["ws"],
                                   a["bytes"], None)
    for bad in (dict(q=0), dict(q=264), dict(dt=5), dict(qs=511), dict(qs=500), dict(batch=-1), dict(heads=0),
                dict(heads=3), dict(table=0), dict(table=258), dict(pages=-1), dict(pages=2), dict(lens=0),
                dict(lens=257), dict(most=-1), dict(most=97), dict(scale=math.nan), dict(scale=math.inf), dict(out=0),
                dict(out=260), dict(os=508)):
        assert call(**bad) == glq.GLQ_ERR_ARG, bad
    for bad in (dict(ws=0), dict(ws=128), dict(bytes=100)):
        assert call(**bad) == glq.GLQ_ERR_WORKSPACE, bad
    assert call(most=2 ** 31 - 1, pages=1 << 40) == glq.GLQ_ERR_UNSUPPORTED
    assert call(batch=1 << 40) == glq.GLQ_ERR_UNSUPPORTED
    assert call(batch=0, q=0, out=0) == glq.GLQ_OK
    assert lib.glq_attn_decode_workspace(ctypes.byref(c), 2, 3, 10) == 0
    assert lib.glq_attn_decode_workspace(ctypes.byref(c), 2, 4, 10) >= 65536


def test_prompt_refusals():
    lib = glq.raw()

    def call(flags=1, **kw):
        a = dict(q=256, k=256, v=256, out=256, dt=1, q_heads=4, kv_heads=2, head_dim=64, q_stride=256, k_stride=128,
                 v_stride=128, out_stride=256, total_q=5, total_k=5, batch=1, cu_q=256, cu_k=256, max_q=5, scale=0.1)
        a.update(kw)
        return lib.glq_attn_prompt(ctypes.byref(glq.PromptStruct(*[a[f[0]] for f in glq.PromptStruct._fields_])),
                                   flags, None)
    for bad in (dict(q=0), dict(k=8), dict(v=0), dict(out=0), dict(dt=2), dict(q_heads=0), dict(q_heads=5),
                dict(kv_heads=0), dict(q_stride=255), dict(k_stride=130), dict(v_stride=64), dict(out_stride=0),
                dict(total_q=-1), dict(total_k=-1), dict(batch=-1), dict(max_q=-1), dict(cu_q=0), dict(cu_k=2),
                dict(scale=math.inf), dict(flags=2)):
        assert call(**bad) == glq.GLQ_ERR_ARG, bad
    for bad in (dict(head_dim=80, q_stride=320, k_stride=160, v_stride=160, out_stride=320),
                dict(total_q=1 << 33), dict(total_k=1 << 33), dict(batch=1 << 40), dict(k_stride=1 << 23)):
        assert call(**bad) == glq.GLQ_ERR_UNSUPPORTED, bad
    assert lib.glq_attn_prompt(None, 0, None) == glq.GLQ_ERR_ARG
    for nothing in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert call(**nothing, q=0, cu_q=0) == glq.GLQ_OK


def test_binding_refuses_host_tensors():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 2], dtype=torch.int32)
    with pytest.raises(ValueError):
        glq.attn_prompt(q, q, q, q.clone(), cu)
    with pytest.raises(ValueError):
        glq.KvCache.empty(2, 16, 1, 64, glq.KV_BF16, device="cpu")
    with pytest.raises(ValueError):
        glq.KvCache.empty(2, 16, 1, 64, 9, device="cpu")


@pytest.mark.gpu
def test_binding_refusals(gen):
    cache, q, table, ln, _, _ = _decode_case(gen, "int8", [20, 3], 4, 2, 64, 16, "bf16")
    ws = torch.zeros(glq.attn_decode_workspace_bytes(cache, 2, 4, 20), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    good = dict(q=q, page_table=table, lens=ln, out=out, workspace=ws, max_len=20)
    glq.attn_decode(cache, **good)
    for bad in (dict(q=q.cpu()), dict(q=q[:, :3].transpose(0, 1)), dict(q=q.half()), dict(lens=ln.long()),
                dict(lens=ln[:1]), dict(page_table=table.long()), dict(out=out.float()), dict(out=out[:1]),
                dict(page_table=table.T), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            glq.attn_decode(cache, **dict(good, **bad))
    for bad in (dict(q=q[:, :3], out=out[:, :3].contiguous()), dict(max_len=2 ** 20)):
        with pytest.raises(glq.GlqError):
            glq.attn_decode(cache, **dict(good, **bad))
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(5, dtype=torch.int32, device="cuda")
    glq.kv_append(cache, k, k, slots)
    for bad in ((k[:, :1], k, slots), (k, k.float(), slots), (k, k[:4], slots), (k, k, slots.long()),
                (k, k, slots[:4]), (k.cpu(), k, slots)):
        with pytest.raises(ValueError):
            glq.kv_append(cache, *bad)
    with pytest.raises(ValueError):
        glq.KvCache(cache.k, cache.v)                # scales missing
    with pytest.raises(ValueError):
        glq.KvCache(cache.k, cache.v[:1], cache.k_scale, cache.v_scale)
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        glq.attn_prompt(k, k, k, k.clone(), cu.long())
    with pytest.raises(ValueError):
        glq.attn_prompt(torch.cat((k, k[:, :1]), 1), k, k, torch.cat((k, k[:, :1]), 1), cu)


# ------------------------------------------------------------------- all together

@pytest.mark.gpu
@pytest.mark.parametrize("cache,most", [("bf16", 0.02), ("int8", 0.025), ("int4", 0.2)])
def test_attention_block_example(cache, most):
    # the example: compressed projections, rotated keys in the cache, a prompt in
    # two chunks, then tokens. bf16: a few roundings of 2^-8 of projections, weights
    # and sums; 8 bits: steps of max / 127 of about 2.5 sigma, 0.006 sigma rms, in
    # keys and values; 4 bits: 0.1 sigma rms in each
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for err in mod.run(cache=cache, tokens=4):
        assert err <= most


# ------------------------------------------------------ sums beyond one lane's keys

def _leading_key(n, dim, at, later, gen):
    """Keys and values of one kept head and two queries of opposite tastes: at scale 1
    query 0 has score 160 on key `at` and 0 elsewhere (230 in base 2: every other
    weight is 0 in float32), query 1 has 32 on the keys `later` and 0 elsewhere, so
    its maximum rises where those begin and the sums of both are rescaled there."""
    k = _normal(gen, n, 1, dim, dtype=torch.bfloat16).float()
    v = _normal(gen, n, 1, dim, dtype=torch.bfloat16)
    k[:, 0, :2] = 0
    k[at, 0, 0] = 10
    k[later, 0, 1] = 2
    q = torch.zeros(2, dim)
    q[0, 0], q[1, 1] = 16, 16
    return q, k, v.float()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_decode_leading_token_before_a_rise(gen, fmt, dim, dtype):
    # the leading token in each quarter of a wave's tokens and in both halves of its
    # tile: lanes that hold only weights of 0 hold other tokens' values all the same
    n, page = 300, 32
    for at in (1, 6, 9, 14, 19, 30):
        q, k, v = _leading_key(n, dim, at, [128, 135, 140, 151, 258], gen)
        k, v, q = k.cuda(), v.cuda(), q.to(DTYPES[dtype]).cuda()[None]
        cache = glq.KvCache.empty(10, page, 1, dim, FORMATS[fmt])
        glq.kv_append(cache, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
        table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
        out, _ = _decode(cache, q, table, torch.tensor([n], dtype=torch.int32, device="cuda"), n, scale=1.0)
        kk, vv = (_ref_values(x.cpu(), fmt)[:, 0] for x in (k, v))
        ref, mag = _ref_attend(q[0].cpu(), kk, vv, 1.0, torch.ones(2, n, dtype=torch.bool))
        assert (ref[0] - vv[at].double()).abs().max() < 1e-60
        _held(out[0], ref, mag, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [128, 600])
def test_prompt_leading_key_before_a_rise(gen, dtype, dim, causal, n):
    # 128 keys: two tiles that the waves share; 600: a wave's own tiles
    for at in (1, 6, 34, 61):
        q, k, v = _leading_key(n, dim, at, list(range(70, n - 1, 64)), gen)
        # the queries as two tokens of one head, and as two heads of each of two tokens
        for heads in (1, 2):
            qq = q[:, None] if heads == 1 else q[None].repeat(2, 1, 1)
            qq, kk, vv = (x.to(DTYPES[dtype]).cuda() for x in (qq, k, v))
            cu = [torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (2, n)]
            out = _prompt(qq, kk, vv, *cu, causal=causal, scale=1.0)
            seen = torch.ones(2, n, dtype=torch.bool)
            if causal:
                seen[0, n - 1] = False
            for h in range(heads):
                ref, mag = _ref_attend(qq[:, h].cpu(), kk[:, 0].cpu(), vv[:, 0].cpu(), 1.0, seen)
                _held(out[:, h], ref, mag, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_decode_sees_values_that_are_not_finite(gen, fmt, dtype, dim, which, bad):
    # a token's head that holds an infinity or a NaN reads back as NaN: so does what sees it,
    # and no other kept head does. Queries of very different sizes: their sums are rounded
    n, heads, kvh = 40, 16, 2
    x = {"k": _normal(gen, n, kvh, dim), "v": _normal(gen, n, kvh, dim)}
    x[which][17, 1, 3] = bad
    cache = glq.KvCache.empty(3, 16, kvh, dim, FORMATS[fmt])
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    glq.kv_append(cache, x["k"].cuda(), x["v"].cuda(), slots)
    q = (_normal(gen, 8, heads, dim) * torch.exp(2 * _normal(gen, 8, heads, dim))).to(DTYPES[dtype]).cuda()
    table = torch.arange(3, dtype=torch.int32, device="cuda")[None].repeat(8, 1)
    out, _ = _decode(cache, q, table, torch.full((8,), n, dtype=torch.int32, device="cuda"), n)
    assert torch.isnan(out[:, heads // 2:]).all()
    assert torch.isfinite(out[:, :heads // 2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("bf16", "f32"), ("int8", "bf16"), ("int8", "f32"),
                                       ("int4", "bf16"), ("int4", "f32")])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens", [[300, 7], [4000, 2500]])
def test_decode_values_near_the_largest(gen, fmt, dtype, dim, lens):
    # finite values of up to 3e38 (the largest bf16 is 3.39e38): their weighted mean is
    # finite, whatever the number of tokens
    heads, page = 2, 32
    pages = [-(-n // page) for n in lens]
    table = torch.zeros(2, max(pages), dtype=torch.int32)
    table[0, :pages[0]] = torch.arange(pages[0])
    table[1, :pages[1]] = pages[0] + torch.arange(pages[1])
    cache = glq.KvCache.empty(sum(pages), page, 1, dim, FORMATS[fmt])
    q = _normal(gen, 2, heads, dim, dtype=DTYPES[dtype]) * 1.5
    out = None
    kv = []
    for b, n in enumerate(lens):
        k = _normal(gen, n, 1, dim, dtype=torch.bfloat16)
        v = (torch.rand(n, 1, dim, generator=gen) * 1e38 + 2e38).to(torch.bfloat16)
        v[..., ::2] *= -1
        slots = table[b].long()[torch.arange(n) // page] * page + torch.arange(n) % page
        glq.kv_append(cache, k.cuda(), v.cuda(), slots.to(torch.int32).cuda())
        kv.append((k, v))
    out, _ = _decode(cache, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens))
    for b, (k, v) in enumerate(kv):
        kk, vv = (_ref_values(x.float(), fmt)[:, 0] for x in (k, v))
        ref, mag = _ref_attend(q[b], kk, vv, dim ** -0.5, torch.ones(heads, lens[b], dtype=torch.bool))
        _held(out[b], ref, mag, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens_q,lens_k", [([150, 90], [150, 90]), ([9, 3], [700, 1500]), ([600, 513, 700], [600, 513, 700])])
def test_prompt_values_near_the_largest(gen, dtype, dim, lens_q, lens_k):
    # shared tiles, few rows on many keys, launches that fill the card
    heads, kvh = (24, 3) if sum(lens_q) > 1000 else (4, 2)
    tq, tk = sum(lens_q), sum(lens_k)
    q = (_normal(gen, tq, heads, dim) * 1.5).to(DTYPES[dtype])
    k = _normal(gen, tk, kvh, dim).to(DTYPES[dtype])
    v = (torch.rand(tk, kvh, dim, generator=gen) * 1e38 + 2e38).to(DTYPES[dtype])
    v[..., ::2] *= -1
    cu_q, cu_k = (torch.tensor(np.concatenate(([0], np.cumsum(x))), dtype=torch.int32) for x in (lens_q, lens_k))
    for causal in (True, False):
        out = _prompt(q.cuda(), k.cuda(), v.cuda(), cu_q.cuda(), cu_k.cuda(), max_q=max(lens_q), causal=causal)
        for b, (n, m) in enumerate(zip(lens_q, lens_k)):
            a, c = slice(cu_q[b], cu_q[b + 1]), slice(cu_k[b], cu_k[b + 1])
            seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n if causal else m)
            for h in range(0, heads, 3):
                g = h // (heads // kvh)
                ref, mag = _ref_attend(q[a, h], k[c, g], v[c, g], dim ** -0.5, seen)
                _held(out[a, h], ref, mag, dtype, True)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prompt_very_many_sequences(gen, dtype):
    # as many sequences as tokens allow, and no bound given on their lengths: the size of the launch
    # comes from the totals
    batch, heads, kvh, dim = 20000, 32, 8, 64
    lens = torch.randint(0, 9, (batch,), generator=gen)
    cu = torch.cat((torch.zeros(1, dtype=torch.long), lens.cumsum(0))).to(torch.int32)
    total = int(cu[-1])
    q = _normal(gen, total, heads, dim, dtype=DTYPES[dtype])
    k, v = (_normal(gen, total, kvh, dim, dtype=DTYPES[dtype]) for _ in range(2))
    out = _prompt(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), None)
    assert not (out == 7).all(-1).any()              # every row is written
    for b in list(range(0, batch, 1111)) + [batch - 1]:
        n, a = int(lens[b]), slice(cu[b], cu[b + 1])
        seen = torch.ones(n, n, dtype=torch.bool).tril()
        for h in (0, 13, 31):
            ref, mag = _ref_attend(q[a, h], k[a, h // 4], v[a, h // 4], dim ** -0.5, seen)
            _held(out[a, h], ref, mag, dtype, True)


def test_launches_past_the_grid_are_refused():
    # threads of a launch are counted in 32 bits: 2^24 - 1 workgroups of 256
    lib = glq.raw()
    c = ctypes.byref(_cache_struct())
    for batch, heads in ((2 ** 23, 4), (2 ** 22, 36)):
        assert lib.glq_attn_decode_workspace(c, batch, heads, 10) == 0
        assert lib.glq_attn_decode(c, 256, 1, 128 * heads, batch, heads, 256, 1, 256, 10, 0.1, 256, 128 * heads, 256,
                                   1 << 40, None) == glq.GLQ_ERR_UNSUPPORTED
    assert lib.glq_attn_decode_workspace(c, 2 ** 23 - 1, 4, 10) >= 65536
    p = dict(q=256, k=256, v=256, out=256, dt=1, q_heads=4, kv_heads=2, head_dim=64, q_stride=256, k_stride=128,
             v_stride=128, out_stride=256, total_q=2 ** 24, total_k=2 ** 24, batch=2 ** 24, cu_q=256, cu_k=256, max_q=1,
             scale=0.1)
    for bad in (dict(), dict(dt=0), dict(batch=2 ** 31 - 1), dict(batch=2 ** 62), dict(total_q=2 ** 31 - 1, max_q=2 ** 31)):
        a = dict(p, **bad)
        assert lib.glq_attn_prompt(ctypes.byref(glq.PromptStruct(*[a[f[0]] for f in glq.PromptStruct._fields_])), 1,
                                   None) == glq.GLQ_ERR_UNSUPPORTED, bad


@pytest.mark.parametrize("kv_heads,q_heads", [(1, 1), (8, 32), (40, 40), (2, 300), (7, 7), (512, 512), (20000, 20000)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_decode_workspace_grows_with_the_batch(kv_heads, q_heads, dim):
    # one workspace for the largest batch and length serves every smaller one
    lib, c = glq.raw(), _cache_struct(kv_heads=kv_heads, head_dim=dim)

    def need(batch, most):
        return lib.glq_attn_decode_workspace(ctypes.byref(c), batch, q_heads, most)
    edge = 16384 // kv_heads
    for most in (100, 129, 5000, 200000):
        sizes = [need(b, most) for b in sorted({1, 2, 63, 64, 65, 100, 300, 2000, 4096, 9000, *range(max(1, edge - 500), edge + 3, 7)})]
        sizes = sizes[:sizes.index(0)] if 0 in sizes else sizes     # (0: past what a launch holds)
        assert sizes == sorted(sizes) and sizes[0] >= 65536
    for b in (1, 64, 65, 300, 3000):
        sizes = [need(b, most) for most in (0, 1, 128, 129, 256, 257, 4000, 10 ** 6)]
        assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_decode_workspace_of_a_larger_batch(gen, dtype):
    # sized for a batch that is not split any more, used for one that is
    cache, q, table, ln, ref, mag = _decode_case(gen, "int8", [3000, 700], 4, 2, 128, 32, dtype)
    ws = torch.zeros(glq.attn_decode_workspace_bytes(cache, 9000, 4, 3000), dtype=torch.uint8, device="cuda")
    out, _ = _decode(cache, q, table, ln, 3000, ws)
    _held(out, ref, mag, dtype)


@pytest.mark.gpu
def test_attention_refuses_another_device(gen, monkeypatch):
    # a launch goes to the current device: tensors or a stream of another one are refused
    cache, q, table, ln, _, _ = _decode_case(gen, "int8", [20, 3], 4, 2, 64, 16, "bf16")
    ws = torch.zeros(glq.attn_decode_workspace_bytes(cache, 2, 4, 20), dtype=torch.uint8, device="cuda")
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(5, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    calls = (lambda **s: glq.kv_append(cache, k, k, slots, **s),
             lambda **s: glq.kv_read(cache, slots, k.clone(), k.clone(), **s),
             lambda **s: glq.attn_decode(cache, q, table, ln, torch.empty_like(q), ws, 20, **s),
             lambda **s: glq.attn_prompt(k, k, k, k.clone(), cu, **s))

    class Elsewhere:
        device = torch.device("cuda", 1)
        cuda_stream = 0
    for call in calls:
        call()
        call(stream=torch.cuda.Stream())
        with pytest.raises(ValueError, match="stream"):
            call(stream=Elsewhere())
    torch.cuda.synchronize()
    monkeypatch.setattr(glq, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["int8", "int4"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("size", [1.0, 1e-25, 1e30])
def test_append_float32_mantissas(gen, fmt, dim, size):
    # float32 inputs with all their bits: the product x Q and the quotient by a are
    # each rounded to float32, the code is that rounded half to even
    tokens, heads, q = 600, 3, np.float32(LEVELS[fmt])
    x = _normal(gen, tokens, heads, dim).numpy() * np.float32(size)
    # quotients next to the halves, where one rounding more or less shows
    a = np.abs(x).max(-1, keepdims=True)
    half = np.float32(0.5) + np.arange(dim, dtype=np.float32) % np.float32(LEVELS[fmt] - 1)
    near = (half * a / q).astype(np.float32)
    for token in range(0, tokens, 2):
        step = token // 2 % 7 - 3
        x[token] = near[token]
        for _ in range(abs(step)):
            x[token] = np.nextafter(x[token], np.float32(np.inf if step > 0 else 0))
        x[token, :, -1] = a[token, :, 0]
    a = np.abs(x).max(-1, keepdims=True)
    want = np.rint((x * q).astype(np.float32) / a)
    assert (x * q).dtype == np.float32 and want.dtype == np.float32
    cache = glq.KvCache.empty(-(-tokens // 64), 64, heads, dim, FORMATS[fmt])
    t = torch.from_numpy(x).cuda()
    glq.kv_append(cache, t, -t, torch.arange(tokens, dtype=torch.int32, device="cuda"))
    at = torch.arange(tokens)
    for codes, scale, sign in zip(_unpack(cache), (cache.k_scale, cache.v_scale), (1, -1)):
        assert torch.equal(codes[at // 64, :, at % 64], sign * torch.from_numpy(want).double())
        assert torch.equal(scale.cpu()[at // 64, :, at % 64], torch.from_numpy((a / q)[..., 0]))


def test_scale_refusals():
    # a scale that is finite, but not once the kernels' exponentials of base 2 are paid for: products
    # of 0 would give NaN
    lib, c = glq.raw(), _cache_struct()
    for scale in (2.4e38, -2.4e38, 3.4e38):
        assert lib.glq_attn_decode(ctypes.byref(c), 256, 1, 512, 2, 4, 256, 3, 256, 96, scale, 256, 512, 256, 1 << 30,
                                   None) == glq.GLQ_ERR_ARG
        st = glq.PromptStruct(256, 256, 256, 256, 1, 4, 2, 64, 256, 128, 128, 256, 5, 5, 1, 256, 256, 5, scale)
        assert lib.glq_attn_prompt(ctypes.byref(st), 1, None) == glq.GLQ_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 1e30])
def test_signs_and_sizes_of_the_scale(gen, dtype, scale):
    # queries made to fit the scale's size: scores of about 0.3 |q.k|
    n, dim = 70, 64
    size = 0.3 / abs(scale) if abs(scale) in (1e-30, 1e30) else 1.0
    q = (_normal(gen, 5, 4, dim) * size).to(DTYPES[dtype])
    k, v = (_normal(gen, n, 2, dim, dtype=torch.bfloat16).to(DTYPES[dtype]) for _ in range(2))
    cu = [torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (5, n)]
    out = _prompt(q.cuda(), k.cuda(), v.cuda(), *cu, causal=False, scale=scale)
    cache = glq.KvCache.empty(5, 16, 2, dim, glq.KV_BF16)
    glq.kv_append(cache, k.cuda(), v.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    table = torch.arange(5, dtype=torch.int32, device="cuda")[None].repeat(5, 1)
    one, _ = _decode(cache, q.cuda(), table, torch.full((5,), n, dtype=torch.int32, device="cuda"), n, scale=scale)
    for h in range(4):
        ref, mag = _ref_attend(q[:, h], k[:, h // 2], v[:, h // 2], float(np.float32(scale)),
                               torch.ones(5, n, dtype=torch.bool))
        _held(out[:, h], ref, mag, dtype, True)
        _held(one[:, h], ref, mag, dtype)


@pytest.mark.gpu
def test_binding_refuses_what_is_no_tensor(gen):
    cache, q, table, ln, _, _ = _decode_case(gen, "int8", [20, 3], 4, 2, 64, 16, "bf16")
    ws = torch.zeros(glq.attn_decode_workspace_bytes(cache, 2, 4, 20), dtype=torch.uint8, device="cuda")
    good = dict(q=q, page_table=table, lens=ln, out=torch.empty_like(q), workspace=ws, max_len=20)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    for bad in (None, [[0, 1]], 7, torch.tensor(3, dtype=torch.int32, device="cuda")):
        for name in ("q", "page_table", "lens", "out"):
            with pytest.raises(ValueError):
                glq.attn_decode(cache, **dict(good, **{name: bad}))
        with pytest.raises(ValueError):
            glq.attn_prompt(k, k, k, k.clone(), bad)
        with pytest.raises(ValueError):
            glq.kv_append(cache, k, k, bad)
        if bad is not None:
            with pytest.raises(ValueError):
                glq.attn_prompt(k, k, k, k.clone(), cu, bad)
    for bad in (None, 7, ws.cpu(), ws[::2]):
        with pytest.raises(ValueError):
            glq.attn_decode(cache, **dict(good, workspace=bad))
    with pytest.raises(glq.GlqError):
        glq.attn_prompt(k, k, k, k.clone(), cu[:0])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prompt_chunks_over_a_cached_prefix(gen, fmt, dtype):
    # a prompt in chunks: each chunk's keys are appended, everything cached is read back
    # through shuffled pages and seen by the chunk's queries; float32 inputs with all their bits
    heads, kvh, dim, page, total = 6, 2, 128, 32, 330
    cache = glq.KvCache.empty(14, page, kvh, dim, FORMATS[fmt])
    table = torch.randperm(14, generator=gen)[:-(-total // page)]
    at = torch.arange(total)
    slots = (table[at // page] * page + at % page).to(torch.int32).cuda()
    q = (_normal(gen, total, heads, dim) * 1.5).to(DTYPES[dtype])
    k, v = (_normal(gen, total, kvh, dim).to(DTYPES[dtype]) for _ in range(2))
    kk, vv = k, v
    if fmt == "bf16":
        kk, vv = (x.to(torch.bfloat16).float() for x in (k, v))
    else:
        def held(x):
            x = x.float().numpy()
            a, levels = np.abs(x).max(-1, keepdims=True), np.float32(LEVELS[fmt])
            return torch.from_numpy(np.rint(x * levels / a) * (a / levels))
        kk, vv = held(k), held(v)
    kk, vv = kk.to(DTYPES[dtype]), vv.to(DTYPES[dtype])
    first = 0
    for n in (130, 1, 70, 2, 127):
        end = first + n
        glq.kv_append(cache, k[first:end].cuda(), v[first:end].cuda(), slots[first:end])
        ko, vo = (torch.empty(end, kvh, dim, dtype=DTYPES[dtype], device="cuda") for _ in range(2))
        glq.kv_read(cache, slots[:end], ko, vo)
        assert torch.equal(ko.cpu(), kk[:end]) and torch.equal(vo.cpu(), vv[:end])
        cu = [torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (n, end)]
        out = _prompt(q[first:end].cuda(), ko, vo, *cu, max_q=n)
        seen = torch.arange(end)[None] <= torch.arange(n)[:, None] + first
        for h in range(heads):
            ref, mag = _ref_attend(q[first:end, h], kk[:end, h // 3], vv[:end, h // 3], dim ** -0.5, seen)
            _held(out[:, h], ref, mag, dtype, True)
        first = end
    assert first == total


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,lens_q,lens_k,heads", [("bf16", [30, 4], [700, 400], 4), ("bf16", [100, 28], [100, 28], 4),
                                                       ("f32", [50, 20], [80, 20], 4), ("f32", [600, 500], [600, 500], 64)])
def test_prompt_and_cache_in_a_graph(gen, dtype, lens_q, lens_k, heads):
    # a captured chunk: write, read back and attention, replayed with other inputs in the same tensors
    # and eager work between, against the eager calls; on a stream that is not the tensors' own
    kvh, dim, page = 2, 64, 16
    q, k, v, cu_q, cu_k, _, _ = _prompt_case(gen, lens_q, lens_k, heads, kvh, dim, dtype, True)
    n = k.shape[0]
    cache = glq.KvCache.empty(-(-n // page), page, kvh, dim, glq.KV_INT8)
    slots = _slots(gen, n, -(-n // page) * page).cuda()
    ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q)

    def step():
        glq.kv_append(cache, k, v, slots)
        glq.kv_read(cache, slots, ko, vo)
        glq.attn_prompt(q, ko, vo, out, cu_q, cu_k, max_q=max(lens_q))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        k.copy_((k.float() * 0.9 + 0.1).to(k.dtype))
        q.copy_(q.flip(0))
        out.zero_(), ko.zero_(), vo.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, ko, vo)]
        out.zero_(), ko.zero_(), vo.zero_()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, ko, vo))) and out.any()
