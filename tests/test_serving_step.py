"""The calls of a serving step run together, as a program would: plan, norms and rotation into
the cache, attention, routing and the experts, eager and in graphs, on other streams, in workspaces that
serve several calls, and at sizes where offsets leave 32 bits.

Each link is held to the plain formula on what the link before it gave, with the tolerances of the tests of the
single calls; graphs, streams and shared workspaces are held to the same bits as plain calls.
"""
import ctypes

import numpy as np
import pytest
import torch

from test_attention import _held as held_attention
from test_attention import _ref_attend, _ref_values
from test_experts import DTYPES, Set, _held, _rows_reference, _tolerance
from test_step import _check_route, _held_turn, _plan_reference, _turn_reference

glq = pytest.importorskip("dequant_e8_codebook_amd.glq")

FORMATS = {"bf16": glq.KV_BF16, "int8": glq.KV_INT8, "int4": glq.KV_INT4}


@pytest.fixture
def gen():
    return torch.Generator().manual_seed(17)


@pytest.fixture(scope="module")
def cb():
    return glq.device_codebook()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Server:
    """A layer's state and buffers for up to `most` new tokens of `batch` requests."""

    def __init__(self, cb, fmt="int8", batch=5, most=96, page=16, max_pages=8, dtype="bf16", heads=6, kv_heads=2, dim=64,
                 hidden=256, inner=512, experts=6, top=2, max_read=0, seed=3):
        gen = torch.Generator().manual_seed(seed)
        dt = self.dt = DTYPES[dtype]
        self.heads, self.kv_heads, self.dim, self.top, self.page, self.max_len = heads, kv_heads, dim, top, page, page * max_pages
        self.most, self.count, self.pages = most, experts, batch * max_pages + 2
        self.free = torch.randperm(self.pages, generator=gen).to(torch.int32)       # on the host, as a server keeps it
        self.free_dev = self.free.cuda()
        self.plan = glq.KvPlan(torch.full((batch, max_pages), -1, dtype=torch.int32, device="cuda"), page, self.pages, most,
                               max_read)
        self.cache = glq.KvCache.empty(self.pages, page, kv_heads, dim, FORMATS[fmt])
        self.table = glq.rotary_table(self.max_len, dim)
        self.wq, self.wk = (torch.rand(dim, generator=gen).cuda() + 0.5 for _ in range(2))
        self.lens, self.added = _ints([0] * batch), _ints([0] * batch)
        self.qkv = torch.zeros(most, heads + 2 * kv_heads, dim, dtype=dt, device="cuda")
        self.out = torch.zeros(most, heads, dim, dtype=dt, device="cuda")
        self.attn_ws = torch.zeros(glq.attn_decode_workspace_bytes(self.cache, batch, heads, self.max_len), dtype=torch.uint8,
                                   device="cuda")
        self.x, self.y = (torch.zeros(most, hidden, dtype=dt, device="cuda") for _ in range(2))
        self.inside = torch.zeros(most * top, inner, dtype=dt, device="cuda")
        self.logits = torch.full((most, experts), -torch.inf, device="cuda")
        self.weights = torch.zeros(most, top, device="cuda")
        self.ids, self.pos = (torch.zeros(most, top, dtype=torch.int32, device="cuda") for _ in range(2))
        self.src, self.offsets = _ints([0] * (most * top)), _ints([0] * (experts + 1))
        self.sets = Set(experts, inner, hidden, 4, seed=seed), Set(experts, hidden, inner, 3, seed=seed + 1, row_scale=True)
        self.up, self.down = (s.device(cb) for s in self.sets)
        self.route_ws = torch.empty(glq.route_workspace_bytes(most, experts, top), dtype=torch.uint8, device="cuda")
        self.expert_ws = torch.empty(max(glq.expert_linear_workspace_bytes(e, most * top) for e in (self.up, self.down)),
                                     dtype=torch.uint8, device="cuda")

    def inputs(self, gen, added):
        """The step's inputs; rows behind the last token stay a padded batch's, with no experts."""
        n = sum(added)
        self.added.copy_(_ints(added))
        self.qkv.zero_()
        self.qkv[:n] = torch.randn(n, *self.qkv.shape[1:], generator=gen).to(self.dt).cuda()
        self.x.copy_(torch.randn(self.x.shape, generator=gen).to(self.dt))
        self.logits.fill_(-torch.inf)
        self.logits[:n] = torch.randn(n, self.count, generator=gen).cuda()
        return n

    def projected(self):
        kv = self.kv_heads
        return self.qkv.split((self.heads, kv, kv), 1)

    def step(self, stream=None):
        """What a graph would hold, for one new token a request or for none (a row of the padded batch)."""
        plan, (q, k, v) = self.plan, self.projected()
        glq.kv_plan(plan, self.lens, self.added, self.free_dev, stream=stream)
        glq.qk_norm_rope(q, k, plan.positions, self.table, q, k, self.wq, self.wk, cache=self.cache, v=v, slots=plan.slots,
                         stream=stream)
        b = plan.batch
        glq.attn_decode(self.cache, q[:b], plan.page_table, plan.new_lens, self.out[:b], self.attn_ws, self.max_len, stream=stream)
        self.feed_forward(stream)

    def feed_forward(self, stream=None):
        glq.route(self.logits, self.top, self.weights, self.ids, self.pos, self.src, self.offsets, self.route_ws, stream=stream)
        glq.expert_linear(self.up, self.x, self.inside, self.offsets, self.expert_ws, src=self.src, stream=stream)
        glq.expert_linear(self.down, self.inside, self.y, self.offsets, self.expert_ws, pos=self.pos, weights=self.weights,
                          stream=stream)

    def after(self):
        """The host's part between steps."""
        used = int(self.plan.used)
        self.free = torch.cat((self.free[used:], self.free[:used] * 0 - 1))
        self.free_dev.copy_(self.free)
        self.lens.copy_(self.plan.new_lens)
        return used

    def results(self):
        p, c = self.plan, self.cache
        return [t.clone() for t in (p.page_table, p.new_lens, p.cu_q, p.slots, p.positions, p.used, self.qkv, c.k, c.v, self.out,
                                    self.weights, self.ids, self.pos, self.src, self.offsets, self.y)]

    def check_feed_forward(self, n, dtype):
        _check_route(self.logits.cpu(), self.top, True, [t.cpu() for t in (self.weights, self.ids, self.pos, self.src, self.offsets)])
        offsets, src = self.offsets.cpu().numpy(), self.src.cpu().numpy()
        rows = int(offsets[-1])
        assert rows == n * self.top
        x = self.x.double().cpu().numpy()
        ref = _rows_reference(self.sets[0], x, offsets, src, len(src))[:rows]
        _held(self.inside[:rows], ref, _tolerance(ref, dtype, x.shape[1]), dtype)
        inside, ids, pos = self.inside.double().cpu().numpy(), self.ids.cpu().numpy(), self.pos.cpu().numpy()
        w, each = self.weights.double().cpu().numpy(), np.zeros((self.most, self.top, x.shape[1]))
        for e in range(self.count):
            t, j = np.nonzero(ids == e)
            if len(t):
                each[t, j] = self.sets[1].reference(e, inside[pos[t, j]])
        _held(self.y, (each * w[..., None]).sum(1), _tolerance(each, dtype, inside.shape[1], w), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prompts_then_tokens(cb, gen, fmt, dtype):
    """Ragged chunks of prompts, read back and attended, then single tokens: every call's output by its formula."""
    s = Server(cb, fmt, dtype=dtype, max_read=700)
    batch, plan, lens, free = 5, s.plan, [0] * 5, s.free.tolist()
    table = plan.page_table.cpu().tolist()
    first = {b: [] for b in range(batch)}                       # keys and values of every request as the cache has them
    for added in [[17, 0, 16, 1, 40], [3, 30, 0, 15, 1], [1, 1, 1, 1, 1], [1, 1, 0, 1, 1], [0, 1, 1, 1, 1]]:
        n = s.inputs(gen, added)
        before = s.qkv.clone()
        decode = added == [1] * 5
        q, k, v = s.projected()
        glq.kv_plan(plan, s.lens, s.added, s.free_dev)
        want, table = _plan_reference(lens, added, table, free, s.page, s.pages, s.most, 700)
        for name, value in want.items():
            assert getattr(plan, name).cpu().tolist() == value, name
        glq.qk_norm_rope(q, k, plan.positions, s.table, q, k, s.wq, s.wk, cache=s.cache, v=v, slots=plan.slots)
        at = plan.positions[:n].long().cpu()
        half = s.dim // 2
        cos, sin = s.table.cpu()[at, :half], s.table.cpu()[at, half:]
        for x, y, w in ((before[:n, :s.heads], q, s.wq), (before[:n, s.heads:s.heads + s.kv_heads], k, s.wk)):
            ref, mag = _turn_reference(x.double().cpu(), w.cpu(), 1e-6, cos, sin, False)
            _held_turn(y[:n], ref, mag, dtype)
        kk, vv = torch.zeros(700, s.kv_heads, s.dim, dtype=s.dt, device="cuda"), torch.zeros(700, s.kv_heads, s.dim, dtype=s.dt,
                                                                                         device="cuda")
        glq.kv_read(s.cache, plan.read_slots, kk, vv)
        i, cu_k = 0, plan.cu_k.cpu().tolist()
        for b in range(batch):
            first[b] += [(k[j].cpu(), v[j].cpu()) for j in range(i, i + added[b])]
            i += added[b]
            for t, (key, value) in enumerate(first[b]):
                for got, x in ((kk, key), (vv, value)):
                    assert torch.equal(got[cu_k[b] + t].cpu(), _ref_values(x.float(), fmt).to(s.dt))
        cu_q = plan.cu_q.cpu().tolist()
        if decode:
            glq.attn_decode(s.cache, q[:batch], plan.page_table, plan.new_lens, s.out[:batch], s.attn_ws, s.max_len)
        else:
            glq.attn_prompt(q[:n], kk, vv, s.out[:n], plan.cu_q, plan.cu_k, max_q=max(added))
        for b in range(batch):
            m, total = added[b], len(first[b])
            seen = torch.ones(m, total, dtype=torch.bool).tril(total - m)
            for h in range(s.heads if m else 0):
                g = h * s.kv_heads // s.heads
                old = slice(cu_k[b], cu_k[b] + total)
                keys, values = ((_ref_values(torch.stack([x[i][g] for x in first[b]]).float(), fmt) for i in range(2))
                                if decode else (kk[old, g].cpu(), vv[old, g].cpu()))
                ref, mag = _ref_attend(q[cu_q[b]:cu_q[b] + m, h].cpu(), keys, values, s.dim ** -0.5, seen)
                held_attention(s.out[cu_q[b]:cu_q[b] + m, h], ref, mag, dtype, not decode)
        s.feed_forward()
        s.check_feed_forward(n, dtype)
        used = s.after()
        free = free[used:] + [-1] * used
        lens = s.lens.cpu().tolist()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(FORMATS))
def test_attention_after_a_plan_without_pages(cb, gen, fmt):
    """A request that got no page attends over what it has in the cache, and over nobody else's tokens."""
    page, dim, lens, added = 16, 64, [16, 16, 30], [1, 1, 1]
    table = torch.full((3, 4), -1, dtype=torch.int32)
    table[0, 0], table[1, 0], table[2, :2] = 0, 3, torch.tensor([2, 1])
    plan = glq.KvPlan(table.cuda(), page, 5, 3)
    cache = glq.KvCache.empty(5, page, 2, dim, FORMATS[fmt])
    old = torch.randn(5 * page, 2, dim, generator=gen).to(torch.bfloat16).cuda()
    glq.kv_append(cache, old, old, _ints(list(range(5 * page))))
    q, k = torch.randn(3, 4, dim, generator=gen).cuda().to(torch.bfloat16), torch.randn(3, 2, dim, generator=gen).cuda().to(torch.bfloat16)
    glq.kv_plan(plan, _ints(lens), _ints(added), _ints([4]))       # one page for the two that need one
    assert plan.used.tolist() == [2] and plan.slots.tolist()[1] == -1 and plan.new_lens.tolist() == [17, 17, 31]
    glq.qk_norm_rope(q, k, plan.positions, glq.rotary_table(64, dim), q, k, cache=cache, v=k, slots=plan.slots)
    out = torch.zeros_like(q)
    ws = torch.zeros(glq.attn_decode_workspace_bytes(cache, 3, 4, 64), dtype=torch.uint8, device="cuda")
    glq.attn_decode(cache, q, plan.page_table, plan.new_lens, out, ws, 64)
    for b, slots in enumerate(([*range(16), 64], list(range(48, 64)), [*range(32, 48), *range(16, 31)])):
        kv = [torch.empty(len(slots), 2, dim, device="cuda") for _ in range(2)]
        glq.kv_read(cache, _ints(slots), *kv)
        for h in range(4):
            ref, mag = _ref_attend(q[b, h:h + 1].cpu(), kv[0][:, h // 2].cpu(), kv[1][:, h // 2].cpu(), dim ** -0.5,
                                   torch.ones(1, len(slots), dtype=torch.bool))
            held_attention(out[b, h:h + 1], ref, mag, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("page", [16, 32])
def test_step_in_a_graph(cb, gen, dtype, page):
    """One captured step replayed with other lengths, pages, inputs and padded rows, against the eager step."""
    captured, eager = (Server(cb, "int8", batch=5, most=5, page=page, dtype=dtype) for _ in range(2))
    steps = [[1, 1, 1, 1, 1]] * 12 + [[1, 1, 1, 0, 0], [1, 0, 0, 0, 0], [0, 0, 0, 0, 0], [1, 1, 1, 1, 1], [1, 1, 1, 1, 0]] * 2
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured.step()                                          # (no tokens yet: changes nothing)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for i, added in enumerate(steps):
        state = gen.get_state()
        captured.inputs(gen, added)
        gen.set_state(state)
        eager.inputs(gen, added)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager.step()
        for a, b in zip(captured.results(), eager.results()):
            assert torch.equal(a, b), i
        captured.after(), eager.after()
        if i % 7 == 3:
            eager.check_feed_forward(sum(added), dtype)
    assert eager.lens.cpu().tolist() == [sum(s[b] for s in steps) for b in range(5)]


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 64])
def test_steps_in_a_graph_without_the_host(cb, gen, page):
    """A captured step that takes its own pages off the free list and hands its lengths on, replayed many times before the
    host looks: what single steps with a list on the host give. A replay that did not would hand out the same pages again."""
    device, host = (Server(cb, "int8", batch=5, most=5, page=page) for _ in range(2))
    at, none = torch.arange(device.pages, device="cuda"), torch.full((1,), -1, dtype=torch.int32, device="cuda")

    def step():
        device.step()
        left = torch.cat((device.free_dev, none))
        device.free_dev.copy_(left[(at + device.plan.used).clamp(max=device.pages)])
        device.lens.copy_(device.plan.new_lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                   # (no tokens yet: changes nothing)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for added in [[1, 1, 1, 1, 1], [1, 0, 1, 0, 1], [0, 0, 0, 0, 0], [1, 1, 1, 1, 0]]:
        state = gen.get_state()
        device.inputs(gen, added)
        gen.set_state(state)
        host.inputs(gen, added)
        torch.cuda.synchronize()
        for _ in range(19):                                      # (q and k are rotated in place, again each time)
            graph.replay()
        for _ in range(19):
            host.step()
            host.after()
        torch.cuda.synchronize()
        for a, b in zip(device.results(), host.results()):
            assert torch.equal(a, b)
        assert torch.equal(device.lens, host.lens) and torch.equal(device.free_dev, host.free_dev)


@pytest.mark.gpu
def test_two_graphs_share_workspaces(cb, gen):
    """Two captured steps of different sizes in the same workspaces, replayed in turn."""
    a, b = Server(cb, batch=3, most=70, seed=5), Server(cb, batch=3, most=3, seed=6)
    b.route_ws, b.expert_ws = a.route_ws, a.expert_ws
    graphs = []
    for s in (a, b):
        s.feed_forward()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.feed_forward()
    for i in range(4):
        for s, counts in ((a, [30, 1 + i, 35]), (b, [1, 1, i % 2])):
            s.inputs(gen, counts)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, n in ((a, 66 + i), (b, 2 + i % 2)):
            got = s.results()
            s.check_feed_forward(n, "bf16")
            s.y.fill_(7), s.src.fill_(7), s.pos.fill_(7)
            s.feed_forward()
            assert all(torch.equal(x, y) for x, y in zip(got, s.results()))


@pytest.mark.gpu
def test_streams(cb, gen):
    """Two servers' steps on two streams at once, each with its own buffers: what each gives alone."""
    servers = [Server(cb, batch=4, most=4, seed=8 + i % 2) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        for s in servers:
            s.inputs(gen, [1, 1, 0, 1])
        for alone, other in ((0, 2), (1, 3)):
            for name in ("qkv", "x", "logits"):
                getattr(servers[other], name).copy_(getattr(servers[alone], name))
        torch.cuda.synchronize()
        for s, stream in zip(servers, streams):
            s.step(stream=stream)
        torch.cuda.synchronize()
        for s in servers[2:]:
            s.step()
        for s, other in ((0, 2), (1, 3)):
            assert all(torch.equal(x, y) for x, y in zip(servers[s].results(), servers[other].results()))
        for s in servers:
            s.after()


# ----------------------------------------------------------- workspaces and what lies behind the outputs

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("count,rows,n,k", [(1, 1, 64, 512), (3, 7, 264, 1024), (2, 300, 512, 2048), (8, 64, 1024, 1024),
                                            (1, 256, 256, 16384), (4, 1, 2048, 4096)])
def test_nothing_behind_the_workspaces(cb, dtype, count, rows, n, k):
    gen = torch.Generator().manual_seed(2)
    handle = Set(count, n, k, 4, seed=1).device(cb)
    need = glq.expert_linear_workspace_bytes(handle, rows)
    x = torch.randn(rows, k, generator=gen).to(DTYPES[dtype]).cuda()
    ends = [0] + [rows * (e + 1) // count for e in range(count)]
    outs = []
    for more in (0, 1000):                                       # a workspace for more rows serves fewer
        size = glq.expert_linear_workspace_bytes(handle, rows + more)
        assert size >= need
        ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        y = torch.full((rows + 1, n), 7.0, dtype=x.dtype, device="cuda")
        glq.expert_linear(handle, x, y[:rows], _ints(ends), ws[:size])
        assert (ws[size:] == 0xA5).all() and (y[rows] == 7).all()
        assert (ws[need:] == 0xA5).all()
        outs.append(y)
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_route_workspace_and_sizes(gen):
    for tokens, experts, top in ((64, 8, 2), (65, 8, 2), (500, 100, 7), (97, 1024, 64)):
        logits = torch.randn(tokens, experts, generator=gen).cuda()
        size = glq.route_workspace_bytes(tokens, experts, top)
        ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        w = torch.full((tokens + 1, top), 7.0, device="cuda")
        ids, pos = (torch.full((tokens + 1, top), 7, dtype=torch.int32, device="cuda") for _ in range(2))
        src, offsets = _ints([7] * (tokens * top + 1)), _ints([7] * (experts + 2))
        glq.route(logits, top, w[:tokens], ids[:tokens], pos[:tokens], src[:-1], offsets[:-1], ws[:size])
        assert (ws[size:] == 0xA5).all() and (w[tokens] == 7).all() and (ids[tokens] == 7).all() and (pos[tokens] == 7).all()
        assert src[-1] == 7 and offsets[-1] == 7
        _check_route(logits.cpu(), top, True, [t.cpu() for t in (w[:tokens], ids[:tokens], pos[:tokens], src[:-1], offsets[:-1])])


def _route_many(gen, tokens, experts, top):
    logits = torch.randn(tokens, experts, generator=gen)
    if tokens > 1000:
        logits[tokens // 2:tokens // 2 + 300] = -torch.inf       # a padded batch's rows in the middle
    size = glq.route_workspace_bytes(tokens, experts, top)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    w = torch.empty(tokens, top, device="cuda")
    ids, pos = (torch.empty(tokens, top, dtype=torch.int32, device="cuda") for _ in range(2))
    src, offsets = torch.empty(tokens * top, dtype=torch.int32, device="cuda"), _ints([0] * (experts + 1))
    glq.route(logits.cuda(), top, w, ids, pos, src, offsets, ws[:size])
    assert (ws[size:] == 0xA5).all()
    score, expert = torch.sort(logits.double(), descending=True, stable=True)
    score, expert = score[:, :top], expert[:, :top]
    real = score > -torch.inf
    assert torch.equal(ids.cpu().long(), torch.where(real, expert, -1))
    flat = torch.where(real, expert, experts).flatten()
    order, rows = torch.argsort(flat, stable=True), int(real.sum())
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order))
    assert torch.equal(pos.cpu().long().flatten(), torch.where(real.flatten(), place, -1))
    assert torch.equal(src.cpu().long()[:rows], order[:rows] // top) and (src[rows:] == -1).all()
    assert torch.equal(offsets.cpu().long()[1:], torch.bincount(flat, minlength=experts + 1)[:experts].cumsum(0)) and offsets[0] == 0
    want = torch.where(real, torch.softmax(score.where(real, -1e300), 1), 0.0)
    reach = (score[:, :1] - score[:, -1:]).nan_to_num(0.0)
    assert ((w.double().cpu() - want).abs() <= (2 * (reach + 2) + 25) * 2.0 ** -24 * want + 2.0 ** -126).all()


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,experts,top", [(2048, 24, 3), (2049, 24, 3), (16384, 16, 2), (16385, 16, 2), (32768, 8, 2),
                                                (32769, 8, 2), (100000, 60, 4), (70000, 300, 2), (300001, 8, 1), (40000, 1024, 3)])
def test_route_of_many_tokens(gen, tokens, experts, top):
    """Each number of tokens a workgroup takes, at its ends, and counts added up by groups."""
    _route_many(gen, tokens, experts, top)


def test_route_workspace_grows():
    for experts in (1, 60, 1024):
        sizes = [glq.route_workspace_bytes(t, experts, 1) for t in (1, 64, 65, 1000, 2048, 2049, 5000, 16384, 16385, 32768, 32769, 10 ** 6)]
        assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("n,k", [(264, 4096), (40, 4104), (520, 1088)])
def test_few_rows_an_expert(cb, dtype, bpw, n, k):
    """Tiles of one to five rows, along k in parts and whole, indices in fours and one by one."""
    experts = Set(7, n, k, bpw, seed=8)
    handle = experts.device(cb)
    for counts in ([1, 0, 0, 0, 0, 0, 0], [1, 4, 5, 0, 2, 3, 1]):
        ends = np.concatenate(([0], np.cumsum(counts)))
        rows = int(ends[-1])
        x = torch.randn(rows, k, generator=torch.Generator().manual_seed(n)).to(DTYPES[dtype]).cuda()
        y = torch.full((rows + 1, n), 7.0, dtype=x.dtype, device="cuda")
        ws = torch.full((glq.expert_linear_workspace_bytes(handle, rows),), 255, dtype=torch.uint8, device="cuda")
        glq.expert_linear(handle, x, y[:rows], _ints(ends.tolist()), ws)
        ref = _rows_reference(experts, x.double().cpu().numpy(), ends, None, rows)
        assert (y[rows] == 7).all()
        _held(y[:rows], ref, _tolerance(ref, dtype, k), dtype)
        for _ in range(25):                                      # the same bits each time, whatever the workspace held
            again = torch.full_like(y, 7.0)
            ws.fill_(255)
            glq.expert_linear(handle, x, again[:rows], _ints(ends.tolist()), ws)
            assert torch.equal(y, again)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [5120, 7168, 6144])
def test_rows_of_several_blocks_and_sizes(cb, k):
    """Rows whose waves transform blocks of their own, neighbours of very different sizes: each row has its own power of two."""
    gen = torch.Generator().manual_seed(k)
    rows, experts = 3500, Set(2, 8, k, 2, seed=4)
    handle = experts.device(cb)
    size = torch.where(torch.arange(rows) % 2 == 0, 2.0 ** 40, 2.0 ** -40)[:, None]
    x = (torch.randn(rows, k, generator=gen) * size).to(torch.bfloat16).cuda()
    y = torch.zeros(rows, 8, device="cuda")
    ws = torch.empty(glq.expert_linear_workspace_bytes(handle, rows), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        glq.expert_linear(handle, x, y, _ints([0, 1701, rows]), ws)
        ref = _rows_reference(experts, x.double().cpu().numpy(), [0, 1701, rows], None, rows)
        # (its size by the whole matrix's rows: 8 outputs are too few to take it from)
        rms = np.sqrt((x.double().cpu().numpy() ** 2).mean(1, keepdims=True)) * np.sqrt(k) * experts.scale.max() * np.sqrt(12.0)
        err = np.abs(y.double().cpu().numpy() - ref)
        assert (err <= _tolerance(np.broadcast_to(rms, ref.shape), "bf16", k)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_offsets_that_go_up_and_down(cb, dtype):
    """Far more rows by the offsets than there are: everything stays in bounds, rows outside the first and last are left."""
    handle = Set(64, 64, 1024, 3, seed=4).device(cb)
    rows = 300
    offsets = [5] + [290 if e % 2 == 0 else 5 for e in range(63)] + [290]
    x = torch.randn(rows, 1024, device="cuda").to(DTYPES[dtype])
    size = glq.expert_linear_workspace_bytes(handle, rows)
    ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
    y = torch.full((rows, 64), 7.0, dtype=x.dtype, device="cuda")
    glq.expert_linear(handle, x, y, _ints(offsets), ws[:size])
    assert (y[:5] == 7).all() and (y[290:] == 7).all() and (ws[size:] == 255).all()


# ----------------------------------------------------------- sizes past 32 bits

@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_rope_into_a_cache_beyond_32_bits(gen, fmt):
    page, heads, dim = 1024, 8, 256
    pages = 1100 if fmt == "bf16" else 4400                      # over 4 GiB a side
    caches = [glq.KvCache.empty(pages, page, heads, dim, FORMATS[fmt]) for _ in range(2)]
    assert caches[0].k.nbytes > 2 ** 32
    tokens = 9
    last = pages * page
    slots = _ints([last - 1, 0, last // 2, last - page, -1, last, last - 2, last // 4 * 3, 2 ** 31 - 1])
    k, v = (torch.randn(tokens, heads, dim, generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.randn(tokens, 16, dim, generator=gen).to(torch.bfloat16).cuda()
    table, pos = glq.rotary_table(50, dim), torch.arange(tokens, dtype=torch.int32).cuda()
    ko = torch.empty_like(k)
    glq.qk_norm_rope(q, k, pos, table, q.clone(), ko, cache=caches[0], v=v, slots=slots)
    glq.kv_append(caches[1], ko, v, slots)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)
    assert caches[0].k[-1].any() and caches[0].k[pages // 2].any()


@pytest.mark.gpu
def test_rope_rows_beyond_32_bits(gen):
    tokens, dim, step = 4, 64, 2 ** 30 + 64                      # bf16 elements between rows: 6 GiB in all
    flat = torch.zeros(3 * step + 3 * dim, dtype=torch.bfloat16, device="cuda")
    rows = flat.as_strided((tokens, 3, dim), (step, dim, 1))
    x = torch.randn(tokens, 3, dim, generator=gen).to(torch.bfloat16).cuda()
    rows.copy_(x)
    table, pos = glq.rotary_table(9, dim), _ints([3, 8, 1, 0])
    w = torch.ones(dim, device="cuda")
    want = [torch.empty(tokens, h, dim, dtype=torch.bfloat16, device="cuda") for h in (2, 1)]
    glq.qk_norm_rope(x[:, :2], x[:, 2:], pos, table, *want, w, w)
    glq.qk_norm_rope(rows[:, :2], rows[:, 2:], pos, table, rows[:, :2], rows[:, 2:], w, w)
    assert torch.equal(rows[:, :2], want[0]) and torch.equal(rows[:, 2:], want[1])


@pytest.mark.gpu
def test_gathered_rows_beyond_32_bits(cb):
    gen = torch.Generator().manual_seed(1)
    experts, k, many = Set(2, 64, 8192, 2, seed=9), 8192, 300000
    handle = experts.device(cb)
    x = torch.zeros(many, k, dtype=torch.bfloat16, device="cuda")
    at = [many - 1, 0, 262143, 262144, 131072, many - 2]
    x[at] = torch.randn(len(at), k, generator=gen).to(torch.bfloat16).cuda()
    y = torch.zeros(len(at), 64, device="cuda")
    ws = torch.empty(glq.expert_linear_workspace_bytes(handle, len(at)), dtype=torch.uint8, device="cuda")
    glq.expert_linear(handle, x, y, _ints([0, 4, 6]), ws, src=_ints(at))
    ref = _rows_reference(experts, x[at].double().cpu().numpy(), [0, 4, 6], None, len(at))
    _held(y, ref, _tolerance(ref, "bf16", k), "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_and_weights_beyond_32_bits(cb, dtype):
    """The indices of the last experts, and in float32 z and y of the last rows, lie past 4 GiB."""
    count, n, k, rows = 600, 8192, 4096, 140000
    gen = torch.Generator(device="cuda").manual_seed(1)
    idx1 = torch.randint(-32768, 32768, (count, n, k // 8), generator=gen, dtype=torch.int16, device="cuda")
    assert idx1.nbytes > 2 ** 32
    sign = [(torch.randint(0, 2, (count, m), generator=gen, device="cuda") * 2 - 1).to(torch.int8) for m in (k, n)]
    scale = torch.full((count,), 0.02, device="cuda")
    handle = glq.Experts(count, n, k, 2, scale, idx1, None, *sign, cb)
    x = torch.randn(rows, k, generator=gen, device="cuda").to(DTYPES[dtype])
    y = torch.empty(rows, n, dtype=x.dtype, device="cuda")
    ends = [0] * (count - 1) + [rows - 5, rows]                  # nearly all rows are of the last but one
    ws = torch.empty(glq.expert_linear_workspace_bytes(handle, rows), dtype=torch.uint8, device="cuda")
    glq.expert_linear(handle, x, y, _ints(ends), ws)
    from oracle import glq as oracle
    for e, take in ((count - 2, [0, 32768, 65535, rows - 6]), (count - 1, [rows - 5, rows - 1])):
        ref = oracle.layer_reference(x[take].double().cpu().numpy(), idx1[e].cpu().numpy().view(np.uint16), None, 2,
                                     np.float32(0.02), sign[1][e].cpu().numpy(), sign[0][e].cpu().numpy())
        _held(y[take], ref, _tolerance(ref, dtype, k), dtype)


# ----------------------------------------------------------- refusals of the binding

@pytest.mark.gpu
def test_refuses_another_device(cb, monkeypatch):
    s = Server(cb, batch=2, most=2)
    q, k, v = s.projected()
    calls = (lambda **c: glq.kv_plan(s.plan, s.lens, s.added, s.free_dev, **c),
             lambda **c: glq.qk_norm_rope(q, k, s.plan.positions, s.table, q, k, s.wq, s.wk, cache=s.cache, v=v,
                                          slots=s.plan.slots, **c),
             lambda **c: glq.route(s.logits, s.top, s.weights, s.ids, s.pos, s.src, s.offsets, s.route_ws, **c),
             lambda **c: glq.expert_linear(s.up, s.x, s.inside, s.offsets, s.expert_ws, src=s.src, **c))

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
def test_binding_refusals(cb):
    s = Server(cb, batch=2, most=70)
    q, k, v = s.projected()
    half = q.to(torch.float16)
    long = s.lens.long()

    def refused(call, *args, **kw):
        with pytest.raises((ValueError, glq.GlqError)):
            call(*args, **kw)
    # the plan
    for lens, added, free in ((long, s.added, s.free_dev), (s.lens[:1], s.added, s.free_dev), (s.lens, s.added.cpu(), s.free_dev),
                              (s.lens, s.added, s.free_dev[::2]), (s.lens, None, s.free_dev),
                              (s.plan.new_lens, s.added, s.free_dev)):      # (where the new lengths go)
        refused(glq.kv_plan, s.plan, lens, added, free)
    refused(glq.KvPlan, s.plan.page_table.long(), 16, 9, 4)
    refused(glq.KvPlan, s.plan.page_table[:, ::2], 16, 9, 4)
    refused(glq.KvPlan, s.plan.page_table, 16, 9, -4)
    refused(glq.kv_plan, glq.KvPlan(s.plan.page_table.clone(), 24, 9, 4), s.lens, s.added, s.free_dev)
    # norms and rotation
    args = dict(q=q, k=k, positions=s.plan.positions, rotary=s.table, q_out=q, k_out=k, q_weight=s.wq, k_weight=s.wk,
                cache=s.cache, v=v, slots=s.plan.slots)
    glq.qk_norm_rope(**args)
    for change in (dict(q=half), dict(k=half), dict(q=q.float()), dict(q=q[:3]), dict(k=k[..., :32]), dict(q=q.transpose(0, 1)),
                   dict(positions=s.plan.positions.long()), dict(positions=s.plan.positions[:2]), dict(positions=None),
                   dict(rotary=s.table[:, :63]), dict(rotary=s.table.double()), dict(rotary=s.table[0]), dict(q_out=q[:2]),
                   dict(k_out=q), dict(q_weight=s.wq[:32]), dict(k_weight=s.wk.double()), dict(v=None), dict(slots=None),
                   dict(v=q), dict(slots=s.plan.slots.long()), dict(cache=None), dict(eps=-1.0), dict(eps=float("nan")),
                   dict(q=q.cpu()), dict(rotary=s.table.cpu()), dict(cache=None, v=None, slots=None, k_out=None)):
        refused(glq.qk_norm_rope, **{**args, **change})
    overlapping = q.as_strided(q.shape, (64, 64, 1))
    refused(glq.qk_norm_rope, **{**args, "q": overlapping})
    packed = s.qkv.view(-1)[:q.numel()].view(q.shape)            # where q begins, in rows of another stride
    refused(glq.qk_norm_rope, **{**args, "q_out": packed})
    # routing
    args = [s.logits, s.top, s.weights, s.ids, s.pos, s.src, s.offsets, s.route_ws]
    glq.route(*args)
    for i, bad in ((0, s.logits.double()), (0, s.logits.cpu()), (0, s.logits.t()), (1, 3), (2, s.weights.double()), (3, s.ids.long()),
                   (4, s.pos[:2]), (5, s.src[1:]), (6, s.offsets[1:]), (7, s.route_ws.cpu()), (7, s.route_ws[1:]), (7, None)):
        refused(glq.route, *[bad if j == i else a for j, a in enumerate(args)])
    # experts
    args = dict(experts=s.down, x=s.inside, y=s.y, offsets=s.offsets, workspace=s.expert_ws, pos=s.pos, weights=s.weights)
    glq.expert_linear(**args)
    for change in (dict(x=s.inside.half()), dict(x=s.inside[:, 8:]), dict(x=s.x), dict(y=s.y[:2]), dict(y=s.inside), dict(weights=None),
                   dict(pos=s.pos.long()), dict(weights=s.weights.double()), dict(offsets=s.offsets[:-1]), dict(pos=None),
                   dict(offsets=s.offsets.long()), dict(workspace=s.expert_ws[:512]), dict(workspace=s.expert_ws[1:]),
                   dict(workspace=s.expert_ws.cpu()), dict(src=s.src.long()), dict(pos=s.pos[:, :0], weights=s.weights[:, :0])):
        refused(glq.expert_linear, **{**args, **change})
    e = s.up
    good = dict(count=e.count, n=e.n, k=e.k, bpw=e.bpw, scale=e.scale, idx1=e.idx1, idx2=e.idx2, sign_k=e.sign_k, sign_n=e.sign_n, cb=e.cb)
    glq.Experts(**good)
    for change in (dict(bpw=5), dict(n=12), dict(count=0), dict(scale=e.scale.double()), dict(idx1=e.idx1[1:]), dict(idx2=None), dict(bpw=2),
                   dict(bpw=3), dict(sign_k=e.sign_n), dict(sign_n=e.sign_n.float()), dict(cb=e.cb[:64]), dict(scale=e.scale.cpu()),
                   dict(row_scale=e.scale)):
        refused(glq.Experts, **{**good, **change})


@pytest.mark.gpu
def test_nothing_to_do(cb):
    """No tokens and no rows: successful calls that touch nothing."""
    s = Server(cb, batch=2, most=4)
    q, k, v = s.projected()
    none = _ints([])
    glq.qk_norm_rope(q[:0], k[:0], none, s.table, q[:0], k[:0], cache=s.cache, v=v[:0], slots=none)
    assert not s.cache.k.any()
    s.offsets.fill_(7)
    glq.route(s.logits[:0], s.top, s.weights[:0], s.ids[:0], s.pos[:0], none, s.offsets, s.route_ws)
    assert not s.offsets.any()
    glq.expert_linear(s.up, s.x, s.inside[:0], s.offsets, s.expert_ws, src=none)
    s.y.fill_(7)
    glq.expert_linear(s.down, s.inside[:0], s.y, s.offsets, s.expert_ws, pos=s.pos, weights=s.weights)
    assert not s.y.any()                                         # tokens without rows
    glq.expert_linear(s.down, s.inside[:0], s.y[:0], s.offsets, s.expert_ws, pos=s.pos[:0], weights=s.weights[:0])


@pytest.mark.gpu
def test_stacked_layers(cb):
    """Experts of single layers, and what does not stack."""
    gen = torch.Generator().manual_seed(4)
    one = Set(3, 64, 128, 3, seed=2)
    layers = [glq.Layer.from_numpy(one.idx1[e], one.idx2[e], one.scale[e], one.sign_n[e], one.sign_k[e], cb) for e in range(3)]
    handle = glq.Experts.stack(layers)
    x = torch.randn(9, 128, generator=gen).cuda()
    y = torch.empty(9, 64, device="cuda")
    ws = torch.empty(glq.expert_linear_workspace_bytes(handle, 9), dtype=torch.uint8, device="cuda")
    glq.expert_linear(handle, x, y, _ints([0, 2, 2, 9]), ws)
    ref = _rows_reference(one, x.double().cpu().numpy(), [0, 2, 2, 9], None, 9)
    _held(y, ref, _tolerance(ref, "f32", 128), "f32")
    other = Set(1, 72, 128, 3, seed=2)
    with pytest.raises(ValueError):
        glq.Experts.stack(layers + [glq.Layer.from_numpy(other.idx1[0], other.idx2[0], other.scale[0], other.sign_n[0],
                                                         other.sign_k[0], cb)])
    with pytest.raises(ValueError):
        glq.Experts.stack([])


# ----------------------------------------------------------- refusals of the C ABI (nothing is launched)

@pytest.mark.parametrize("change,status", [({"max_tokens": 2 ** 31 - 4096}, -2), ({"max_read": 2 ** 31 - 4096}, -2),
                                           ({"batch": 2 ** 20, "max_pages": 2 ** 11}, -2), ({"batch": -1}, -1)])
def test_plan_refuses_lists_past_32_bits(change, status):
    p = 4096
    st = glq.PlanStruct(2, 4, 100, 16, p, p + 64, p + 128, 5, p + 256, p + 512, p + 576, 7, p + 640, p + 768, 9, p + 896,
                        p + 960, p + 1024)
    for name, value in change.items():
        setattr(st, name, value)
    assert glq.raw().glq_kv_plan(ctypes.byref(st), None) == status


@pytest.mark.parametrize("change", [{"q_out_stride": 512}, {"k_out_stride": 512}])
def test_norm_rope_refuses_its_input_in_another_stride(change):
    p = 4096
    st = glq.QkStruct(p, p + 512, p, p + 512, 1, 4, 2, 64, 256, 128, 256, 128, 3, p, p, 1e-6, 64, p, p, 10, 0, 0, 0)
    for name, value in change.items():
        setattr(st, name, value)
    assert glq.raw().glq_qk_norm_rope(ctypes.byref(st), None, 0, None) == -1
