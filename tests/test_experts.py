"""Compressed linears of experts on ragged groups of rows: GPU results against the plain
float64 oracle of one layer per expert, the refusals on the CPU, and a step of routing and experts.

Tolerances, per output element, with S the 2-norm over sqrt(n) of its row of the reference (the
transforms keep 2-norms, so z's rows have it too):
  bf16     x~ is rounded to bf16: at most 2^-8 relative an element, uniform errors of at most 2^-8 /
           sqrt(3) in the mean square; their products with independent weights add up to the same part of
           S. Six standard deviations of it, and half a step of the output, 2^-8 of the value.
  float32  products of float32 operands, whose float32 sums have 3 k + log2 k + log2 n roundings of
           2^-24 S at random (log2 k + log2 n <= 28): sqrt(3 k + 28) 2^-24 S, six standard deviations of it
           (over sqrt(3)). A part of x~ that got lost is 2^-17 of it.
A token's sum of rows: the sum of weight times either.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import glq as oracle

glq = pytest.importorskip("dequant_e8_codebook_amd.glq")

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


class Set:
    """Experts of random indices on the device, and each as the oracle takes it."""

    def __init__(self, count, n, k, bpw, seed=0, row_scale=False):
        rng = np.random.default_rng(seed)
        self.count, self.n, self.k, self.bpw = count, n, k, bpw
        self.idx1 = rng.integers(0, 65536, (count, n, k // 8)).astype(np.uint16)
        self.idx2 = None if bpw == 2 else rng.integers(0, 256 if bpw == 3 else 65536, self.idx1.shape).astype(
            np.uint8 if bpw == 3 else np.uint16)
        self.sign_k, self.sign_n = (rng.integers(0, 2, (count, m)).astype(np.int8) * 2 - 1 for m in (k, n))
        self.scale = rng.uniform(0.01, 0.03, count).astype(np.float32)
        self.row_scale = rng.uniform(0.5, 2, (count, n)).astype(np.float32) if row_scale else None

    def device(self, cb):
        def dev(a):
            return None if a is None else torch.from_numpy(a).cuda()
        i2 = self.idx2.view(np.int16) if self.bpw == 4 else self.idx2
        return glq.Experts(self.count, self.n, self.k, self.bpw, dev(self.scale), dev(self.idx1.view(np.int16)), dev(i2),
                           dev(self.sign_k), dev(self.sign_n), cb, dev(self.row_scale))

    def reference(self, e, x):
        scale = self.scale[e] if self.row_scale is None else self.scale[e] * self.row_scale[e]
        return oracle.layer_reference(x, self.idx1[e], None if self.idx2 is None else self.idx2[e], self.bpw, scale,
                                      self.sign_n[e], self.sign_k[e])


@pytest.fixture(scope="module")
def cb():
    return glq.device_codebook()


def _rows_reference(experts, x, offsets, src, rows):
    """float64 [rows, n] by the words; rows that are no expert's stay NaN."""
    out = np.full((rows, experts.n), np.nan)
    for e in range(experts.count):
        at = np.arange(max(offsets[e], 0), min(offsets[e + 1], rows))
        if len(at):
            of = at if src is None else src[at]
            take = np.where(((of >= 0) & (of < len(x)))[:, None], x[np.clip(of, 0, len(x) - 1)], 0.0)
            out[at] = experts.reference(e, take)
    return out


def _tolerance(ref, dtype, k, weights=None):
    """[rows, n]: see above; with weights [tokens, top], ref is [tokens, top, n]."""
    size = np.sqrt((ref ** 2).mean(-1, keepdims=True))
    part = 6 / np.sqrt(3) * (2.0 ** -8 if dtype == "bf16" else np.sqrt(3 * k + 28) * 2.0 ** -24) * size
    if weights is not None:
        part = (part * np.abs(weights)[..., None]).sum(1)
    return part + 1e-30


def _held(y, ref, tol, y_dtype):
    got = y.double().cpu().numpy()
    tol = tol + (2.0 ** -8 if y_dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + tol)
    err = np.abs(got - ref)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), f"worst {(err / tol).max():.3g} of the tolerance"


def _inputs(seed, rows, k, dtype):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(rows, k, generator=gen).to(DTYPES[dtype]).cuda()


def _workspace(experts, rows, fill=255):
    return torch.full((glq.expert_linear_workspace_bytes(experts, rows),), fill, dtype=torch.uint8, device="cuda")


def _check_rows(cb, experts, counts, dtype, y_dtype=None, first=0, behind=0, seed=1):
    """Counts of rows an expert, `first` rows before them and `behind` after them that are none's."""
    y_dtype = y_dtype or dtype
    offsets = np.concatenate(([first], first + np.cumsum(counts)))
    rows = int(offsets[-1]) + behind
    x = _inputs(seed, rows, experts.k, dtype)
    y = torch.full((rows, experts.n), 7.0, dtype=DTYPES[y_dtype], device="cuda")
    handle = experts.device(cb)
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, rows)
    assert (y[:first] == 7).all() and (y[int(offsets[-1]):] == 7).all()
    own = slice(first, int(offsets[-1]))
    _held(y[own], ref[own], _tolerance(ref[own], dtype, experts.k), y_dtype)


COUNTS = {"one": [1], "one of many": [0, 0, 1, 0], "empty between": [3, 0, 17, 0, 0, 1], "tiles": [16, 15, 17, 32, 33],
          "more": [64, 65, 1, 130, 0], "many": [300, 5, 257]}


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("n,k", [(64, 128), (200, 328), (256, 512)])
def test_rows(cb, dtype, bpw, counts, n, k):
    counts = COUNTS[counts]
    _check_rows(cb, Set(len(counts), n, k, bpw, seed=n + bpw), counts, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,bpw", [(8, 8, 4), (8, 4096, 2), (1416, 16, 3), (24, 1000, 4), (2048, 2048, 4), (1024, 4096, 3),
                                     (4096, 1024, 2), (520, 2056, 3)])
def test_shapes(cb, dtype, n, k, bpw):
    _check_rows(cb, Set(3, n, k, bpw, seed=k), [5, 0, 40], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(16384, 64), (64, 16384), (8192, 256), (256, 8192), (9216, 128), (128, 10240), (24, 16392),
                                 (20480, 64)])
def test_long_rows(cb, n, k):
    """Hadamard blocks of 8192 and 16384, rows longer than a workgroup holds."""
    _check_rows(cb, Set(2, n, k, 2, seed=3), [2, 3], "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("n,k", [(64, 49152), (49152, 64), (64, 24576), (24576, 64), (128, 10240), (24, 16392), (8, 20480)])
def test_rows_longer_than_a_workgroup(cb, dtype, bpw, n, k):
    """Rows in several segments: their sums, their three parts in float32, blocks of 16384 more than once."""
    experts = Set(2, n, k, bpw, seed=3)
    offsets, x = [0, 2, 5], _inputs(1, 5, k, dtype)
    handle, y = experts.device(cb), torch.full((6, n), 7.0, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y[:5], torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, 5))
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, 5)
    # (the size of 8 outputs by the whole matrix's rows)
    size = ref if n > 8 else np.broadcast_to(np.sqrt(k * 12.0) * experts.scale.max(), ref.shape)
    assert (y[5] == 7).all()
    _held(y[:5], ref, _tolerance(size, dtype, k), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,bpw,counts", [(264, 4096, 3, [40]), (64, 8192, 4, [300]), (512, 2048, 4, [33, 70]),
                                            (256, 1096, 2, [70, 0]), (1000, 1416, 3, [257, 100, 31])])
def test_split_along_k(cb, dtype, n, k, bpw, counts):
    """Few tiles: their parts along k run side by side and meet in the output's transform."""
    _check_rows(cb, Set(len(counts), n, k, bpw, seed=2), counts, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("bpw", [3, 4])
def test_whole_rounds_and_a_split_rest(cb, bpw):
    """More tiles than the card has places: 16 whole units as they are, what is left in two parts."""
    _check_rows(cb, Set(2, 4096, 1024, bpw, seed=2), [4200, 152], "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("size", [2.0 ** -120, 1e-30, 1e30, 2.0 ** 120])
@pytest.mark.parametrize("counts", [[3, 1], [70, 40]])
def test_sizes_of_inputs(cb, size, counts):
    """What lies between the product and the output's transform keeps its bits at any size of a row."""
    experts = Set(2, 128, 256, 4)
    handle, offsets, rows = experts.device(cb), [0, counts[0], sum(counts)], sum(counts)
    x = (_inputs(3, rows, 256, "bf16").double() * size).to(torch.bfloat16)
    x[0] = 0
    x[0, 3] = size                                         # one element alone, after a transform all of them
    x[rows - 1, :] = x[rows - 1, 0]                        # equal ones, after it one of each block
    y = torch.empty(rows, 128, dtype=torch.bfloat16, device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, rows)
    _held(y, ref, _tolerance(ref, "bf16", 256), "bf16")


def _held_at_the_ends(experts, x, y, offsets, y_dtype):
    """As _held, with no absolute term but a few of the smallest numbers (x~ and z are at least as large as y here)."""
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, len(x))
    size = np.sqrt((ref ** 2).mean(-1, keepdims=True))
    tol = 6 / np.sqrt(3) * 2.0 ** -8 * size
    tol = tol + (2.0 ** -8 if y_dtype == "bf16" else 2.0 ** -24) * (np.abs(ref) + tol) + 2.0 ** -126
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), f"worst {(np.abs(got - ref) / tol).max():.3g} of the tolerance"


@pytest.mark.gpu
@pytest.mark.parametrize("y_dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,rows", [(128, 256, 3), (1024, 4096, 3), (1024, 1024, 700), (264, 5120, 40)])
@pytest.mark.parametrize("size,scale", [(123, 0), (123, -30), (110, 13), (60, 60), (-60, -60), (-110, 0), (-126, 0), (-126, 100), (-130, 120)])
def test_factors_at_the_ends_of_float32(cb, y_dtype, n, k, rows, size, scale):
    """A row's power of two times its scale may leave the range that y does not leave."""
    experts = Set(2, n, k, 2, seed=7)
    experts.scale[:] = 2.0 ** scale
    handle, x = experts.device(cb), torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    x[torch.arange(rows), torch.arange(rows) * 7 % k] = 2.0 ** size
    offsets = [0, rows // 3, rows]
    y = torch.empty(rows, n, dtype=DTYPES[y_dtype], device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    _held_at_the_ends(experts, x, y, offsets, y_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,k", [(64, 128), (1024, 1024)])
def test_scales_of_any_sign(cb, dtype, n, k):
    """An expert's scale is a factor like any other: below zero, and zero."""
    experts = Set(3, n, k, 4, seed=7)
    experts.scale[:] = -0.02, 0.0, -1.5 * 2.0 ** -70
    handle, offsets = experts.device(cb), [0, 5, 9, 12]
    x = _inputs(2, 12, k, dtype)
    x[9:] *= 2.0 ** 60
    y = torch.empty(12, n, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, 12))
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, 12)
    _held(y, ref, _tolerance(ref, dtype, k), dtype)
    assert not y[5:9].any()


@pytest.mark.gpu
@pytest.mark.parametrize("k,rows", [(256, 3), (4096, 3), (1024, 1400), (2048, 3), (16384, 3), (5120, 40)])
@pytest.mark.parametrize("size,scale", [(127, -24), (126, -24), (-126, 60), (-133, 60), (-110, 60)])
def test_rows_at_the_ends_of_bfloat16(cb, k, rows, size, scale):
    """Sums of neighbours that float32 does not hold, and elements below the normal numbers."""
    experts = Set(2, 256, k, 2, seed=7)
    experts.scale[:] = 2.0 ** scale
    gen = torch.Generator().manual_seed(k)
    x = ((1 + 0.99 * torch.rand(rows, k, generator=gen, dtype=torch.float64)) * 2.0 ** size).to(torch.bfloat16)
    x = torch.where(torch.rand(rows, k, generator=gen) < 0.5, -x, x).clamp(-torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).max).cuda()
    handle, offsets = experts.device(cb), [0, rows // 3, rows]
    y = torch.empty(rows, 256, device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    _held_at_the_ends(experts, x, y, offsets, "f32")


def _held_to_float32(experts, x, y, offsets, y_dtype, partial=1.0):
    """For x whose x~ is exact in bf16: what is left are float32 sums (of parts `partial` times as large as z), and y's rounding."""
    ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, len(x))
    tol = _tolerance(ref, "f32", experts.k) * partial
    _held(y, ref, tol, y_dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("row_scale", [False, True])
@pytest.mark.parametrize("count,rows,n,k", [(2, 3, 1024, 4096), (2, 40, 136, 256), (2, 700, 1024, 1024), (3, 300, 264, 1024),
                                            (2, 1100, 2048, 256)])
def test_float32_outputs_of_bfloat16_rows(cb, bpw, row_scale, count, rows, n, k):
    """Nothing but x~ has fewer than float32's bits on the way to a float32 y: rows of two elements, whose x~ are 1 + 2^-6 or 1 - 2^-6
    times a power of two, so that z has more bits than 11."""
    experts = Set(count, n, k, bpw, seed=5, row_scale=row_scale)
    handle, x = experts.device(cb), torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    r = torch.arange(rows)                                       # (odd elements: x~ changes its sign from one to the next)
    x[r, r * 6 % k + 1] = 2.0
    x[r, (r * 6 + 2 + 2 * (r % 5)) % k + 1] = 2.0 ** -5
    offsets = [rows * e // count for e in range(count + 1)]
    y = torch.empty(rows, n, device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    _held_to_float32(experts, x, y, offsets, "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("y_dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,counts", [(256, 4096, [3]), (1024, 4096, [2, 1]), (264, 1024, [40, 20]), (4096, 1024, [2100, 76])])
def test_parts_along_k_that_cancel(cb, bpw, y_dtype, n, k, counts):
    """Sums of parts are float32 sums: the weights of both halves of a row are the same and x~ of the second is that of
    the first with another sign, but for 2^-6 of it, which is all that z is."""
    experts = Set(len(counts), n, k, bpw, seed=5)
    for idx in (experts.idx1, experts.idx2):
        if idx is not None:
            idx[:, :, k // 16:] = idx[:, :, :k // 16]
    rows, offsets = sum(counts), np.concatenate(([0], np.cumsum(counts)))
    handle, x = experts.device(cb), torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(rows) * 6 % (k // 2) + 1
    x[torch.arange(rows), k // 2 + at] = 2.0
    x[torch.arange(rows), at] = 2.0 ** -5
    y = torch.empty(rows, n, dtype=DTYPES[y_dtype], device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows))
    _held_to_float32(experts, x, y, offsets, y_dtype, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("n,k", [(1000, 64), (1024, 128), (8200, 64)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_and_outputs_of_8_million_elements(cb, n, k, dtype):
    """Where z of bfloat16 calls is float16: just below that size, at it and above, summed up and not."""
    experts = Set(3, n, k, 3, seed=11)
    handle, most = experts.device(cb), -(-2 ** 23 // n)
    for rows in (most - 1, most, most + 300):
        offsets, x = [0, 100, rows // 2, rows], _inputs(rows, rows, k, dtype)
        y = torch.empty(rows, n, dtype=x.dtype, device="cuda")
        dev = torch.tensor(offsets, dtype=torch.int32).cuda()
        glq.expert_linear(handle, x, y, dev, _workspace(handle, rows))
        ref = _rows_reference(experts, x.double().cpu().numpy(), offsets, None, rows)
        _held(y, ref, _tolerance(ref, dtype, k), dtype)
        pos = torch.tensor([[0, rows - 1], [rows // 2, -1], [rows - 2, 150]], dtype=torch.int32)
        w = torch.tensor([[0.5, 2.0], [1.0, 3.0], [-1.0, 0.25]])
        s = torch.empty(3, n, dtype=x.dtype, device="cuda")
        glq.expert_linear(handle, x, s, dev, _workspace(handle, rows), pos=pos.cuda(), weights=w.cuda())
        each = np.where((pos >= 0).numpy()[..., None], ref[pos.numpy().clip(0)], 0.0)
        _held(s, (each * w.numpy()[..., None]).sum(1), _tolerance(each, dtype, k, w.numpy()), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("bpw", [2, 3, 4])
@pytest.mark.parametrize("dtype,y_dtype", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_row_scales_and_rows_of_none(cb, bpw, dtype, y_dtype):
    _check_rows(cb, Set(4, 136, 256, bpw, seed=9, row_scale=True), [7, 70, 0, 20], dtype, y_dtype, first=3, behind=11)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [136, 1024, 8192])
@pytest.mark.parametrize("at", [1, 2, 3])
def test_row_scales_at_any_word(cb, n, at):
    experts = Set(2, n, 256, 3, seed=9, row_scale=True)
    handle, x, offsets = experts.device(cb), _inputs(4, 30, 256, "bf16"), torch.tensor([0, 11, 30], dtype=torch.int32).cuda()
    y, moved = (torch.empty(30, n, device="cuda") for _ in range(2))
    glq.expert_linear(handle, x, y, offsets, _workspace(handle, 30))
    flat = torch.zeros(2 * n + at, device="cuda")
    flat[at:] = handle.row_scale.flatten()
    off = glq.Experts(2, n, 256, 3, handle.scale, handle.idx1, handle.idx2, handle.sign_k, handle.sign_n, cb, flat[at:].view(2, n))
    assert off.row_scale.data_ptr() % 16 == 4 * at
    glq.expert_linear(off, x, moved, offsets, _workspace(off, 30))
    assert torch.equal(y, moved)
    ref = _rows_reference(experts, x.double().cpu().numpy(), [0, 11, 30], None, 30)
    _held(y, ref, _tolerance(ref, "bf16", 256), "f32")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_experts(cb, dtype):
    rng = np.random.default_rng(4)
    counts = rng.integers(0, 6, 300) * (rng.random(300) < 0.6)
    counts[-1] = 70
    _check_rows(cb, Set(300, 64, 64, 3, seed=8), counts, dtype)
    counts = np.zeros(1024, int)
    counts[[0, 63, 64, 1023]] = 1, 20, 3, 2
    _check_rows(cb, Set(1024, 16, 64, 2, seed=8), counts, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,count,top,n,k,bpw", [(1, 8, 2, 256, 512, 4), (1, 1, 1, 64, 64, 2), (33, 16, 4, 128, 256, 3),
                                                      (200, 6, 2, 200, 264, 2), (90, 60, 6, 64, 128, 4)])
def test_routed(cb, dtype, tokens, count, top, n, k, bpw):
    """route, then the experts with gathered rows and weighted sums; some tokens have no experts."""
    gen = torch.Generator().manual_seed(tokens)
    logits = torch.randn(tokens, count, generator=gen)
    if tokens > 2:
        logits[tokens - 2:] = -torch.inf
        logits[0, 1:] = -torch.inf
    weights, x = torch.empty(tokens, top, device="cuda"), _inputs(2, tokens, k, dtype)
    ids, pos = (torch.empty(tokens, top, dtype=torch.int32, device="cuda") for _ in range(2))
    src, offsets = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (tokens * top, count + 1))
    ws = torch.empty(glq.route_workspace_bytes(tokens, count, top), dtype=torch.uint8, device="cuda")
    glq.route(logits.cuda(), top, weights, ids, pos, src, offsets, ws)
    experts = Set(count, n, k, bpw, seed=6)
    handle = experts.device(cb)
    y = torch.full((tokens, n), 7.0, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y, offsets, _workspace(handle, tokens * top), src=src, pos=pos, weights=weights)
    xn, w, ids = x.double().cpu().numpy(), weights.double().cpu().numpy(), ids.cpu().numpy()
    each = np.zeros((tokens, top, n))
    for e in range(count):
        t, j = np.nonzero(ids == e)
        if len(t):
            each[t, j] = experts.reference(e, xn[t])
    _held(y, (each * w[..., None]).sum(1), _tolerance(each, dtype, k, w), dtype)
    # the same rows, neither gathered nor summed: the sums' parts
    rows = int(offsets[-1])
    part = torch.zeros(tokens * top, n, device="cuda")
    xr = x[src.long().clamp(min=0)]
    glq.expert_linear(handle, xr, part, offsets, _workspace(handle, tokens * top, 0))
    again = torch.zeros(tokens, n, device="cuda")
    for j in range(top):                                   # in the order of the choices
        p = pos[:, j].long()
        again = torch.where((p >= 0)[:, None], torch.addcmul(again, part[p.clamp(min=0)], weights[:, j:j + 1]), again)
    assert rows == (ids >= 0).sum()
    # u = 2^-24 of the sum of the terms' sizes: a sum rounds its factor (weight / sqrt(b), times the scale) twice, each
    # multiply-add once; a part its factor once and its product once, and here the weight's product once and each sum
    # once: 2 + 2 + 1 u, and 2 u for each of the top_k sums. For bf16 the one rounding of y, half a step.
    err = (again - y.float()).abs().cpu().numpy()
    tol = (5 + 2 * top) * 2.0 ** -24 * np.abs(each * w[..., None]).sum(1) * 1.01
    assert (err <= tol + (2.0 ** -8 * (np.abs(again.cpu().numpy()) + tol) if dtype == "bf16" else 0)).all()


def _combined(rows, pos, weights, dtype, k):
    """The sums of rows that pos [tokens, top] names (none where it is -1), and what _tolerance gives them."""
    out, tol = np.zeros((len(pos), rows.shape[1])), 0.0
    for p, w in zip(pos.T, weights.T):
        each = np.where((p >= 0)[:, None], rows[p.clip(0)], 0.0)
        out += each * w[:, None]
        tol = tol + _tolerance(each, dtype, k) * np.abs(w)[:, None]
    return out, tol


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("row_scale", [False, True])
@pytest.mark.parametrize("tokens,count,top,n,k,bpw", [
    (1, 4, 2, 1024, 1024, 2), (1, 3, 1, 8192, 2048, 3), (5, 8, 8, 2048, 1024, 4), (64, 8, 3, 1024, 4096, 2), (256, 6, 2, 4096, 1024, 3),
    (257, 6, 2, 4096, 1024, 3), (300, 5, 3, 5120, 2048, 2), (40, 8, 8, 1024, 5120, 4), (9, 2, 2, 16384, 1024, 2), (33, 7, 5, 6144, 6144, 3)])
def test_routed_rows_of_whole_blocks(cb, dtype, row_scale, tokens, count, top, n, k, bpw):
    """Sets of waves that share a token's choices and one alone; tokens without experts or with fewer than top."""
    gen = torch.Generator().manual_seed(tokens + n)
    logits = torch.randn(tokens, count, generator=gen)
    if tokens > 4:
        logits[1] = logits[tokens - 1] = -torch.inf
        logits[3, 1:] = -torch.inf
    weights, x = torch.empty(tokens, top, device="cuda"), _inputs(2, tokens, k, dtype)
    ids, pos = (torch.empty(tokens, top, dtype=torch.int32, device="cuda") for _ in range(2))
    src, offsets = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (tokens * top, count + 1))
    ws = torch.empty(glq.route_workspace_bytes(tokens, count, top), dtype=torch.uint8, device="cuda")
    glq.route(logits.cuda(), top, weights, ids, pos, src, offsets, ws)
    experts = Set(count, n, k, bpw, seed=6, row_scale=row_scale)
    handle = experts.device(cb)
    y = torch.full((tokens + 1, n), 7.0, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y[:tokens], offsets, _workspace(handle, tokens * top), src=src, pos=pos, weights=weights)
    rows = np.nan_to_num(_rows_reference(experts, x.double().cpu().numpy(), offsets.cpu().numpy(), src.cpu().numpy(), tokens * top))
    ref, tol = _combined(rows, pos.cpu().numpy(), weights.double().cpu().numpy(), dtype, k)
    _held(y[:tokens], ref, tol, dtype)
    assert (y[tokens] == 7).all() and (tokens <= 4 or not y[[1, tokens - 1]].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,top,n", [(4700, 8, 8192), (2400, 7, 16384), (300, 64, 5120), (200, 100, 1024)])
def test_many_choices_a_workgroup(cb, dtype, tokens, top, n):
    """More than 64 choices for a workgroup or a set of its waves, whose rows are looked up 64 at a time; some are none."""
    experts, rows = Set(2, n, 128, 2, seed=6, row_scale=True), 90
    handle, x = experts.device(cb), _inputs(3, rows, 128, dtype)
    rng = np.random.default_rng(tokens)
    pos = rng.integers(-1, rows, (tokens, top)).astype(np.int32)
    weights = (rng.random((tokens, top)) / top).astype(np.float32)
    y = torch.empty(tokens, n, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor([0, 31, rows], dtype=torch.int32).cuda(), _workspace(handle, rows),
                      pos=torch.from_numpy(pos).cuda(), weights=torch.from_numpy(weights).cuda())
    each = _rows_reference(experts, x.double().cpu().numpy(), [0, 31, rows], None, rows)
    ref, tol = _combined(each, pos, weights.astype(np.float64), dtype, 128)
    # (the float32 sum of `top` terms has as many roundings more, of 2^-24 of their sizes)
    tol = tol + top * 2.0 ** -24 * np.abs(each).max() * np.abs(weights).sum(1, keepdims=True)
    _held(y, ref, tol, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("k,rows", [(16384, 17000), (8192, 33500)])
def test_long_runs_of_gathered_rows(cb, dtype, k, rows):
    """More than 64 gathered rows a workgroup of the input transform, whose sources are read 64 at a time."""
    experts, tokens = Set(3, 8, k, 2, seed=6), 50
    handle, x = experts.device(cb), _inputs(3, tokens, k, dtype)
    src = np.random.default_rng(k).integers(-1, tokens + 1, rows).astype(np.int32)
    offsets = [0, rows // 3, rows // 3, rows]
    y = torch.empty(rows, 8, device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, rows), src=torch.from_numpy(src).cuda())
    xn = np.concatenate((x.double().cpu().numpy(), np.zeros((1, k))))
    at = np.where((src >= 0) & (src < tokens), src, tokens)
    e = np.where(np.arange(rows) < offsets[1], 0, 2)
    ref = np.stack([experts.reference(i, xn) for i in range(3)])[e, at]
    # (its size by the whole matrix's rows: 8 outputs are too few to take it from)
    size = np.sqrt((xn ** 2).mean(1, keepdims=True))[at] * np.sqrt(k) * experts.scale.max() * np.sqrt(12.0)
    _held(y, ref, _tolerance(np.broadcast_to(size, ref.shape), dtype, k), "f32")


@pytest.mark.gpu
def test_odd_sources_and_positions(cb):
    """Sources outside x are rows of zeros, positions that are no expert's row add nothing, one row serves twice."""
    experts = Set(3, 64, 128, 4)
    handle, x = experts.device(cb), _inputs(5, 6, 128, "f32")
    src = np.array([5, -1, 6, 0, 5, 2 ** 31 - 1, -2 ** 31, 3], np.int32)
    offsets = [1, 3, 3, 7]
    pos = np.array([[1, 2], [3, 3], [0, 7], [-1, 8], [6, 4], [2 ** 31 - 1, -2 ** 31]], np.int32)
    weights = np.random.default_rng(0).random((6, 2)).astype(np.float32)
    y = torch.full((6, 64), 7.0, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (src, pos, weights)]
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, 8), src=dev[0], pos=dev[1],
                      weights=dev[2])
    ref = np.nan_to_num(_rows_reference(experts, x.double().cpu().numpy(), offsets, src, 8))
    ok = (pos >= 1) & (pos < 7)
    each = np.where(ok[..., None], ref[np.clip(pos, 0, 7)], 0.0)
    _held(y, (each * weights[..., None]).sum(1), _tolerance(each, "f32", 128, weights), "f32")
    assert (y[2:4] == 0).all() and (y[5] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("offsets", [[0, 9, 4, 9], [-5, 3, 3, 100], [9, 0, 0, 0], [0, 0, 0, 0], [2 ** 31 - 1] * 4, [-1] * 4])
def test_offsets_out_of_order_or_range(cb, offsets):
    """Such offsets may give any rows their values, but leave what is around them and end."""
    experts = Set(3, 64, 128, 2)
    handle, x = experts.device(cb), _inputs(5, 9, 128, "bf16")
    y = torch.full((11, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    glq.expert_linear(handle, x, y[:9], torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, 9, 0))
    assert torch.isfinite(y).all() and (y[9:] == 7).all()
    if offsets == [-5, 3, 3, 100]:
        ref = _rows_reference(experts, x.double().cpu().numpy(), [0, 3, 3, 9], None, 9)
        _held(y[:9], ref, _tolerance(ref, "bf16", 128), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_that_are_not_finite(cb, dtype, bad):
    """They stay in their rows."""
    experts = Set(2, 64, 128, 3)
    handle, x = experts.device(cb), _inputs(5, 40, 128, dtype)
    ref = _rows_reference(experts, x.double().cpu().numpy(), [0, 17, 40], None, 40)
    x[[3, 39], 5] = bad
    y = torch.empty(40, 64, dtype=DTYPES[dtype], device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor([0, 17, 40], dtype=torch.int32).cuda(), _workspace(handle, 40))
    rows = [r for r in range(40) if r not in (3, 39)]
    _held(y[rows], ref[rows], _tolerance(ref[rows], dtype, 128), dtype)
    assert not torch.isfinite(y[[3, 39]]).any()


@pytest.mark.gpu
def test_no_rows(cb):
    handle = Set(3, 64, 128, 4).device(cb)
    off = torch.zeros(4, dtype=torch.int32).cuda()
    ws = _workspace(handle, 0)
    none = torch.zeros(0, 128, device="cuda")
    glq.expert_linear(handle, none, torch.zeros(0, 64, device="cuda"), off, ws)
    y = torch.full((5, 64), 7.0, device="cuda")
    glq.expert_linear(handle, none, y, off, ws, src=torch.zeros(0, dtype=torch.int32).cuda(),
                      pos=torch.full((5, 2), -1, dtype=torch.int32).cuda(), weights=torch.ones(5, 2, device="cuda"))
    assert (y == 0).all()


@pytest.mark.gpu
def test_agrees_with_single_layers(cb):
    """Experts stacked from layers give what glq_fused_linear gives for each (another order of sums)."""
    experts = Set(3, 256, 512, 3)
    layers = [glq.Layer.from_numpy(experts.idx1[e], experts.idx2[e], experts.scale[e], experts.sign_n[e], experts.sign_k[e], cb)
              for e in range(3)]
    handle, x, offsets = glq.Experts.stack(layers), _inputs(1, 60, 512, "f32"), [0, 20, 21, 60]
    y, one = torch.empty(60, 256, device="cuda"), torch.empty(60, 256, device="cuda")
    glq.expert_linear(handle, x, y, torch.tensor(offsets, dtype=torch.int32).cuda(), _workspace(handle, 60))
    for e, layer in enumerate(layers):
        part = slice(offsets[e], offsets[e + 1])
        ws = torch.zeros(glq.workspace_bytes(layer, 60), dtype=torch.uint8, device="cuda")
        one[part] = glq.fused_linear(layer, x[part].contiguous(), one[part].contiguous(), ws)
    size = one.double().pow(2).mean(1, keepdim=True).sqrt()
    tol = 2 * 6 / np.sqrt(3) * np.sqrt(3 * 512 + 28) * 2.0 ** -24
    assert ((y.double() - one.double()).abs() <= tol * size).all()


# ------------------------------------------------- refusals (nothing is launched)

def _experts_struct(**change):
    st = glq.ExpertsStruct(4, 64, 128, 4, 2, 4096, 4096, 4096, 4096, 4096, 4096, 0)
    for name, value in change.items():
        setattr(st, name, value)
    return ctypes.byref(st)


def _rows_struct(**change):
    st = glq.ExpertRowsStruct(4096, 8192, 1, 1, 10, 20, 4096, 4096, 4096, 4096, 5, 4)
    for name, value in change.items():
        setattr(st, name, value)
    return ctypes.byref(st)


@pytest.mark.parametrize("change,status", [
    ({"count": 0}, -1), ({"n": 0}, -1), ({"n": 60}, -1), ({"k": 4}, -1), ({"k": 132}, -1), ({"bpw": 5}, -1),
    ({"resid_shift": 1}, -1), ({"scale": 0}, -1), ({"idx1": 0}, -1), ({"idx2": 0}, -1), ({"sign_k": 0}, -1), ({"sign_n": 0}, -1),
    ({"cb": 0}, -1), ({"scale": 4098}, -1), ({"row_scale": 4098}, -1), ({"idx1": 4104}, -1), ({"idx2": 4104}, -1),
    ({"sign_k": 4100}, -1), ({"sign_n": 4100}, -1), ({"cb": 4100}, -1), ({"count": 1025}, -2), ({"k": 32768}, -2),
    ({"n": 32768}, -2), ({"n": 1 << 25}, -2)])
def test_experts_refusals(change, status):
    lib, st = glq.raw(), _experts_struct(**change)
    assert lib.glq_expert_linear(st, _rows_struct(), 4096, 1 << 40, None) == status
    assert lib.glq_expert_linear_workspace(st, 20) == 0


@pytest.mark.parametrize("change,status", [
    ({"x_dt": 2}, -1), ({"y_dt": -1}, -1), ({"rows": -1}, -1), ({"x_rows": -1}, -1), ({"tokens": -1}, -1), ({"top_k": 0}, -1),
    ({"weights": 0}, -1), ({"weights": 4098}, -1), ({"pos": 4098}, -1), ({"src": 4098}, -1), ({"src": 0}, -1), ({"y": 0}, -1),
    ({"y": 8200}, -1), ({"x": 0}, -1), ({"x": 4104}, -1), ({"offsets": 0}, -1), ({"offsets": 4098}, -1), ({"rows": 1 << 23}, -2),
    ({"tokens": 1 << 23}, -2), ({"x_rows": 1 << 32}, -2), ({"top_k": 2000}, -2), ({"tokens": 0}, 0),
    ({"pos": 0, "rows": 0}, 0)])
def test_rows_refusals(change, status):
    assert glq.raw().glq_expert_linear(_experts_struct(), _rows_struct(**change), 4096, 1 << 40, None) == status


def test_workspace_refusals():
    lib, st = glq.raw(), _experts_struct()
    need = lib.glq_expert_linear_workspace(st, 20)
    assert need > 0 and lib.glq_expert_linear_workspace(st, -1) == 0
    assert lib.glq_expert_linear(st, _rows_struct(), 0, need, None) == -4
    assert lib.glq_expert_linear(st, _rows_struct(), 4100, need, None) == -4
    assert lib.glq_expert_linear(st, _rows_struct(), 4096, need - 1, None) == -4
    assert lib.glq_expert_linear(None, _rows_struct(), 4096, need, None) == -1
    assert lib.glq_expert_linear(st, None, 4096, need, None) == -1
    assert all(lib.glq_expert_linear_workspace(st, r) >= lib.glq_expert_linear_workspace(st, r - 1) for r in range(1, 700))


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError):
        glq.Experts(1, 8, 8, 2, torch.ones(1), torch.zeros(1, 8, 1, dtype=torch.int16), None, torch.ones(1, 8, dtype=torch.int8),
                    torch.ones(1, 8, dtype=torch.int8), torch.zeros(1 << 20, dtype=torch.uint8))
