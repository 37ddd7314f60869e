"""A compressed attention block serving one user: prompt in chunks, then tokens.

The q/k/v and output projections are compressed linears (glq_fused_linear), the
keys and values live in a paged 8-bit or 4-bit cache, rotated along the head dimension
before they are written (glq_rht_apply; queries and keys get the same rotation,
so their scores do not change, and outlier channels spread over the codes).

  prompt chunk   projections -> rotate -> glq_kv_append -> glq_kv_read of what
                 is cached -> glq_attn_prompt -> output projection
  next token     projections -> rotate -> glq_kv_append -> glq_attn_decode ->
                 output projection

Run on an MI355X:  python examples/attention_block.py [--cache int4] [--tokens 8]
It prints how far the outputs are from the same block in float64 on the dense weights.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dequant_e8_codebook_amd import glq  # noqa: E402


class Linear:
    """One compressed linear and its workspace."""

    def __init__(self, n, k, bpw, rng, codebook, rows):
        signs = [rng.integers(0, 2, m).astype(np.int8) * 2 - 1 for m in (n, k)]
        w = rng.standard_normal((n, k)).astype(np.float32) / np.sqrt(k)
        i1, i2, scale = glq.encode_ref(w, bpw, *signs)
        self.layer = glq.Layer.from_numpy(i1, i2, scale, *signs, codebook)
        self.ws = torch.zeros(glq.workspace_bytes(self.layer, rows), dtype=torch.uint8, device="cuda")

    def __call__(self, x):
        y = torch.empty(x.shape[0], self.layer.n, dtype=x.dtype, device=x.device)
        return glq.fused_linear(self.layer, x, y, self.ws)

    def dense(self):
        """The weights in the original basis, float64: what the layer multiplies by."""
        eye = torch.eye(self.layer.k, device="cuda")
        ws = torch.zeros(glq.workspace_bytes(self.layer, self.layer.k), dtype=torch.uint8, device="cuda")
        y = torch.empty(self.layer.k, self.layer.n, device="cuda")
        return glq.fused_linear(self.layer, eye, y, ws).double().T.cpu()


class Block:
    def __init__(self, hidden, heads, kv_heads, dim, cache_format, max_tokens, bpw=4, page=32, seed=0):
        rng = np.random.default_rng(seed)
        cb = glq.device_codebook()
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.qkv = Linear((heads + 2 * kv_heads) * dim, hidden, bpw, rng, cb, max_tokens)
        self.out = Linear(hidden, heads * dim, bpw, rng, cb, max_tokens)
        self.signs = torch.from_numpy(rng.integers(0, 2, dim).astype(np.int8) * 2 - 1).cuda()
        pages = -(-max_tokens // page)
        self.page, self.cache = page, glq.KvCache.empty(pages + 3, page, kv_heads, dim, cache_format)
        # the user's pages, wherever they were free
        self.table = torch.from_numpy(rng.permutation(pages + 3)[:pages].astype(np.int32)).cuda()[None]
        self.ws = torch.zeros(glq.attn_decode_workspace_bytes(self.cache, 1, heads, max_tokens), dtype=torch.uint8,
                              device="cuda")
        self.max_tokens, self.length = max_tokens, 0

    def _slots(self, first, count):
        t = torch.arange(first, first + count, device="cuda")
        return (self.table[0].long()[t // self.page] * self.page + t % self.page).to(torch.int32)

    def _project(self, x):
        """Rotated queries and keys, and values, of new tokens; keys and values cached."""
        parts = self.qkv(x).view(x.shape[0], -1, self.dim).split((self.heads, self.kv_heads, self.kv_heads), 1)
        q, k = (p.contiguous() for p in parts[:2])
        for p in (q, k):
            glq.rht_apply(p, p, self.signs, False)
        glq.kv_append(self.cache, k, parts[2], self._slots(self.length, x.shape[0]))
        self.length += x.shape[0]
        return q

    def prompt(self, x):
        """The next tokens of the prompt, [tokens, hidden]."""
        q = self._project(x)
        k, v = (torch.empty(self.length, self.kv_heads, self.dim, dtype=x.dtype, device="cuda") for _ in range(2))
        glq.kv_read(self.cache, self._slots(0, self.length), k, v)
        cu = torch.tensor([[0, x.shape[0]], [0, self.length]], dtype=torch.int32, device="cuda")
        o = glq.attn_prompt(q, k, v, torch.empty_like(q), cu[0], cu[1], max_q=x.shape[0])
        return self.out(o.flatten(1))

    def token(self, x):
        """One new token, [1, hidden]."""
        q = self._project(x)
        lens = torch.tensor([self.length], dtype=torch.int32, device="cuda")
        o = glq.attn_decode(self.cache, q, self.table, lens, torch.empty_like(q), self.ws, self.max_tokens)
        return self.out(o.flatten(1))

    def reference(self, x):
        """All tokens at once in float64 on the dense weights, nothing quantised."""
        x = x.double().cpu()
        n, d, g = x.shape[0], self.dim, self.heads // self.kv_heads
        q, k, v = (x @ self.qkv.dense().T).view(n, -1, d).split((self.heads, self.kv_heads, self.kv_heads), 1)
        k, v = (t.repeat_interleave(g, 1).transpose(0, 1) for t in (k, v))
        s = q.transpose(0, 1) @ k.transpose(1, 2) * d ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool).triu(1), -torch.inf)
        return (torch.softmax(s, -1) @ v).transpose(0, 1).reshape(n, -1) @ self.out.dense().T


def run(cache="int8", tokens=8, chunks=(75, 40), hidden=512, heads=8, kv_heads=2, dim=64, seed=0):
    """Chunks of a prompt, then single tokens. Returns the relative error (2-norm) of
    the prompt's and of the tokens' outputs against the float64 block."""
    fmt = {"bf16": glq.KV_BF16, "int8": glq.KV_INT8, "int4": glq.KV_INT4}[cache]
    total = sum(chunks) + tokens
    block = Block(hidden, heads, kv_heads, dim, fmt, total, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x = torch.randn(total, hidden, generator=gen).to(torch.bfloat16).cuda()
    got, at = [], 0
    for n in chunks:
        got.append(block.prompt(x[at:at + n]))
        at += n
    for t in range(at, total):
        got.append(block.token(x[t:t + 1]))
    ref, y = block.reference(x), torch.cat(got).double().cpu()
    err = [((y[s] - ref[s]).norm() / ref[s].norm()).item() for s in (slice(0, at), slice(at, total))]
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--cache", choices=("bf16", "int8", "int4"), default="int8")
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    prompt, tokens = run(a.cache, a.tokens)
    print(f"{a.cache} cache: relative error of the prompt's outputs {prompt:.4f}, of the new tokens' {tokens:.4f}")
