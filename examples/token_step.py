"""A stream that is generated token by token: one block's step with its weights and its cache in four bits.

The keys and values of the prompts are made and stored first (many rows: the quantised linear; nothing else of a single block
needs them), then every step takes one token of each sequence through

    h     = norm of x before the attention                          h3fp4_block_norm
    qkv   = linear of the few rows, activations as they are         h3fp4_linear_rows
    q, k  = per-head norm and rotation, in place on qkv's views     h3fp4_qk_norm_rope
    cache <- k, v                                                   h3fp4_cache_append
    attn  = attention to each sequence's cached tokens              h3fp4_cache_attn
    y     = linear of attn                                          h3fp4_linear_rows
    x, h  = x + gate * norm(y), and the norm before the MLP          h3fp4_block_norm
    g     = SwiGLU of the gate and up projections                   h3fp4_linear_rows
    x     = x + gate * (linear of g)                                h3fp4_linear_rows

Lengths and page tables are on the device, so that the whole step is one captured graph, whatever the lengths.

Run on a GB300:  python examples/token_step.py
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import audio_dit_gb300 as A
from audio_dit_gb300.graphs import GraphBuckets


class TokenBlock:
    """Weights, cache and buffers of one block for `seqs` sequences of up to `room` tokens."""

    def __init__(self, seqs, room, heads=32, kv_heads=8, dim=128, hidden=8192, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.seqs, self.heads, self.kv_heads, self.dim = seqs, heads, kv_heads, dim
        self.width = K = heads * dim
        self.w, self.bias = {}, {}
        for name, n, k in (("qkv", (heads + 2 * kv_heads) * dim, K), ("out", K, K), ("up", 2 * hidden, K), ("down", K, hidden)):
            self.w[name] = A.alloc_nvfp4(n, k)
            A.h3fp4_quantize_weight(rn(n, k, std=0.02).bfloat16(), *self.w[name], A.alloc_workspace(n, 0, k))
            self.bias[name] = rn(n, std=0.01).bfloat16()
        self.norm1, self.norm2, self.post = (1 + rn(1, K, std=0.1) for _ in range(3))
        self.gate1, self.gate2 = 0.5 + rn(1, K, std=0.1), 0.5 + rn(K, std=0.1)
        self.q_weight, self.k_weight = 1 + rn(1, dim, std=0.1), 1 + rn(1, dim, std=0.1)
        # angles of every position, looked up by the step's lengths
        angle = torch.arange(room, device="cuda")[:, None] * 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))
        self.all_cos, self.all_sin = torch.cos(angle).float(), torch.sin(angle).float()
        # pages, handed out in the order of the sequences; scales with room above what the norm leaves
        pages = (room + page - 1) // page
        self.cache = A.alloc_kv_cache(seqs * pages, kv_heads, dim, page)
        self.table = torch.arange(seqs * pages, dtype=torch.int32, device="cuda").view(seqs, pages)
        self.length = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.k_gscale = torch.full((kv_heads,), 16.0 / 2688, device="cuda")
        self.v_gscale = torch.full((kv_heads,), 16.0 / 2688, device="cuda")
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.x = rn(seqs, K).bfloat16()
        self.h, self.y, self.attn = bf(seqs, K), bf(seqs, K), bf(seqs, K)
        self.qkv, self.up = bf(seqs, heads + 2 * kv_heads, dim), bf(seqs, hidden)
        self.cos, self.sin = (torch.empty(seqs, dim // 2, device="cuda") for _ in range(2))
        self.ws = {name: A.alloc_rows_workspace(seqs, w[0].shape[0], 2 * w[0].shape[1]) for name, w in self.w.items()}
        self.ws_attn = A.alloc_cache_attn_workspace(seqs, seqs, heads, kv_heads, dim)

    def views(self, qkv):
        return qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv_heads], qkv[:, self.heads + self.kv_heads:]

    def prompt(self, x, lengths):
        """Packed rows x of the sequences' prompts: their keys and values into the cache."""
        M, n = x.shape[0], (self.heads + 2 * self.kv_heads) * self.dim
        h, amax, gs = torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
        qkv = torch.empty(M, self.heads + 2 * self.kv_heads, self.dim, dtype=torch.bfloat16, device="cuda")
        ws = A.alloc_workspace(M, n, self.width)
        A.h3fp4_block_norm(x, h, weight=self.norm1, out_amax=amax)
        A.h3fp4_gscale_from_amax(amax, gs)
        A.h3fp4_linear(h, *self.w["qkv"], qkv.view(M, -1), ws, a_gscale=gs, gscale_given=True, bias=self.bias["qkv"])
        _, k, v = self.views(qkv)
        at = torch.cat([torch.arange(t, device="cuda") for t in lengths])
        A.h3fp4_qk_norm_rope(k, None, k, None, q_weight=self.k_weight, cos=self.all_cos[at], sin=self.all_sin[at])
        self.length.copy_(torch.tensor(lengths, dtype=torch.int32))
        off = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32).cuda()
        A.h3fp4_cache_append(k, v, self.cache, self.table, self.length, off, k_gscale=self.k_gscale, v_gscale=self.v_gscale)
        A.h3fp4_check(ws)

    def step(self, key=None):
        """One token of each sequence: self.x in, self.x out, the lengths one longer."""
        w, ws, b = self.w, self.ws, self.bias
        q, k, v = self.views(self.qkv)
        scales = dict(k_gscale=self.k_gscale, v_gscale=self.v_gscale)
        torch.index_select(self.all_cos, 0, self.length, out=self.cos)
        torch.index_select(self.all_sin, 0, self.length, out=self.sin)
        self.length.add_(1)
        A.h3fp4_block_norm(self.x, self.h, weight=self.norm1)
        A.h3fp4_linear_rows(self.h, *w["qkv"], self.qkv.view(self.seqs, -1), ws["qkv"], bias=b["qkv"])
        A.h3fp4_qk_norm_rope(q, k, q, k, q_weight=self.q_weight, k_weight=self.k_weight, cos=self.cos, sin=self.sin)
        A.h3fp4_cache_append(k, v, self.cache, self.table, self.length, **scales)
        A.h3fp4_cache_attn(q, self.cache, self.table, self.length, self.attn.view(self.seqs, self.heads, self.dim),
                           self.ws_attn, **scales)
        A.h3fp4_linear_rows(self.attn, *w["out"], self.y, ws["out"], bias=b["out"])
        A.h3fp4_block_norm(self.x, self.h, y=self.y, x_out=self.x, gate=self.gate1, post_norm=True, y_weight=self.post,
                           weight=self.norm2)
        A.h3fp4_linear_rows(self.h, *w["up"], self.up, ws["up"], bias=b["up"], swiglu=True)
        A.h3fp4_linear_rows(self.up, *w["down"], self.x, ws["down"], bias=b["down"], gate=self.gate2, resid=self.x)

    def check(self):
        for ws in (*self.ws.values(), self.ws_attn):
            A.h3fp4_check(ws)


def main():
    lengths = [700, 64, 1999, 1300]
    block = TokenBlock(len(lengths), 4096)
    block.prompt(torch.randn(sum(lengths), block.width, device="cuda").bfloat16(), lengths)
    graphs = GraphBuckets(block.step)          # (the capture's warm-up is a step too)
    for _ in range(10):
        graphs.run(len(lengths))
    block.check()
    t = time.perf_counter()
    for _ in range(200):
        graphs.run(len(lengths))
    block.check()
    us = (time.perf_counter() - t) / 200 * 1e6
    print(f"one block's step for {len(lengths)} sequences of {block.length.tolist()} tokens: {us:.1f} us")


if __name__ == "__main__":
    main()
