"""The attention half of a joint video/audio block, from the modulated rows to the gated residual.

Two samples of one prompt are packed one after the other; every row attends to the prompt's states (stored once, shared
by the samples) and to all rows of its own sample, and its queries to a second encoder's states as well:

    qkv   = NVFP4 linear of the modulated rows                    h3fp4_linear
    q, k  = per-head norm and rotation, in place on qkv's views    h3fp4_qk_norm_rope
    attn  = attention over the shared prompt and the sample        h3fp4_shared_attn
    x     = x + gate * (NVFP4 linear of attn)                      h3fp4_linear
    cross = attention of the rows to other states                  h3fp4_cross_attn

Run on a GB300:  python examples/attention_block.py
Everything the calls need is allocated before the first step, so the steps can be captured into a CUDA graph.
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import audio_dit_gb300 as A


class AttentionBlock:
    """Weights, buffers and workspaces of one block for packed samples of fixed lengths."""

    def __init__(self, rows, prompt, other, heads=24, dim=128, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
        self.heads, self.dim, self.width = heads, dim, heads * dim
        self.off = [0]
        for n in rows:
            self.off.append(self.off[-1] + n)
        self.M, K = self.off[-1], self.width
        self.one = [0, self.M]
        self.w, self.bias = {}, {}
        for name, n in (("qkv", 3 * K), ("out", K)):
            self.w[name] = A.alloc_nvfp4(n, K)
            A.h3fp4_quantize_weight(rn(n, K, std=0.02).bfloat16(), *self.w[name], A.alloc_workspace(n, 0, K))
            self.bias[name] = rn(n, std=0.01).bfloat16()
        self.shift, self.scale, self.gate = rn(1, K, std=0.1), rn(1, K, std=0.1), rn(1, K, std=0.1) + 0.5
        self.q_weight, self.k_weight = 1 + rn(1, dim, std=0.1), 1 + rn(1, dim, std=0.1)
        # three position axes, dealt out over the pairs of a head
        pos = torch.stack([torch.arange(self.M, device="cuda") // s % 64 for s in (1, 64, 4096)], 1).float()
        freq = 10000.0 ** (-torch.arange(dim // 2, device="cuda").float() / (dim // 2))
        angle = pos[:, torch.arange(dim // 2, device="cuda") % 3] * freq
        self.cos, self.sin = torch.cos(angle).contiguous(), torch.sin(angle).contiguous()
        bf = lambda n: rn(n, heads, dim).bfloat16()  # noqa: E731
        self.k_ctx, self.v_ctx = bf(prompt), bf(prompt)
        self.k_other, self.v_other = bf(other), bf(other)
        self.ctx_mask = torch.arange(prompt, device="cuda") < prompt - prompt // 4     # a padded prompt
        self.x = rn(self.M, K).bfloat16()
        self.qkv = torch.empty(self.M, 3 * K, dtype=torch.bfloat16, device="cuda")
        self.attn, self.y, self.cross = (torch.empty(self.M, K, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.ws = A.alloc_workspace(self.M, 3 * K, K)
        self.ws_attn = A.alloc_attn_workspace(self.M, self.M, heads, heads, dim, q_off=self.off, kv_off=self.off,
                                              ctx=prompt)
        self.ws_cross = A.alloc_attn_workspace(self.M, other, heads, heads, dim)

    def views(self):
        """Q, K and V as strided views of the projection's output."""
        v = self.qkv.view(self.M, 3, self.heads, self.dim)
        return v[:, 0], v[:, 1], v[:, 2]

    def step(self):
        h = lambda t: t.view(self.M, self.heads, self.dim)  # noqa: E731
        q, k, v = self.views()
        A.h3fp4_linear(self.x, *self.w["qkv"], self.qkv, self.ws, shift=self.shift, scale=self.scale,
                       bias=self.bias["qkv"], seg_off=self.one)
        A.h3fp4_qk_norm_rope(q, k, q, k, q_weight=self.q_weight, k_weight=self.k_weight, cos=self.cos, sin=self.sin)
        A.h3fp4_shared_attn(q, k, v, self.k_ctx, self.v_ctx, h(self.attn), self.ws_attn, q_off=self.off,
                            kv_off=self.off, ctx_mask=self.ctx_mask)
        A.h3fp4_linear(self.attn, *self.w["out"], self.y, self.ws, bias=self.bias["out"], gate=self.gate,
                       resid=self.x, seg_off=self.one)
        A.h3fp4_cross_attn(q, self.k_other, self.v_other, h(self.cross), self.ws_cross)

    def check(self):
        for ws in (self.ws, self.ws_attn, self.ws_cross):
            A.h3fp4_check(ws)


def main():
    block = AttentionBlock(rows=[4096, 4096], prompt=512, other=300)
    for _ in range(3):
        block.step()
    block.check()
    t = time.perf_counter()
    for _ in range(20):
        block.step()
    block.check()
    ms = (time.perf_counter() - t) / 20 * 1e3
    print(f"attention half of a block, {block.M} rows, {block.heads} heads of {block.dim}: {ms:.3f} ms")


if __name__ == "__main__":
    main()
