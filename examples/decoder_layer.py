"""One decoder layer served with the package: attention over a paged cache, then the MoE layer.

    python examples/decoder_layer.py

A step takes the hidden states of some sequences' new tokens (whole prompts, chunks of them, single tokens, or all of
these together) and runs

    norm                                  add_rms_norm         (one launch)
    qkv projection                        torch matmul
    norm + rotation of q and k, append    PagedKV.append       (one launch)
    attention over the pages              PagedKV.attend       (one launch)
    output projection                     torch matmul
    residual + norm, in 16 bits for the   add_rms_norm         (one launch)
      router and in MXFP8 for the experts
    routing + experts, residual           MoeLayer             (MXFP4 weights, MXFP8 tokens)

The cache holds 16 bits an element, or 8 (PagedKV8).  The script prefills two prompts of different lengths, decodes a few
tokens of each, and compares the decoded tokens' hidden states with those of one prefill of everything.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_weight_moe_gb300 as kt                       # noqa: E402
from mxfp4_weight_moe_gb300 import synthetic as syn        # noqa: E402


class Pages:
    """Hands out cache pages to sequences and describes a step's batch."""

    def __init__(self, num_pages: int, page_size: int, device):
        self.free, self.page_size, self.device = list(range(num_pages)), page_size, device
        self.pages, self.length = [], []

    def add_sequence(self) -> int:
        self.pages.append([])
        self.length.append(0)
        return len(self.pages) - 1

    def step(self, new: list[int]):
        """(block_table, cu_q, seq_lens, max_q_len) of a step in which sequence b gets new[b] tokens."""
        for b, n in enumerate(new):
            self.length[b] += n
            while len(self.pages[b]) * self.page_size < self.length[b]:
                self.pages[b].append(self.free.pop())
        width = max(len(p) for p in self.pages)
        table = torch.tensor([p + [-1] * (width - len(p)) for p in self.pages], dtype=torch.int32)
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        lens = torch.tensor(self.length, dtype=torch.int32)
        return tuple(t.to(self.device) for t in (table, cu, lens)) + (max(new),)


class DecoderLayer:
    def __init__(self, hidden: int, q_heads: int, kv_heads: int, head_dim: int, experts: int, top_k: int, inter: int,
                 num_pages: int, page_size: int = 16, max_positions: int = 4096, seed: int = 0, device="cuda",
                 cache_bits: int = 16):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)

        self.hq, self.hk, self.d, self.top_k = q_heads, kv_heads, head_dim, top_k
        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_o = weight(hidden, q_heads * head_dim)
        self.w_router = weight(experts, hidden)
        self.q_norm = torch.ones(head_dim, dtype=torch.bfloat16, device=device)
        self.k_norm = torch.ones(head_dim, dtype=torch.bfloat16, device=device)
        self.rope = kt.rope_table(max_positions, head_dim, device=device)
        self.in_norm, self.out_norm = (torch.ones(hidden, dtype=torch.bfloat16, device=device) for _ in range(2))
        pages = torch.empty(2, num_pages, page_size, kv_heads, head_dim, device=device,
                            dtype=torch.bfloat16 if cache_bits == 16 else torch.float8_e4m3fn)
        if cache_bits == 16:
            self.cache = kt.PagedKV(pages[0], pages[1])
        else:
            scales = torch.empty(2, num_pages, page_size // kt.PagedKV8.BLOCK, kv_heads, dtype=torch.uint8, device=device)
            self.cache = kt.PagedKV8(pages[0], pages[1], scales[0], scales[1], torch.bfloat16)
        packed = [syn.make_expert(e, hidden, inter, seed, device) for e in range(experts)]
        self.moe = kt.MoeLayer(*[torch.stack(t).contiguous() for t in zip(*packed)], top_k)

    def __call__(self, x: torch.Tensor, block_table, cu_q, seq_lens, max_q_len) -> torch.Tensor:
        """x: bf16 [tokens, hidden] of the step; returns the layer's output of the same shape."""
        n = x.shape[0]
        h, _, _ = kt.add_rms_norm(x, self.in_norm)
        qkv = (h @ self.w_qkv.T).view(n, self.hq + 2 * self.hk, self.d)
        q, k, v = qkv.split((self.hq, self.hk, self.hk), dim=1)
        q = self.cache.append(k, v, block_table, cu_q, seq_lens, self.rope, q=q, q_weight=self.q_norm,
                              k_weight=self.k_norm)
        y = self.cache.attend(q, block_table, cu_q, seq_lens, max_q_len)
        h, x, tokens = kt.add_rms_norm(y.view(n, -1) @ self.w_o.T, self.out_norm, x, mx=True)
        out, _, _ = self.moe(tokens, (h @ self.w_router.T).float())
        return x + out


def run(prompts=(37, 150), decode=4, hidden=1024, q_heads=16, kv_heads=2, head_dim=128, experts=16, top_k=4, inter=512,
        seed=0, device="cuda", cache_bits=16):
    """Largest relative difference (per token, by norm) of the decoded tokens between serving and one prefill."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    total = [p + decode for p in prompts]
    layer = DecoderLayer(hidden, q_heads, kv_heads, head_dim, experts, top_k, inter,
                         num_pages=2 * sum(-(-t // 16) for t in total), device=device, cache_bits=cache_bits)
    xs = [torch.randn(t, hidden, generator=g, device=device).to(torch.bfloat16) for t in total]
    pages = Pages(layer.cache.num_pages, layer.cache.page_size, device)
    for _ in prompts:
        pages.add_sequence()
    layer(torch.cat([x[:p] for x, p in zip(xs, prompts)]), *pages.step(list(prompts)))      # prefill
    served = []
    for i in range(decode):                                                                # then token by token
        served.append(layer(torch.stack([x[p + i] for x, p in zip(xs, prompts)]), *pages.step([1] * len(prompts))))
    served = torch.stack(served, dim=1)                                                    # [sequence, token, hidden]
    again = Pages(layer.cache.num_pages, layer.cache.page_size, device)
    again.free = pages.free
    for _ in prompts:
        again.add_sequence()
    whole = layer(torch.cat(xs), *again.step(total)).split(total)
    whole = torch.stack([w[-decode:] for w in whole])
    assert layer.cache.read_error() == 0
    diff = (served.float() - whole.float()).norm(dim=-1) / whole.float().norm(dim=-1)
    return float(diff.max())


if __name__ == "__main__":
    for bits in (16, 8):
        print(f"decoded tokens against one prefill, {bits}-bit cache: largest relative difference "
              f"{run(cache_bits=bits):.2e}")
