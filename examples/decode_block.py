"""One transformer block of a decode step on the library's calls alone.

    h    = rms_norm(x += delta)                  moe_rmsnorm
    qkv  = W_qkv h (+ the request's adapter)     moe_lora_project
    rotate q, k; k, v into the paged cache       moe_kv_append
    a    = attention of q over the cache         moe_attn_decode
    o    = W_o a (+ the request's adapter)       moe_lora_project
    h    = rms_norm(x += o)                      moe_rmsnorm
    y    = MoE layer of h                        moe_layer_forward / deamoe_layer_forward

``x`` is the residual stream (fp32, one row per request); ``delta`` is what the
block before this one adds to it, and ``y`` what the next one will.  All
buffers are the block's own, so that a step can be captured in a CUDA graph.

With ``keep`` pages the heads of q and k are normed, and attention reads that many pages of a
request per key-value head, those that its query can score highest in:

    norm and rotate q, k; k, v into the cache    moe_qk_norm_append
    bounds of the page just written to           moe_page_bounds
    what q can score in each page                moe_page_scores
    the first, the last two and the best ones    moe_page_select
    a    = attention of q over these             moe_attn_pages

    python examples/decode_block.py [--requests 16] [--context 2048] [--steps 32] [--cache e4m3] [--keep 32]

runs the block of the 2048-wide DeaMoE layer on random weights, captured once
and replayed, and prints the time of a step.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_decode_layer_fp32_gb300 import binding as B  # noqa: E402
from moe_decode_layer_fp32_gb300 import synth  # noqa: E402

EPS = 1e-5


class DecodeBlock:
    """Weights, cache, workspaces and buffers of one block for ``requests``
    requests of up to ``max_len`` tokens; ``keep``: pages that attention reads (0: all)."""

    def __init__(self, shape: synth.LayerShape, requests: int, max_len: int, heads: int, kv_heads: int,
                 head_dim: int, page: int = 16, adapters: int = 4, rank: int = 16, cache: str = "bf16",
                 seed: int = 0, device="cuda", keep: int = 0):
        self.shape, self.heads, self.kv_heads, self.head_dim = shape, heads, kv_heads, head_dim
        T, d, D = requests, shape.d, head_dim
        wide = (heads + 2 * kv_heads) * D
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*size, std=1.0, dtype=torch.bfloat16):
            return (torch.randn(size, generator=g, device=device) * std).to(dtype)

        self.norm1, self.norm2 = normal(d, std=0.1) + 1, normal(d, std=0.1) + 1
        self.w_qkv, self.w_o = normal(wide, d, std=0.02), normal(d, heads * D, std=0.02)
        self.lora_qkv = (normal(adapters, rank, d, std=0.02), normal(adapters, wide, rank, std=0.02),
                         torch.ones(adapters, device=device))
        self.lora_o = (normal(adapters, rank, heads * D, std=0.02), normal(adapters, d, rank, std=0.02),
                       torch.ones(adapters, device=device))
        self.layer = synth.make_layer(shape, seed, device)

        half = D // 2
        freq = 10000.0 ** (-torch.arange(half, device=device, dtype=torch.float64) / half)
        angle = torch.arange(max_len, device=device, dtype=torch.float64)[:, None] * freq
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], dim=1).float()

        per = -(-max_len // page)
        e4m3 = cache == "e4m3"
        kv = [torch.zeros(T * per, page, kv_heads, D, device=device,
                          dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16) for _ in range(2)]
        scale = torch.full((kv_heads,), 8.0 / 448, device=device) if e4m3 else None
        self.cache = B.KvCache(kv[0], kv[1], scale, scale)
        # the pages of a request lie anywhere in the cache
        self.block_table = torch.randperm(T * per, generator=g, device=device).to(torch.int32).view(T, per)

        self.ws_qkv, self.ws_o = B.new_lora_workspace(T, d, rank), B.new_lora_workspace(T, heads * D, rank)
        self.ws_attn = B.new_attn_workspace(T, heads, kv_heads, D)
        dept = shape.g if shape.I_sh > 0 else 1
        self.ws_moe = B.new_workspace(T, shape.n, shape.k, dept, device)

        def buffer(*size, dtype=torch.bfloat16):
            return torch.empty(size, dtype=dtype, device=device)

        self.h1, self.qkv, self.attn = buffer(T, d), buffer(T, wide), buffer(T, heads, D)
        self.o, self.h2, self.y = (buffer(T, d, dtype=torch.float32) for _ in range(3))
        self.topk_idx = buffer(T, shape.k, dtype=torch.int32)
        self.topk_w = buffer(T, shape.k, dtype=torch.float32)
        self.keep, self.page = keep, page
        if keep:
            self.q_norm, self.k_norm = normal(D, std=0.1) + 1, normal(D, std=0.1) + 1
            self.bounds = B.new_page_bounds(self.cache)
            self.scores = buffer(T, kv_heads, per, dtype=torch.float32)
            self.tables, self.lens = buffer(T, kv_heads, keep, dtype=torch.int32), buffer(T, kv_heads, dtype=torch.int32)

    def prompt(self, seq_lens):
        """The first ``seq_lens`` (int32 [T]) tokens of each request have been written to the cache."""
        if self.keep:
            B.moe_page_bounds(self.cache, self.bounds, self.block_table, seq_lens)

    def step(self, delta, x, positions, seq_lens, adapter):
        """One new token per request: ``delta`` and ``x`` float32 [T, d] (x is
        updated), ``positions`` and ``seq_lens`` = positions + 1 int32 [T],
        ``adapter`` int32 [T] (-1: none).  Returns y, float32 [T, d]."""
        H, KV, D = self.heads, self.kv_heads, self.head_dim
        B.moe_rmsnorm(delta, self.norm1, EPS, self.h1, residual=x, residual_out=x)
        B.moe_lora_project(self.h1, self.w_qkv, self.qkv, self.ws_qkv, lora=self.lora_qkv, adapter=adapter)
        heads = self.qkv.view(-1, H + 2 * KV, D)
        q, k, v = heads[:, :H], heads[:, H:H + KV], heads[:, H + KV:]
        if self.keep:
            B.moe_qk_norm_append(q, k, v, self.q_norm, self.k_norm, EPS, self.cache, self.block_table, positions, q,
                                 cos_sin=self.cos_sin)
            B.moe_page_bounds(self.cache, self.bounds, self.block_table, seq_lens, first=positions)
            B.moe_page_scores(q, self.cache, self.bounds, self.block_table, seq_lens, self.scores)
            B.moe_page_select(self.scores, self.block_table, seq_lens, self.page, self.tables, self.lens,
                              sinks=min(1, self.keep - 1), recent=min(2, self.keep))
            B.moe_attn_pages(q, self.cache, self.tables, self.lens, D ** -0.5, self.attn, self.ws_attn)
        else:
            B.moe_kv_append(k, v, self.cache, self.block_table, positions, cos_sin=self.cos_sin, q=q, q_out=q)
            B.moe_attn_decode(q, self.cache, self.block_table, seq_lens, D ** -0.5, self.attn, self.ws_attn)
        B.moe_lora_project(self.attn.view(-1, H * D), self.w_o, self.o, self.ws_o, lora=self.lora_o, adapter=adapter)
        B.moe_rmsnorm(self.o, self.norm2, EPS, self.h2, residual=x, residual_out=x)
        s, L = self.shape, self.layer
        shared = (L["sgate"], L["sup"], L["sdown"]) if s.I_s else None
        if s.I_sh > 0:
            private = (L["pgate"], L["pup"], L["pdown"]) if s.I_pr else None
            B.deamoe_layer_forward(self.h2, s.k, 1.0, L["router"], L["bias"], s.g, (L["dgate"], L["dup"], L["ddown"]),
                                   private, shared, self.ws_moe, self.topk_idx, self.topk_w, self.y)
        else:
            B.moe_layer_forward(self.h2, s.k, 1.0, L["router"], L["bias"], L["gate"], L["up"], L["down"], shared,
                                self.ws_moe, self.topk_idx, self.topk_w, self.y)
        return self.y

    def status(self) -> int:
        """First device-side error of any of the block's workspaces (0: none); synchronises."""
        return next((s for s in (B.moe_read_status(w)[0] for w in
                                 (self.ws_qkv, self.ws_attn, self.ws_o, self.ws_moe)) if s), 0)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--context", type=int, default=2048, help="tokens already in each request's cache")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--keep", type=int, default=0, help="pages that attention reads of a request (0: all)")
    a = ap.parse_args()
    T, shape = a.requests, synth.DEAMOE_7B
    block = DecodeBlock(shape, T, a.context + a.steps + 8, heads=16, kv_heads=4, head_dim=128, cache=a.cache,
                        keep=a.keep)
    x, delta = torch.zeros(T, shape.d, device="cuda"), synth.hidden(T, shape.d, 1, "cuda")
    positions = torch.full((T,), a.context, dtype=torch.int32, device="cuda")
    seq_lens = positions + 1
    adapter = torch.tensor([t % 5 - 1 for t in range(T)], dtype=torch.int32, device="cuda")
    block.prompt(positions)
    block.step(delta, x, positions, seq_lens, adapter)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.step(delta, x, positions, seq_lens, adapter)
        positions += 1
        seq_lens += 1
    x.zero_()
    positions.fill_(a.context)
    seq_lens.fill_(a.context + 1)
    first, last = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == 2:
            first.record()
        graph.replay()
    last.record()
    torch.cuda.synchronize()
    status = block.status()
    if status:
        raise SystemExit(f"device status {status}")
    us = first.elapsed_time(last) * 1e3 / max(1, a.steps - 2)
    kept = f", {a.keep} pages of each" if a.keep else ""
    print(f"{T} requests of {a.context} tokens, {a.cache} cache{kept}: {us:.1f} us a block step "
          f"({us / T:.2f} us a token), |y| = {block.y.norm().item():.4g}")


if __name__ == "__main__":
    main()
