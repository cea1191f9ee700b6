"""A decoder block of a grouped-query model on the library: one step of a batch whose sequences
share a prefix, from the residual stream through attention and the MoE expert layer back to it.

    residual += y                              lily_attn_add_rmsnorm (8-bit rows with scales)
    q, k, v = rows @ w_qkv                     the caller's projection, here a plain product of
                                               the rows taken back to bf16; an 8-bit one would
                                               take codes and scales as they are
    rotate q and k, append k and v             lily_attn_rope_append
    attention                                  lily_attn_shared_prefix
    residual += heads @ w_o                    lily_attn_add_rmsnorm (bf16 rows)
    y = experts(rows)                          lily_moe_decode (up to 8 rows) / lily_moe_forward

    python examples/decoder_block.py           # on a GB300: a prefix, then some decode steps

Weights are random; nothing is allocated between steps."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4_grouped_gemm_gb300 as lily  # noqa: E402
from w4_grouped_gemm_gb300 import synth  # noqa: E402

EPS = 1e-6


class DecoderBlock:
    """Weights and caches of one block for `seqs` sequences of up to `own` tokens each behind a
    prefix of `prefix` tokens that they share.  Steps of `q_len` new tokens per sequence."""

    def __init__(self, d=512, hq=8, hkv=2, D=64, rot=64, experts=32, top_k=4, ff=128, seqs=4,
                 q_len=1, prefix=100, own=64, page=16, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        bf = dict(dtype=torch.bfloat16, device=device)
        self.d, self.hq, self.hkv, self.D, self.rot, self.page = d, hq, hkv, D, rot, page
        self.seqs, self.q_len, self.prefix, self.own = seqs, q_len, prefix, own
        T = self.T = seqs * q_len
        width = (hq + 2 * hkv) * D
        self.w_qkv = (rnd(d, width) * d ** -0.5).to(torch.bfloat16)
        self.w_o = (rnd(hq * D, d) * (hq * D) ** -0.5).to(torch.bfloat16)
        self.norm1, self.norm2 = 1 + 0.1 * rnd(d), 1 + 0.1 * rnd(d)
        layer = synth.make_layer(synth.LayerShape(T=T, d=d, E=experts, k=top_k, F=ff), seed=seed + 1,
                                 device=device)
        self.moe_w = lily.LayerWeights(layer["router_w"], layer["router_b"], layer["experts"])
        self.moe_w.split_router()
        self.moe_dims = lily.make_dims(T, d, experts, top_k, ff, 32)
        self.routing = lily.RoutingBuffers(self.moe_dims, device)
        self.moe_ws = lily.alloc_workspace(lily.lily_moe_workspace_bytes(self.moe_dims), device)

        # the cache: the prefix's pages, then each sequence's own
        shared, each = -(-prefix // page), -(-own // page)
        k = torch.zeros(shared + each * seqs, page, hkv, D, **bf)
        self.cache = lily.PagedCache(k, torch.zeros_like(k))
        pages = torch.arange(shared + each * seqs, dtype=torch.int32, device=device)
        self.prefix_pages = pages[:shared].clone()
        self.table = pages[shared:].view(seqs, each).contiguous()
        self.seq_lens = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.inv_freq = 1e6 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)

        # buffers of a step
        self.h8 = torch.empty(T, d, dtype=torch.float8_e4m3fn, device=device)
        self.scales = torch.empty(T, 1, device=device)
        self.qkv = torch.empty(T, width, **bf)
        self.heads = torch.empty(T, hq, D, **bf)
        self.lse = torch.empty(T, hq, device=device)
        self.proj = torch.empty(T, d, **bf)
        self.x = torch.empty(T, d, **bf)
        self.y = torch.zeros(T, d, dtype=torch.float32, device=device)
        q, kk, v = self.split(self.qkv)
        f32, b16 = torch.float32, torch.bfloat16
        self.dims8 = lily.make_norm_dims(T, d, f32, f32, f32, torch.float8_e4m3fn, eps=EPS)
        self.dims16 = lily.make_norm_dims(T, d, b16, f32, f32, b16, eps=EPS)
        self.rope_dims = lily.make_rope_dims(q, kk, v, q, rot)  # q turns in place
        self.attn_dims = lily.make_attn_dims(q, self.heads, seqs, q_len, prefix, own,
                                             self.table.shape[1], D ** -0.5)
        self.attn_ws = lily.alloc_workspace(
            lily.lily_attn_workspace_bytes(self.attn_dims, self.cache), device)

    def split(self, qkv):
        """q, k and v as views of the fused projection's rows."""
        T, n, m = qkv.shape[0], self.hq * self.D, self.hkv * self.D
        return (qkv[:, :n].view(T, self.hq, self.D), qkv[:, n:n + m].view(T, self.hkv, self.D),
                qkv[:, n + m:].view(T, self.hkv, self.D))

    def fill_prefix(self, k, v):
        """Append the prefix's keys and values [prefix][hkv][D] (positions 0 ..)."""
        dev = k.device
        at = torch.arange(self.prefix, device=dev)
        slots = self.prefix_pages.long()[at // self.page] * self.page + at % self.page
        lily.lily_attn_rope_append(lily.make_rope_dims(None, k, v, None, self.rot), self.cache, None,
                                   k, v, at.int(), slots, self.inv_freq, None, self.attn_ws)

    def slots_of(self, lens):
        """Where the next q_len tokens of every sequence go, and their positions.  A token past a
        sequence's room goes nowhere (slot -1; its step's attention then sets BAD_LEN)."""
        at = (lens[:, None] + torch.arange(self.q_len, device=lens.device)).long()
        pages = torch.gather(self.table.long(), 1, (at // self.page).clamp(max=self.table.shape[1] - 1))
        slots = torch.where(at < self.own, pages * self.page + at % self.page, -1)
        return slots.view(-1), (at.view(-1) + self.prefix).int()

    def step(self, residual, y):
        """residual [T][d] fp32, updated in place; y [T][d] fp32: what the block before adds to it.
        Returns this block's own y, still to be added."""
        lily.lily_attn_add_rmsnorm(self.dims8, y, residual, self.norm1, residual, self.h8, self.scales)
        rows = (self.h8.float() * self.scales).to(torch.bfloat16)
        torch.mm(rows, self.w_qkv, out=self.qkv)
        q, k, v = self.split(self.qkv)
        slots, positions = self.slots_of(self.seq_lens)
        lily.lily_attn_rope_append(self.rope_dims, self.cache, q, k, v, positions, slots,
                                   self.inv_freq, q, self.attn_ws)
        self.seq_lens += self.q_len
        lily.lily_attn_shared_prefix(self.attn_dims, self.cache, q, self.prefix_pages, None,
                                     self.seq_lens, self.table, self.heads, self.lse, self.attn_ws)
        torch.mm(self.heads.view(self.T, -1), self.w_o, out=self.proj)
        lily.lily_attn_add_rmsnorm(self.dims16, self.proj, residual, self.norm2, residual, self.x)
        run = lily.lily_moe_decode if self.T <= 8 else lily.lily_moe_forward
        run(self.moe_dims, self.x, self.moe_w, self.routing, self.y, self.moe_ws)
        return self.y

    def status(self):
        return lily.lily_moe_status(self.attn_ws) | lily.lily_moe_status(self.moe_ws)


def main():
    block = DecoderBlock(d=2048, hq=16, hkv=2, D=128, rot=128, experts=256, top_k=8, ff=512, seqs=8,
                         prefix=4096, own=256, page=64)
    gen = torch.Generator(device="cuda").manual_seed(7)
    kv = torch.randn(2, block.prefix, block.hkv, block.D, generator=gen, device="cuda").bfloat16()
    block.fill_prefix(kv[0], kv[1])
    residual = torch.randn(block.T, block.d, generator=gen, device="cuda")
    y = torch.zeros_like(residual)
    for _ in range(3):
        y = block.step(residual, y)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    steps = 100
    for _ in range(steps):
        y = block.step(residual, y)
    b.record()
    torch.cuda.synchronize()
    assert block.status() == 0 and bool(torch.isfinite(y).all())
    print(f"{block.seqs} sequences behind {block.prefix} shared tokens: "
          f"{a.elapsed_time(b) * 1e3 / steps:.1f} us per block and step")


if __name__ == "__main__":
    main()
