"""A small decoder on the library, from a batch's tokens to its next ones: 4-bit projections, an
8-bit paged cache, MoE experts, and sampling.

    residual += y                              lily_attn_add_rmsnorm (bf16 rows)
    q, k, v = rows W_qkv^T                     lily_decode_linear (4-bit weights)
    rotate q and k, append k and v in 8 bits   lily_attn_rope_append8
    attention                                  lily_attn_decode8
    heads W_o^T                                lily_decode_linear
    residual += that                           lily_attn_add_rmsnorm
    y = experts(rows)                          lily_moe_decode (up to 8 rows) / lily_moe_forward
    ... and after the last block
    logits = rows W_head^T                     lily_attn_add_rmsnorm, lily_decode_linear
    the next tokens                            lily_decode_sample

    python examples/token_step.py              # on a GB300: some tokens, eager and from a graph

Weights are random; a step is captured into a CUDA graph as it is."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4_grouped_gemm_gb300 as lily  # noqa: E402
from w4_grouped_gemm_gb300 import synth  # noqa: E402

EPS = 1e-6
BF, F32 = torch.bfloat16, torch.float32


def quantised4(w, group=64, symmetric=False):
    """w [N][K] as 4-bit codes with a scale, and unless symmetric a bias, for each group."""
    N, K = w.shape
    g = w.float().view(N, K // group, group)
    if symmetric:
        scale, bias = (g.abs().amax(-1) / 7.5).to(BF), None
        low = -8 * scale.float()
    else:
        low = g.amin(-1)
        scale, bias = ((g.amax(-1) - low) / 15).to(BF), low.to(BF)
        low = bias.float()
    step = torch.where(scale > 0, scale.float(), 1.0)
    q = ((g - low[..., None]) / step[..., None]).round().clamp(0, 15).to(torch.uint8).view(N, K)
    return lily.W4Matrix((q[:, 0::2] | q[:, 1::2] << 4).contiguous(), scale.contiguous(), bias)


class Block:
    """One block's weights, its cache, and what its operators hand on."""

    def __init__(self, model, seed, device):
        gen = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        d, hq, hkv, D, T = model.d, model.hq, model.hkv, model.D, model.T
        width = (hq + 2 * hkv) * D
        self.w_qkv = quantised4(rnd(width, d) * d ** -0.5, model.group)
        self.w_o = quantised4(rnd(d, hq * D) * (hq * D) ** -0.5, model.group)
        self.norm1, self.norm2 = 1 + 0.1 * rnd(d), 1 + 0.1 * rnd(d)
        layer = synth.make_layer(synth.LayerShape(T=T, d=d, E=model.experts, k=model.top_k, F=model.ff),
                                 seed=seed + 1, device=device)
        self.moe = lily.LayerWeights(layer["router_w"], layer["router_b"], layer["experts"])
        self.moe.split_router()
        shape = (model.pages, model.page, hkv, D)
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.zeros(shape[:3], device=device) for _ in range(2)]
        self.cache = lily.PagedCache8(*codes, *scales)
        self.x = torch.empty(T, d, dtype=BF, device=device)
        self.qkv = torch.empty(T, width, dtype=BF, device=device)
        self.q = torch.empty(T, hq, D, dtype=BF, device=device)
        self.heads = torch.empty(T, hq, D, dtype=BF, device=device)
        self.lse = torch.empty(T, hq, device=device)
        self.proj = torch.empty(T, d, dtype=BF, device=device)
        self.x2 = torch.empty(T, d, dtype=BF, device=device)
        self.y = torch.zeros(T, d, dtype=F32, device=device)
        self.routing = lily.RoutingBuffers(model.moe_dims, device)


class TokenModel:
    """`seqs` sequences of up to `room` tokens each; a step takes each one's token to its next."""

    def __init__(self, vocab=1003, blocks=2, d=512, hq=8, hkv=2, D=64, rot=64, experts=32, top_k=4, ff=128,
                 seqs=4, room=64, page=16, group=64, seed=0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
        self.vocab, self.d, self.hq, self.hkv, self.D, self.rot = vocab, d, hq, hkv, D, rot
        self.experts, self.top_k, self.ff, self.page, self.group = experts, top_k, ff, page, group
        self.room, T = room, seqs
        self.T = T
        each = -(-room // page)
        self.pages = each * seqs
        self.table = torch.randperm(self.pages, generator=gen, device=device).int().view(seqs, each).contiguous()
        self.moe_dims = lily.make_dims(T, d, experts, top_k, ff, 32)
        self.moe_ws = lily.alloc_workspace(lily.lily_moe_workspace_bytes(self.moe_dims), device)
        self.blocks = [Block(self, seed + 10 * i + 1, device) for i in range(blocks)]
        self.embedding = rnd(vocab, d)
        self.norm = 1 + 0.1 * rnd(d)
        self.head = quantised4(rnd(vocab, d) * 4 * d ** -0.5, group, symmetric=True)
        self.inv_freq = 1e6 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / max(rot, 1))

        self.tokens = torch.zeros(seqs, dtype=torch.int32, device=device)  # in, and out
        self.seq_lens = torch.zeros(seqs, dtype=torch.int32, device=device)
        self.residual = torch.empty(T, d, device=device)
        self.rows = torch.empty(T, d, dtype=BF, device=device)
        self.logits = torch.empty(T, vocab, device=device)
        self.logprobs = torch.empty(T, device=device)
        # how each sequence samples; u: its uniform number, the caller's, a new one for each step
        self.temperature = torch.ones(seqs, device=device)
        self.k = torch.full((seqs,), 50, dtype=torch.int32, device=device)
        self.p = torch.full((seqs,), 0.95, device=device)
        self.min_p = torch.full((seqs,), 0.01, device=device)
        self.u = torch.zeros(seqs, device=device)

        b = self.blocks[0]
        q, k, v = self.split(b.qkv)
        self.norm_first = lily.make_norm_dims(T, d, F32, F32, F32, BF, eps=EPS)
        self.norm_second = lily.make_norm_dims(T, d, BF, F32, F32, BF, eps=EPS)
        self.rope_dims = lily.make_rope_dims(q, k, v, b.q, rot)
        self.attn_dims = lily.make_attn_dims(b.q, b.heads, seqs, 1, 0, room, each, D ** -0.5)
        self.attn_ws = lily.alloc_workspace(lily.lily_attn_decode8_workspace_bytes(self.attn_dims, b.cache), device)
        self.qkv_dims = lily.make_linear_dims(b.x, b.w_qkv, b.qkv)
        self.o_dims = lily.make_linear_dims(b.heads.view(T, -1), b.w_o, b.proj)
        self.head_dims = lily.make_linear_dims(self.rows, self.head, self.logits)
        self.sample_dims = lily.make_sample_dims(self.logits)
        self.sample_ws = lily.alloc_workspace(256, device)

    def split(self, qkv):
        """q, k and v as views of the fused projection's rows."""
        T, n, m = qkv.shape[0], self.hq * self.D, self.hkv * self.D
        return (qkv[:, :n].view(T, self.hq, self.D), qkv[:, n:n + m].view(T, self.hkv, self.D),
                qkv[:, n + m:].view(T, self.hkv, self.D))

    def slots(self):
        """Where the next token of every sequence goes; nowhere (-1) once its room is full."""
        at = self.seq_lens.long()
        pages = torch.gather(self.table.long(), 1, (at // self.page).clamp(max=self.table.shape[1] - 1)[:, None])[:, 0]
        return torch.where(at < self.room, pages * self.page + at % self.page, -1)

    def embed(self):
        """The tokens' rows; row 0 for a sequence that got none (-1: its logits were nothing but -infinity or NaN)."""
        torch.index_select(self.embedding, 0, self.tokens.clamp(min=0), out=self.residual)

    def step(self):
        """self.tokens to the next ones, in place."""
        self.embed()
        slots, positions = self.slots(), self.seq_lens.clone()
        self.seq_lens += 1
        y = None
        for b in self.blocks:
            # (the first block's rows are the embedding's: nothing is added)
            if y is None:
                lily.lily_attn_add_rmsnorm(self.norm_first, self.residual, None, b.norm1, None, b.x)
            else:
                lily.lily_attn_add_rmsnorm(self.norm_first, y, self.residual, b.norm1, self.residual, b.x)
            lily.lily_decode_linear(self.qkv_dims, b.x, b.w_qkv, b.qkv)
            q, k, v = self.split(b.qkv)
            lily.lily_attn_rope_append8(self.rope_dims, b.cache, q, k, v, positions, slots, self.inv_freq, b.q,
                                        self.attn_ws)
            lily.lily_attn_decode8(self.attn_dims, b.cache, b.q, None, self.seq_lens, self.table, b.heads, b.lse,
                                   self.attn_ws)
            lily.lily_decode_linear(self.o_dims, b.heads.view(self.T, -1), b.w_o, b.proj)
            lily.lily_attn_add_rmsnorm(self.norm_second, b.proj, self.residual, b.norm2, self.residual, b.x2)
            run = lily.lily_moe_decode if self.T <= 8 else lily.lily_moe_forward
            run(self.moe_dims, b.x2, b.moe, b.routing, b.y, self.moe_ws)
            y = b.y
        lily.lily_attn_add_rmsnorm(self.norm_first, y, self.residual, self.norm, self.residual, self.rows)
        lily.lily_decode_linear(self.head_dims, self.rows, self.head, self.logits)
        lily.lily_decode_sample(self.sample_dims, self.logits, self.temperature, self.k, self.p, self.min_p, self.u,
                                self.tokens, self.logprobs, self.sample_ws)

    def status(self):
        return (lily.lily_moe_status(self.attn_ws) | lily.lily_moe_status(self.moe_ws)
                | lily.lily_moe_status(self.sample_ws))


def main():
    steps = 100
    model = TokenModel(vocab=131072, blocks=4, d=2048, hq=16, hkv=2, D=128, rot=128, experts=256, top_k=8, ff=512,
                       seqs=8, room=steps + 40, page=64)
    gen = torch.Generator(device="cuda").manual_seed(7)
    for _ in range(3):
        model.u.uniform_(generator=gen)
        model.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        model.step()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    a.record()
    for _ in range(steps):
        model.u.uniform_(generator=gen)
        graph.replay()
    b.record()
    torch.cuda.synchronize()
    assert model.status() == 0 and bool((model.tokens >= 0).all())
    print(f"{model.T} sequences, {len(model.blocks)} blocks, vocabulary {model.vocab}: "
          f"{a.elapsed_time(b) * 1e3 / steps:.1f} us a step")


if __name__ == "__main__":
    main()
