"""The decoder block of examples/decoder_block.py: its attention half, step after step, against the
same step in 64 bits from the residual and the weights, and its MoE half against the FP64 oracle."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import synth

from attn_ref import norm_ref, rope_ref
from gpu_util import assert_layer_close

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len,seqs", [(1, 4), (2, 3), (1, 40)])
def test_block_steps(oracle_lib, q_len, seqs):
    """Three steps.  The block's own rounded values (8-bit rows, projections) enter the 64-bit step
    where it rounds them, so that what is compared is one operator's error at a time."""
    from decoder_block import EPS, DecoderBlock
    b = DecoderBlock(seqs=seqs, q_len=q_len, prefix=37, own=16, seed=5)
    gen = torch.Generator().manual_seed(6)
    pre = torch.randn(2, b.prefix, b.hkv, b.D, generator=gen).bfloat16()
    b.fill_prefix(pre[0].cuda(), pre[1].cuda())
    residual = torch.randn(b.T, b.d, generator=gen).cuda()
    y = torch.randn(b.T, b.d, generator=gen).cuda()
    k_pre, _ = rope_ref(pre[0], torch.arange(b.prefix), b.inv_freq.cpu(), b.rot, 0)
    keys, values = [[k_pre.bfloat16().double()] for _ in range(seqs)], [[pre[1].double()] for _ in range(seqs)]
    for step in range(3):
        r0, y0 = residual.clone(), y.clone()
        y = b.step(residual, y)
        torch.cuda.synchronize()
        assert b.status() == 0
        # 8-bit rows: half a step of e4m3, or of its subnormals, at the row's scale
        r, n = norm_ref(y0, r0, b.norm1, EPS)
        rows = b.h8.double().cpu() * b.scales.double().cpu()
        tol = (2.0 ** -4 + 2.0 ** -15) * n.abs() + 2.0 ** -10 * b.scales.double().cpu() * 1.01
        assert bool(((rows - n).abs() <= tol).all())
        # the projection, rotated; bf16 rounds twice (product, rotation)
        qkv = (rows.float().bfloat16().double() @ b.w_qkv.double().cpu())
        q64, k64, v64 = b.split(qkv)
        lens = step * q_len
        pos = (b.prefix + lens + torch.arange(q_len)).repeat(seqs)
        q64, qm = rope_ref(q64, pos, b.inv_freq.cpu(), b.rot, 0)
        k64, km = rope_ref(k64, pos, b.inv_freq.cpu(), b.rot, 0)
        q_got, _, v_got = (x.double().cpu() for x in b.split(b.qkv))
        assert bool(((q_got - q64).abs() <= 2.0 ** -7 * qm + 1e-5).all())
        assert bool(((v_got - v64).abs() <= 2.0 ** -7 * v64.abs() + 1e-5).all())
        # what the cache holds of the new tokens is k to the same bound
        slots, _ = b.slots_of(b.seq_lens - q_len)
        k_got = b.cache.k.view(-1, b.hkv, b.D)[slots].double().cpu()
        assert bool(((k_got - k64).abs() <= 2.0 ** -7 * km + 1e-5).all())
        assert torch.equal(b.cache.v.view(-1, b.hkv, b.D)[slots].double().cpu(), v_got)
        # attention from the cached values: bf16 probabilities and output
        G = b.hq // b.hkv
        for s in range(seqs):
            new = slice(s * q_len, (s + 1) * q_len)
            keys[s].append(k_got[new])
            values[s].append(v_got[new])
            kk, vv = torch.cat(keys[s]), torch.cat(values[s])
            for j in range(q_len):
                n_seen = b.prefix + lens + j + 1
                for h in range(b.hq):
                    a = kk[:n_seen, h // G] @ q_got[s * q_len + j, h] / math.sqrt(b.D)
                    p = torch.softmax(a, 0)
                    want = p @ vv[:n_seen, h // G]
                    got = b.heads[s * q_len + j, h].double().cpu()
                    bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * (p @ vv[:n_seen, h // G].abs())
                    assert bool(((got - want).abs() <= bound).all())
        # second addition and norm, then the experts
        r2, n2 = norm_ref(b.proj, r.float().cuda(), b.norm2, EPS)
        assert bool(((residual.double().cpu() - r2).abs() <= 2.0 ** -23 * r2.abs() + 1e-6).all())
        assert bool(((b.x.double().cpu() - n2).abs() <= (2.0 ** -8 + 2.0 ** -15) * n2.abs() + 1e-30).all())
        ro = oracle.route(b.routing.logits.cpu().numpy(), b.moe_dims.top_k, b.moe_dims.tile_rows)
        ref = oracle.moe_rows(synth.bf16_bits(b.x), synth.experts_to_numpy(b.moe_w.experts), ro["ids"],
                              ro["gates"], np.arange(b.T))
        assert_layer_close(y.cpu().numpy(), ref, f"step {step}")
        y = y.clone()


def test_block_step_in_a_graph(oracle_lib):
    """A whole step captured and replayed gives what eager steps give (the lengths grow on the GPU)."""
    from decoder_block import DecoderBlock
    outs = []
    for graph in (False, True):
        b = DecoderBlock(seqs=4, prefix=20, own=32, seed=8)
        gen = torch.Generator().manual_seed(9)
        pre = torch.randn(2, b.prefix, b.hkv, b.D, generator=gen).bfloat16().cuda()
        b.fill_prefix(pre[0], pre[1])
        residual = torch.randn(b.T, b.d, generator=gen).cuda()
        b.y.copy_(torch.randn(b.T, b.d, generator=gen))
        b.step(residual, b.y)
        if graph:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                b.step(residual, b.y)
            for _ in range(3):
                g.replay()
        else:
            for _ in range(3):
                b.step(residual, b.y)
        torch.cuda.synchronize()
        assert b.seq_lens.tolist() == [4] * 4
        outs.append((residual.clone(), b.y.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
