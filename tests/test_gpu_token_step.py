"""The decoder of examples/token_step.py, step after step, each operator against its definition in 64 bits from what
the one before it handed on; the same steps from a graph."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
import w4_grouped_gemm_gb300 as lily
from w4_grouped_gemm_gb300 import synth

from attn8_ref import attn8_ref
from attn_ref import E4M3_HALF, HALF, norm_ref, rope_ref
from decode_ref import linear_ref, linear_tol, sample_ref
from gpu_util import assert_layer_close

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _product(x, w, y, what):
    want, fp32 = linear_ref(x, w.q, w.scale, w.bias, w.group)
    err = (y.double().cpu() - want).abs()
    assert bool((err <= linear_tol(want, fp32, y.dtype)).all()), what


def _norm(got, r, w, what):
    """fp32 sums of a residual that is itself fp32 (2^-23 of the largest terms): bf16's half step and 2^-15."""
    from token_step import EPS
    _, n = norm_ref(r, None, w, EPS)
    assert bool(((got.double().cpu() - n).abs() <= (2.0 ** -8 + 2.0 ** -15) * n.abs() + 1e-5).all()), what


def _cache_rows(c, x):
    return x.reshape(-1, *x.shape[2:])  # [slot][head] ([D])


@pytest.mark.parametrize("seqs,kw", [(4, {}), (1, dict(hq=4, hkv=4, rot=32)), (11, dict(group=128, D=96, rot=96, hq=8, hkv=2)),
                                     (3, dict(group=32, page=32, hq=16, hkv=1))])
def test_steps(oracle_lib, seqs, kw):
    from token_step import TokenModel
    m = TokenModel(seqs=seqs, room=32, seed=5, **kw)
    gen = torch.Generator().manual_seed(6)
    m.tokens.copy_(torch.randint(0, m.vocab, (seqs,), generator=gen))
    m.temperature.copy_(torch.tensor([0.0, 0.7, 1.0, 1.5] * 3)[:seqs])
    scale = m.D ** -0.5
    for step in range(4):
        m.u.copy_(torch.rand(seqs, generator=gen))
        r = m.embedding[m.tokens.long()].double().cpu()
        slots = m.slots().cpu()
        m.step()
        torch.cuda.synchronize()
        assert m.status() == 0 and m.seq_lens.tolist() == [step + 1] * seqs
        pos = torch.full((seqs,), step)
        for n, b in enumerate(m.blocks):
            what = f"step {step} block {n}"
            if n:
                r = r + m.blocks[n - 1].y.double().cpu()
            _norm(b.x, r, b.norm1, what)
            _product(b.x, b.w_qkv, b.qkv, what)
            q, k, v = m.split(b.qkv)
            q64, qm = rope_ref(q, pos, m.inv_freq.cpu(), m.rot, 0)
            k64, km = rope_ref(k, pos, m.inv_freq.cpu(), m.rot, 0)
            assert bool(((b.q.double().cpu() - q64).abs() <= HALF[BF] * (q64.abs() + 2.0 ** -20 * qm) + 2.0 ** -21 * qm).all())
            # what the cache holds of the new tokens: half a step of e4m3, or of its subnormals, at the scale
            c = b.cache
            for new, mag, codes, scales in ((k64, km, c.k, c.k_scales), (v.double().cpu(), torch.zeros_like(km), c.v, c.v_scales)):
                s = _cache_rows(c, scales).cpu()[slots].double()
                got = _cache_rows(c, codes.view(torch.uint8)).cpu()[slots].view(torch.float8_e4m3fn).double() * s[..., None]
                near = 2.0 ** -21 * mag + 2.0 ** -22 * new.abs()
                assert bool(((got - new).abs() <= E4M3_HALF * (new.abs() + near) + near + 2.0 ** -10 * s[..., None]).all()), what
            # attention over what the cache holds
            G, kv = m.hq // m.hkv, [_cache_rows(c, x) for x in (c.k, c.k_scales, c.v, c.v_scales)]
            for i in range(seqs):
                at = torch.arange(step + 1, device="cuda")
                own = m.table[i].long()[at // m.page] * m.page + at % m.page
                for h in range(m.hkv):
                    out, lse, tol, tol_lse = attn8_ref(b.q[i, h * G:(h + 1) * G], *(
                        x.view(torch.uint8)[own][:, h].view(torch.float8_e4m3fn) if x.dtype == torch.float8_e4m3fn else x[own][:, h]
                        for x in kv), scale, [step + 1] * G)
                    assert bool(((b.heads[i, h * G:(h + 1) * G].double() - out).abs() <= tol).all()), what
                    assert bool(((b.lse[i, h * G:(h + 1) * G].double() - lse).abs() <= tol_lse).all()), what
            _product(b.heads.view(seqs, -1), b.w_o, b.proj, what)
            r = r + b.proj.double().cpu()
            _norm(b.x2, r, b.norm2, what)
            ro = oracle.route(b.routing.logits.cpu().numpy(), m.moe_dims.top_k, m.moe_dims.tile_rows)
            ref = oracle.moe_rows(synth.bf16_bits(b.x2), synth.experts_to_numpy(b.moe.experts), ro["ids"], ro["gates"],
                                  np.arange(seqs))
            assert_layer_close(b.y.cpu().numpy(), ref, what)
        _norm(m.rows, r + m.blocks[-1].y.double().cpu(), m.norm, f"step {step}")
        _product(m.rows, m.head, m.logits, f"step {step} head")
        for i in range(seqs):
            _, _, fits = sample_ref(m.logits[i], float(m.temperature[i]), int(m.k[i]), float(m.p[i]), float(m.min_p[i]),
                                    float(m.u[i]))
            assert fits(int(m.tokens[i]))
            assert float(m.logprobs[i]) <= 0


def test_steps_in_a_graph(oracle_lib):
    """Eager steps and replays of one captured step: the same tokens, log probabilities and caches."""
    from token_step import TokenModel
    seen = []
    u = torch.rand(6, 4, generator=torch.Generator().manual_seed(3)).cuda()
    for graph in (False, True):
        m = TokenModel(seed=8)
        m.tokens.copy_(torch.tensor([1, 2, 1000, 500]))
        m.u.copy_(u[0])
        m.step()
        run = m.step
        if graph:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                m.step()
            run = g.replay
        said = [m.tokens.clone()]
        for i in range(1, 6):
            m.u.copy_(u[i])
            run()
            said += [m.tokens.clone(), m.logprobs.clone()]
        torch.cuda.synchronize()
        assert m.status() == 0 and m.seq_lens.tolist() == [6] * 4
        seen.append(said + [b.cache.k.view(torch.uint8) for b in m.blocks] + [b.cache.v_scales for b in m.blocks])
    assert all(torch.equal(a, b) for a, b in zip(*seen))


def test_a_sequence_whose_room_is_full(oracle_lib):
    """Its token goes nowhere and its attention tells; the others' tokens are what they are without it."""
    from token_step import TokenModel
    said = []
    for lens in ((3, 16, 5), (3, 7, 5)):
        m = TokenModel(seqs=3, room=16, seed=9)
        m.seq_lens.copy_(torch.tensor(lens))
        m.tokens.copy_(torch.tensor([10, 20, 30]))
        m.u.fill_(0.4)
        m.step()
        torch.cuda.synchronize()
        assert m.status() == (lily.LILY_STATUS_BAD_LEN if 16 in lens else 0)
        said.append((m.tokens[[0, 2]].tolist(), m.logits[[0, 2]].clone()))
    assert said[0][0] == said[1][0] and torch.equal(said[0][1], said[1][1])


def test_a_sequence_without_a_token(oracle_lib):
    """-1, which the sampler gives for a row of nothing, steps as token 0 does; the others are what they are."""
    from token_step import TokenModel
    said = []
    for token in (-1, 0):
        m = TokenModel(seqs=3, room=16, seed=9)
        m.tokens.copy_(torch.tensor([10, token, 30]))
        m.u.fill_(0.4)
        m.step()
        torch.cuda.synchronize()
        assert m.status() == 0
        said.append((m.tokens.tolist(), m.logits.clone()))
    assert said[0][0] == said[1][0] and torch.equal(said[0][1], said[1][1])
