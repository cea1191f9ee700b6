"""lily_attn_decode8 with scales over all of fp32's range: what the append writes of the largest and smallest 16-bit
values, and scales of a caller's own."""
import pytest
import torch

import test_gpu_attn8
from attn8_ref import E4M3, attn8_ref
from test_gpu_attn8 import BF, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _subnormal_outputs(monkeypatch):
    """bf16 numbers below 2^-126 are whole multiples of 2^-133, so an output there is rounded by up to half of that:
    by 2^-134, however small it is (2^-8 of it elsewhere, which attn8_ref's bound has)."""
    def with_step(*args):
        out, lse, tol, tol_lse = attn8_ref(*args)
        return out, lse, tol + 2.0 ** -134, tol_lse
    monkeypatch.setattr(test_gpu_attn8, "attn8_ref", with_step)


SIZES = {  # of key i's value
    "largest": lambda i: 2.0 ** 125 * (1 + 0 * i),
    "smallest": lambda i: 2.0 ** -118 * (1 + 0 * i),
    "in turn": lambda i: torch.where(i % 2 == 0, 2.0 ** -110, 2.0 ** 100),
    "few large": lambda i: torch.where(i % 97 == 50, 2.0 ** 120, 2.0 ** -118),
    "growing": lambda i: 2.0 ** (-115 + 235 * i / i.numel()),
    "falling": lambda i: 2.0 ** (120 - 235 * i / i.numel()),
}


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_value_sizes(size, D):
    """bf16's values from 2^-118 to 2^125 times a normal number: scales of 2^-126 to 2^119.  The unnormalised sums of
    the largest are past fp32's range."""
    Case(8, 2, D, [600, 50, 1], v_size=SIZES[size], dtype=BF, seed=D).run().check()


@pytest.mark.parametrize("size", SIZES)
def test_value_sizes_split_over_ctas(size):
    """The same in partial outputs."""
    Case(8, 2, 128, [9000, 40], v_size=SIZES[size], dtype=BF, page=64, seed=3).run().check()


def _put(c, s, codes, scales, cache, cache_scales):
    """Sequence s's codes [len][hkv][D] and scales into the cache (layout nhd)."""
    at = torch.arange(codes.shape[0], device="cuda")
    pg, row = c.table[s].long()[at // c.page], at % c.page
    cache.view(torch.uint8)[pg, row] = codes.view(torch.uint8)
    cache_scales[pg, row] = scales


@pytest.mark.parametrize("scale", [2.0 ** 126, 2.0 ** -126, 2.0 ** -140])
def test_own_scales(scale):
    """Codes of 1, 0 and -1 under the largest power of two, and codes of up to 448 under the least normal number and
    one that is none."""
    c = Case(8, 2, 128, [300, 20], dtype=BF, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    for s, (kc, ks, vc, vs) in enumerate(c.seqs):
        if scale > 1:
            vc = torch.randint(-1, 2, vc.shape, generator=gen, device="cuda").float().to(E4M3)
        vs = torch.full_like(vs, scale)
        c.seqs[s] = kc, ks, vc, vs
        _put(c, s, vc, vs, c.v, c.vs)
    c.run().check()


def test_negative_scales():
    """A scale's sign is part of the number."""
    c = Case(8, 2, 128, [300, 20], seed=7)
    for s, (kc, ks, vc, vs) in enumerate(c.seqs):
        sign = torch.where(torch.arange(ks.shape[0], device="cuda") % 3 == 0, -1.0, 1.0)[:, None]
        c.seqs[s] = kc, ks * sign, vc, vs * sign.flip(0)
        _put(c, s, kc, ks * sign, c.k, c.ks)
        _put(c, s, vc, vs * sign.flip(0), c.v, c.vs)
    c.run().check()
