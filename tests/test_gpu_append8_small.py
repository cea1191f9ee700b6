"""lily_attn_rope_append8's codes of heads whose numbers are near fp32's least: those of fp32's x / s."""
import pytest
import torch

from attn8_ref import E4M3
from test_gpu_append8 import BF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [-117, -112, -108, -105, -90, -80, -40])
@pytest.mark.parametrize("rot", [0, 2])  # by runs of eight elements, and one by one
def test_codes_of_small_heads(exponent, rot):
    """Whatever bits below a largest number about 2^exponent; exact, since neither V nor K without a rotation is rounded
    before, and the host's quotient is IEEE's."""
    c = Case(300, 0, 4, 256, rot, seed=-exponent)
    c.positions.zero_()
    gen = torch.Generator().manual_seed(-exponent)
    bits = torch.randint(0, (127 + exponent) << 7, (2, 300, 4, 256), generator=gen)
    bits[..., 0] = ((127 + exponent) << 7) + torch.randint(0, 128, bits.shape[:-1], generator=gen)
    sign = torch.randint(0, 2, bits.shape, generator=gen) << 15
    new = (bits | sign).to(torch.int32).to(torch.int16).view(BF)
    c.nk.copy_(new[0])
    c.nv.copy_(new[1])
    c.call()
    for x, codes, scales in ((new[0], c.k, c.ks), (new[1], c.v, c.vs)):
        x = x.float()
        s = x.abs().amax(-1) / 448.0
        assert bool((s >= 2.0 ** -126).all())
        assert torch.equal(c.rows(scales)[c.slots].cpu(), s)
        want = (x / s[..., None]).to(E4M3).float()
        got = c.rows(codes)[c.slots].cpu().view(E4M3).float()
        assert int((got != want).sum()) == 0  # (as numbers: either zero for -0)
