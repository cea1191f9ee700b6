"""Cases at the ends of the attention-side operators' ranges: values near the end of fp32, offsets
past 32 bits, arguments at their bounds, and waits that run out."""
import math

import pytest
import torch

import w4_grouped_gemm_gb300 as lily

pytestmark = pytest.mark.gpu
B, H, F, Q = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.mark.parametrize("d,group,x_pad,out_pad", [
    (256, 0, 0, 0), (256, 64, 0, 0), (256, 128, 0, 0),   # whole vectors, a scale per row or group
    (257, 0, 0, 0),                                      # rows at all distances from a vector
    (256, 64, 0, 3), (256, 0, 1, 0)])                    # element by element
def test_norm_maximum_whose_scale_rounds_to_zero(oracle_lib, d, group, x_pad, out_pad):
    """A row or group that is zero but for a denormal below 448 * 2^-150: its scale is 0, its codes
    are 0, and no other row changes."""
    T = 5
    x = torch.zeros(T, d + x_pad, device="cuda")[:, :d]
    x[:, 0] = 1.0
    x[1::2, 1:] = 1.0
    w = torch.ones(d, device="cuda")
    w[0] = 2.0 ** -147                                   # n[0] = sqrt(d) 2^-147 in the even rows
    top = math.sqrt(d) * 2.0 ** -147
    assert 0 < top / 448 < 2.0 ** -150
    out = torch.full((T, d + out_pad), 7.0, device="cuda").to(Q)
    scales = torch.full((T, d // group if group else 1), -1.0, device="cuda")
    dims = lily.make_norm_dims(T, d, F, F, F, Q, group=group, eps=0.0, x_stride=d + x_pad,
                               out_stride=d + out_pad)
    lily.lily_attn_add_rmsnorm(dims, x, None, w, None, out, scales)
    torch.cuda.synchronize()
    codes = out[:, :d].float().cpu()
    assert bool((codes[0::2] == 0).all()) and bool((scales[0::2] == 0).all())
    assert bool((codes[1::2, 1:] == 448).all()) and bool((codes[1::2, 0] == 0).all())
    # (rows of ones: n = 1 to a few roundings of fp32)
    assert bool(((scales[1::2].double() * 448 - 1).abs() <= 2.0 ** -20).all())
