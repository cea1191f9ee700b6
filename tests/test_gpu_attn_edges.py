"""Cases at the ends of the attention-side operators' ranges: values near the end of fp32, offsets
past 32 bits, arguments at their bounds, and waits that run out."""
import math

import pytest
import torch

import w4_grouped_gemm_gb300 as lily

from test_gpu_attn import Batch
from test_gpu_attn_norm_rope import _check_norm

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


# widths that fill eight warps, nearly, and not quite, with one, two and four chunks a thread
@pytest.mark.parametrize("d", [1536, 1656, 1664, 1984, 2048, 2056, 3320, 3328, 3968, 4096, 6592, 6656, 7936, 8192, 8200])
@pytest.mark.parametrize("xt,rt,ot", [(B, F, Q), (F, F, Q), (H, H, Q), (B, B, B), (F, B, H)])
def test_norm_widths_about_eight_warps(oracle_lib, d, xt, rt, ot):
    _check_norm(9, d, xt, rt, F, ot, 0, seed=d)
    if ot is Q and d % 64 == 0:
        _check_norm(9, d, xt, rt, F, ot, 64, seed=d)
    if ot is Q and d % 128 == 0:
        _check_norm(9, d, xt, rt, F, ot, 128, seed=d)


# ------------------------------------------------------------------------------------ rope, append
def _turn(x, positions, rot, freq):
    """Half-split rotation in 64 bits of x [T][heads][D]."""
    x = x.double().clone()
    angle = positions.double()[:, None, None] * freq
    a, b = x[..., :rot // 2].clone(), x[..., rot // 2:rot].clone()
    x[..., :rot // 2] = a * angle.cos() - b * angle.sin()
    x[..., rot // 2:rot] = b * angle.cos() + a * angle.sin()
    return x


@pytest.mark.parametrize("rot", [20, 64])                # element by element; in vectors
def test_rope_head_offsets_past_31_bits(oracle_lib, rot):
    """Heads so far apart that a head's offset passes 2^31 elements: q and q_out, k and v lie in two
    buffers, token by token behind one another within a head."""
    T, heads, D = 3, 3, 64
    stride = (1 << 31) - 8                               # elements, the largest that is taken
    gen = torch.Generator().manual_seed(rot)
    far = [torch.empty(2 * stride + 1024, dtype=B, device="cuda") for _ in range(2)]
    q, q_out, k, v = (far[i // 2][512 * (i % 2):].as_strided((T, heads, D), (D, stride, 1))
                      for i in range(4))
    data = [torch.randn(T, heads, D, generator=gen).to(B) for _ in range(3)]
    for at, x in zip((q, k, v), data):
        at.copy_(x)
    kc, vc = (torch.zeros(1, 16, heads, D, dtype=B, device="cuda") for _ in range(2))
    pos = torch.tensor([5, 1000, 77], dtype=torch.int32)
    freq = 1e4 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ws = lily.alloc_workspace(256)
    lily.lily_attn_rope_append(lily.make_rope_dims(q, k, v, q_out, rot), lily.PagedCache(kc, vc), q, k,
                               v, pos.cuda(), torch.tensor([9, 0, 4], device="cuda"), freq.cuda(),
                               q_out, ws)
    torch.cuda.synchronize()
    assert lily.lily_moe_status(ws) == 0
    slots = [9, 0, 4]
    for got, x in ((q_out, data[0]), (kc[0, slots], data[1])):
        want = _turn(x, pos, rot, freq)
        # bf16's rounding, and fp32 sines of both of a pair's elements (at most 6 in size)
        assert bool(((got.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + 12 * 2.0 ** -20).all())
    assert torch.equal(vc[0, slots].cpu(), data[2])


def test_rope_largest_number_of_tokens(oracle_lib):
    """T = 2^31 - 1, all tokens the same row (stride 0): the call is taken, not refused for a grid
    that wrapped."""
    q = torch.randn(1, 1, 8, generator=torch.Generator().manual_seed(2)).to(B).cuda()
    out = torch.zeros_like(q)
    kc, vc = (torch.zeros(1, 16, 1, 8, dtype=B, device="cuda") for _ in range(2))
    dims = lily.make_rope_dims(q, None, None, out, 0)
    dims.T, dims.q_token_stride, dims.qo_token_stride = 2 ** 31 - 1, 0, 0
    ws = lily.alloc_workspace(256)
    lily.lily_attn_rope_append(dims, lily.PagedCache(kc, vc), q, None, None, None, None, None, out, ws)
    torch.cuda.synchronize()
    assert lily.lily_moe_status(ws) == 0 and torch.equal(out, q)


# ------------------------------------------------------------------------------------ attention: waits
def _workspace(b):
    """A workspace of the batch's call whose contents behind the status are no sensible number."""
    out = torch.empty(b.q.shape, dtype=b.q.dtype, device="cuda")
    dims = lily.make_attn_dims(b.q, out, len(b.own), b.max_q, b.prefix, b.max_own, b.table.shape[1],
                               b.scale)
    ws = lily.alloc_workspace(lily.lily_attn_workspace_bytes(dims, b.cache()))
    ws[256:] = 0x7F
    return ws


def _give_up_then_recover(b):
    """With a limit of 0 the warps that compute give up while copies and products are in flight: the
    call ends with TIMEOUT.  With the limit restored the same workspace gives the right outputs."""
    want, want_lse = b.run()
    ws = _workspace(b)
    prev = lily.lily_attn_set_wait_ns(0)
    try:
        b.run(ws=ws, status=lily.LILY_STATUS_TIMEOUT, repeat=5)
    finally:
        assert lily.lily_attn_set_wait_ns(prev) == 0
    assert prev == 2_000_000_000
    out, lse = b.run(ws=ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    b.check(out, lse, skip=range(2, len(b.own)))


# prefixes on the tensor cores: one row block of two streams, pairs of row blocks (the last of one
# block only), and heads over 128
@pytest.mark.parametrize("D,hq,hkv,seqs,prefix,dtype", [
    (64, 8, 1, 16, 8200, B), (128, 8, 1, 16, 8200, H), (64, 8, 1, 40, 4000, H), (128, 8, 2, 44, 4000, B),
    (192, 1, 1, 100, 17000, H), (256, 8, 1, 40, 8000, B)])
def test_prefix_whose_waits_run_out(oracle_lib, D, hq, hkv, seqs, prefix, dtype):
    _give_up_then_recover(Batch(hq=hq, hkv=hkv, D=D, own=[0] * seqs, prefix=prefix, page=64, dtype=dtype,
                                seed=D))


# own pages and a prefix on mma.sync: 8, 16, 32 and 64 rows a unit, several units a block
@pytest.mark.parametrize("D,hq,hkv,q_len,seqs,own,prefix,dtype", [
    (64, 4, 2, 1, 40, 300, 0, B), (128, 8, 1, 1, 300, 60, 0, H), (256, 4, 4, 1, 5, 2000, 130, B),
    (128, 8, 1, 2, 30, 200, 0, B), (64, 8, 1, 4, 20, 200, 700, H), (256, 8, 1, 8, 9, 150, 0, H),
    (128, 8, 2, 5, 12, 500, 333, B)])
def test_own_pages_whose_waits_run_out(oracle_lib, D, hq, hkv, q_len, seqs, own, prefix, dtype):
    _give_up_then_recover(Batch(hq=hq, hkv=hkv, D=D, own=[max(q_len, own - 7 * i) for i in range(seqs)],
                                q_lens=[q_len] * seqs, prefix=prefix, dtype=dtype, seed=D + q_len))


def test_waits_that_run_out_leave_no_way_out_of_the_partials(oracle_lib):
    """A block that gives up has not written where its rows' partials lie.  What stands there instead,
    as another call's leftovers could, names the right sequence and partials far outside."""
    for q_len, prefix in ((1, 0), (3, 500)):
        b = Batch(hq=8, hkv=2, D=128, own=[400 - 9 * i for i in range(40)], q_lens=[q_len] * 40,
                  prefix=prefix, seed=q_len)
        want, want_lse = b.run()
        ws = _workspace(b)
        rows = sum(b.q_lens) * b.hq
        # (the table of the rows is the workspace's last part: four words a row)
        table = ws[-(-(-rows * 16 // 256) * 256):].view(torch.int32)[:4 * rows].view(-1, 4)
        prev = lily.lily_attn_set_wait_ns(0)
        try:
            for first, number in ((1 << 30, 1 << 20), (-(1 << 30), 7), (0, 1 << 30), (1 << 30, -5)):
                table[:, 0], table[:, 1], table[:, 2] = first, 1 << 28, number
                table[:, 3] = torch.arange(rows, dtype=torch.int32) // (q_len * b.hq)
                b.run(ws=ws, status=lily.LILY_STATUS_TIMEOUT)
        finally:
            lily.lily_attn_set_wait_ns(prev)
        out, lse = b.run(ws=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


# ------------------------------------------------------------------------------------ attention: small weights
# (tensor-core kernel or mma.sync, by the rows; one and two row blocks; heads over 128; as many heads as
# SMs, so that a block keeps a unit's keys together)
@pytest.mark.parametrize("D,seqs,up", [(64, 1, 14), (128, 3, 14), (256, 1, 14), (64, 65, 7), (128, 130, 7),
                                       (192, 65, 7)])
@pytest.mark.parametrize("floor,spread", [(26, 0), (20, 16), (26, 16)])
@pytest.mark.parametrize("dtype", [H, B])
def test_many_small_weights_beside_a_large_one(oracle_lib, D, seqs, up, floor, spread, dtype):
    """One key takes nearly all of a row, 2047 others have a weight near 2^-20 or 2^-26 each: together
    they are what the output shows, for the large one's value is 0."""
    n, heads = 2048, 152
    b = Batch(hq=heads, hkv=heads, D=D, own=[0] * seqs, prefix=n, page=64, dtype=dtype, seed=D)
    gen = torch.Generator().manual_seed(floor + spread)
    b.scale = math.log(2.0)                                    # scores are powers of two
    b.q.zero_()
    b.q[..., 0] = 4.0
    below = floor + 0.25 * torch.randint(0, spread + 1, (n,), generator=gen)
    below[0] = 0.0
    k = torch.zeros(n, D)
    k[:, 0] = 2.0 - below / 4                                  # exact in fp16 and bf16
    v = (torch.randn(n, D, generator=gen) if spread else torch.ones(n, D)).to(dtype)
    v[0] = 0.0
    b.keys[b.prefix_cells], b.values[b.prefix_cells] = k.to(dtype)[:, None], v[:, None]
    out, lse = b.run()
    v = v.double()
    p = torch.exp2(-below.double())
    want_lse = torch.log(p.sum()) + 8.0 * math.log(2.0)
    p /= p.sum()
    want = p @ v
    # roundings of the output and of the probabilities; scores' products are exact, their factor (fp32
    # log2 e times scale) is off by 2^-24 of up to 40; exponentials and sums 2^-18; fp16 probabilities
    # that are subnormal by 2^-25, at 2^up times their size
    half = torch.finfo(dtype).eps / 2
    tol = half * want.abs() + (half + 40 * 2.0 ** -23 + 2.0 ** -18) * (p @ v.abs())
    if dtype is H:
        tol = tol + n * 2.0 ** (-25 - up) * float(v.abs().max()) + 2.0 ** -25
    err = (out.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    assert bool(((lse.double() - want_lse).abs() <= 2.0 ** -20 * (1 + abs(float(want_lse)))).all())


# (one partial per row: a prefix of one tile, or as many units as SMs, so that no unit is cut.  Where
# partials meet, their weights are 2^lse, and an fp32 lse near 2^25 is as coarse as the scores.)
@pytest.mark.parametrize("D,seqs,heads,n", [(64, 1, 8, 64), (128, 3, 8, 50), (256, 1, 2, 64), (64, 130, 152, 2048),
                                            (128, 130, 152, 2048), (256, 65, 152, 2048)])
def test_fp16_scores_near_which_numbers_are_coarse(oracle_lib, D, seqs, heads, n):
    """Scores up to 2^25: the probabilities stay within fp16 and the output is the average of the keys
    of the largest score."""
    b = Batch(hq=heads, hkv=heads, D=D, own=[0] * seqs, prefix=n, page=64, dtype=H, seed=D)
    gen = torch.Generator().manual_seed(D)
    for q_top, k_top in ((8000.0, 4000.0), (3000.0, 700.0), (300.0, -900.0)):
        b.q.zero_()
        b.q[..., 0] = q_top
        k = torch.zeros(n, D)
        k[:, 0] = k_top - 32.0 * torch.randint(0, 4, (n,), generator=gen)
        b.keys[b.prefix_cells] = k.to(H)[:, None]
        b.scale = 1.0
        out, lse = b.run()
        v = b.values[b.prefix_cells].double()
        best = k[:, 0] == k[:, 0].max()
        want = v[best].mean(0)
        # all of the best keys have the same score, whatever it was rounded to, and the next one is
        # thousands below: roundings of P and of the output alone
        tol = 2.0 ** -11 * want.abs() + (2.0 ** -11 + 2.0 ** -18) * v[best].abs().mean(0) + 2.0 ** -25
        assert bool(((out.double() - want).abs() <= tol).all()), (q_top, k_top)


# ------------------------------------------------------------------------------------ attention: bad lengths
@pytest.mark.parametrize("seqs,prefix", [(2, 20), (2, 0), (70, 20)])
def test_bad_lengths_where_no_sequence_may_have_keys(oracle_lib, seqs, prefix):
    """max_seq_len 0: a length above or below it, and a range past the tokens, set BAD_LEN here too."""
    b = Batch(own=[0] * seqs, prefix=prefix, seed=seqs)
    for at, n in ((seqs - 1, 1), (0, -3)):
        lens = [0] * seqs
        lens[at] = n
        b.check(*b.run(lens=lens, status=lily.LILY_STATUS_BAD_LEN))
    b.check(*b.run())
    b.q_start[seqs] = seqs + 7
    out, lse = b.run(status=lily.LILY_STATUS_BAD_LEN)
    b.check(out, lse, skip=[seqs - 1])
