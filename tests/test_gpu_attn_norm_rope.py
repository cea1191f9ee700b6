"""Residual addition with RMSNorm, and rotation with the paged append, against 64-bit references."""
import math

import pytest
import torch

import w4_grouped_gemm_gb300 as lily

from attn_ref import E4M3_HALF, HALF, norm_ref, rope_ref

pytestmark = pytest.mark.gpu
B, H, F, Q = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


def _rows(T, d, dtype, gen, pad=0):
    """[T][d] view of rows that are d + pad apart."""
    return torch.randn(T, d + pad, generator=gen).to(dtype).cuda()[:, :d]


# The sum of squares is a tree of at most 32 + 5 + 16 + ... additions: 2^-18 relative at 16384 wide,
# half of it in the square root; the products and the weight two more roundings.
FACTOR = 2.0 ** -17


def _check_norm(T, d, xt, rt, wt, ot, group, x_pad=0, out_pad=0, res=True, weight=True, seed=0,
                scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = _rows(T, d, xt, gen, x_pad)
    r = _rows(T, d, rt, gen) * 3 if res else None
    w = (1 + 0.2 * torch.randn(d, generator=gen)).to(wt).cuda() if weight else None
    x *= scale
    res_out = torch.empty(T, d, dtype=rt, device="cuda")
    out = torch.full((T, d + out_pad), 7.0, device="cuda").to(ot)
    groups = d // group if group else 1
    scales = torch.full((T, groups), -1.0, device="cuda") if ot is Q else None
    dims = lily.make_norm_dims(T, d, xt, rt, wt, ot, group=group, eps=1e-6, x_stride=d + x_pad,
                               out_stride=d + out_pad)
    lily.lily_attn_add_rmsnorm(dims, x, r, w, res_out, out, scales)
    torch.cuda.synchronize()
    r64, n64 = norm_ref(x, r, w, 1e-6)
    want = x.float() + r.float() if res else x.float()
    assert torch.equal(res_out, want.to(rt))                  # one fp32 addition, rounded once
    if out_pad:
        assert bool((out[:, d:].float() == 7.0).all())        # nothing past a row is touched
    got = out[:, :d].double().cpu()
    if ot is not Q:
        tol = (HALF[ot] + FACTOR) * n64.abs() + (2.0 ** -25 if ot is H else 1e-38)
        assert bool(((got - n64).abs() <= tol).all())
        return
    g = n64.view(T, groups, -1)
    s64 = g.abs().amax(-1) / 448
    s = scales.double().cpu()
    assert bool(((s - s64).abs() <= FACTOR * s64).all())
    assert float(got.abs().max()) <= 448
    each = s.repeat_interleave(d // groups, 1)
    # half a step of 3 mantissa bits, or of the subnormals' 2^-9, at the scale in use
    tol = (E4M3_HALF + 2 * FACTOR) * n64.abs() + 2.0 ** -10 * each * (1 + 2.0 ** -10)
    assert bool(((got * each - n64).abs() <= tol).all())
    full = got.view(T, groups, -1).abs().amax(-1)
    assert bool(((full == 448) | (s64 == 0)).all())           # the largest value takes the range


@pytest.mark.parametrize("d", [1, 7, 8, 64, 200, 257, 1000, 1024, 2048, 4096, 5003, 8192, 16384])
@pytest.mark.parametrize("T", [1, 3])
def test_norm_widths(oracle_lib, d, T):
    _check_norm(T, d, B, F, F, B, 0, seed=d)


@pytest.mark.parametrize("xt,rt,wt,ot", [(B, B, B, B), (H, H, H, H), (F, F, F, H), (H, F, H, B),
                                         (F, B, B, B), (B, F, F, Q), (H, H, H, Q), (F, F, F, Q)])
def test_norm_types(oracle_lib, xt, rt, wt, ot):
    _check_norm(37, 320, xt, rt, wt, ot, 0, seed=1)
    _check_norm(5, 321, xt, rt, wt, ot, 0, seed=2)


# rows of odd widths one behind the other: each row begins at another place between two vectors
@pytest.mark.parametrize("d", [3, 9, 15, 250, 255, 1019, 1419, 2035, 2049, 4083, 4426, 8185, 16371, 16383])
@pytest.mark.parametrize("xt,rt,wt,ot", [(F, F, F, Q), (B, F, B, B), (H, H, F, Q), (F, B, H, H)])
def test_norm_odd_rows(oracle_lib, d, xt, rt, wt, ot):
    _check_norm(17, d, xt, rt, wt, ot, 0, seed=d)
    _check_norm(17, d, xt, rt, wt, ot, 0, x_pad=16, out_pad=8, seed=d)


@pytest.mark.parametrize("d,group", [(64, 64), (128, 128), (192, 64), (2048, 128), (4096, 64),
                                     (16384, 64), (16384, 128), (640, 128)])
@pytest.mark.parametrize("out_pad", [0, 3])
def test_norm_groups(oracle_lib, d, group, out_pad):
    _check_norm(6, d, B, F, B, Q, group, out_pad=out_pad, seed=d + group)


def test_norm_strides_and_options(oracle_lib):
    _check_norm(9, 256, B, F, F, B, 0, x_pad=8, out_pad=16)      # aligned gaps
    _check_norm(9, 256, B, F, F, B, 0, x_pad=1, out_pad=5)       # none
    _check_norm(9, 256, B, F, F, B, 0, res=False)
    _check_norm(9, 256, B, F, F, Q, 64, weight=False)
    _check_norm(9, 1000, H, F, F, H, 0, res=False, weight=False)
    _check_norm(700, 96, B, F, F, Q, 0)


def test_norm_in_place_and_zero_rows(oracle_lib):
    """The residual may be updated in place; a row of zeros gives zeros with scale 0; a NaN or an
    infinity stays in its row."""
    T, d = 5, 512
    gen = torch.Generator().manual_seed(3)
    x, res = _rows(T, d, B, gen), _rows(T, d, F, gen)
    x[1], res[1] = 0, 0
    x[2, 17] = math.nan
    x[3, 100] = math.inf
    want = x.float() + res
    out = torch.empty(T, d, dtype=Q, device="cuda")
    scales = torch.empty(T, d // 64, device="cuda")
    dims = lily.make_norm_dims(T, d, B, F, F, Q, group=64)
    lily.lily_attn_add_rmsnorm(dims, x, res, None, res, out, scales)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(res), torch.nan_to_num(want))
    assert bool((out[1].float() == 0).all()) and bool((scales[1] == 0).all())
    assert bool(scales[2].isnan().all()) and bool(out[2].float().isnan().all())
    assert bool(scales[3, 100 // 64].isnan())
    for row in (0, 4):
        assert bool(scales[row].isfinite().all()) and bool(out[row].float().isfinite().all())


def test_norm_tiny_values_keep_their_scale(oracle_lib):
    """A weight of 2^-120 takes n far below the reciprocal's range; the 8-bit rows stay right."""
    T, d = 2, 256
    gen = torch.Generator().manual_seed(4)
    x = _rows(T, d, F, gen)
    w = torch.full((d,), 2.0 ** -110, device="cuda")
    out = torch.empty(T, d, dtype=Q, device="cuda")
    scales = torch.empty(T, 1, device="cuda")
    lily.lily_attn_add_rmsnorm(lily.make_norm_dims(T, d, F, F, F, Q), x, None, w, None, out, scales)
    torch.cuda.synchronize()
    _, n = norm_ref(x, None, w, 1e-6)
    s = scales.double().cpu()
    tol = (E4M3_HALF + 2.0 ** -12) * n.abs() + 2.0 ** -9 * s
    assert bool((s > 0).all()) and bool(((out.double().cpu() * s - n).abs() <= tol).all())


# ------------------------------------------------------------------------------------ rope, append
def _cache(pages, page, hkv, D, layout, dtype, gen):
    shape = (pages, page, hkv, D) if layout == "nhd" else (pages, hkv, page, D)
    return [torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2)]


def _tokens(cache, layout):
    """[pages * page][hkv][D] view (copy) of a cache."""
    c = cache if layout == "nhd" else cache.transpose(1, 2)
    return c.reshape(-1, c.shape[2], c.shape[3])


def _check_rope(T, hq, hkv, D, rot, style, dtype, page=16, layout="nhd", far=100000, gap=0, seed=0,
                theta=1e6):
    gen = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * D + gap
    qkv = torch.randn(T, width, generator=gen).to(dtype).cuda()
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
    v = qkv[:, (hq + hkv) * D:(hq + 2 * hkv) * D].view(T, hkv, D)
    pages = T // page + 4
    kc, vc = _cache(pages, page, hkv, D, layout, dtype, gen)
    k0, v0 = _tokens(kc, layout).clone(), _tokens(vc, layout).clone()
    slots = torch.randperm(pages * page, generator=gen)[:T]
    slots[T // 2] = -1 if T > 1 else slots[T // 2]
    positions = torch.randint(0, far, (T,), generator=gen, dtype=torch.int32)
    positions[0] = far
    inv_freq = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    q_out = torch.empty(T, hq, D, dtype=dtype, device="cuda")
    ws = lily.alloc_workspace(256)
    dims = lily.make_rope_dims(q, k, v, q_out, rot, style=style)
    lily.lily_attn_rope_append(dims, lily.PagedCache(kc, vc, layout), q, k, v, positions.cuda(),
                               slots.cuda(), inv_freq.cuda(), q_out, ws)
    torch.cuda.synchronize()
    assert lily.lily_moe_status(ws) == 0
    qr, qm = rope_ref(q, positions, inv_freq, rot, style)
    kr, km = rope_ref(k, positions, inv_freq, rot, style)
    live = slots >= 0
    got_k, got_v = _tokens(kc, layout), _tokens(vc, layout)
    # half a step of the type, and 2^-20 of the pair for fp32 sines of an exact angle
    sub = 2.0 ** -25 if dtype is H else 0.0
    for got, ref, mag in ((q_out, qr, qm), (got_k[slots[live].cuda()], kr[live], km[live])):
        assert bool(((got.double().cpu() - ref).abs() <= HALF[dtype] * ref.abs() + 2.0 ** -20 * mag
                     + sub).all())
    assert torch.equal(got_v[slots[live].cuda()], v[live.cuda()])
    other = torch.ones(pages * page, dtype=torch.bool)
    other[slots[live]] = False                                  # all other cells keep their bits
    assert torch.equal(got_k[other.cuda()], k0[other.cuda()])
    assert torch.equal(got_v[other.cuda()], v0[other.cuda()])


@pytest.mark.parametrize("style", [0, 1])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (256, 64), (256, 256), (96, 96),
                                   (80, 80), (80, 20), (72, 6), (64, 0), (8, 8), (192, 96)])
def test_rope_heads(oracle_lib, D, rot, style):
    _check_rope(7, 4, 2, D, rot, style, B, seed=D + rot)


@pytest.mark.parametrize("T", [1, 2, 33, 1025, 4099])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_rope_lengths(oracle_lib, T, layout):
    _check_rope(T, 5, 1, 64, 64, 0, H, page=32, layout=layout, gap=24, seed=T)


def test_norm_huge_values_keep_their_codes(oracle_lib):
    """Maxima near the end of fp32's range: their reciprocals are small, not zero."""
    x = torch.zeros(2, 128, device="cuda")
    x[0, 0], x[1, :2] = 1.0, 1.0
    w = torch.full((128,), 2.0 ** 123, device="cuda")
    w[1] = 2.0 ** 122
    out, scales = torch.empty(2, 128, dtype=Q, device="cuda"), torch.empty(2, 1, device="cuda")
    dims = lily.make_norm_dims(2, 128, F, F, F, Q, eps=0.0)
    lily.lily_attn_add_rmsnorm(dims, x, None, w, None, out, scales)
    torch.cuda.synchronize()
    # rows' norms: sqrt(128) and 8 times w, the largest above 2^126
    codes = out.float().cpu()
    assert codes[0, 0] == 448 and codes[1, 0] == 448 and codes[1, 1] == 224 and not codes[:, 2:].any()
    top = torch.tensor([math.sqrt(128.0), 8.0], dtype=torch.float64) * 2.0 ** 123 / 448
    assert ((scales[:, 0].cpu().double() - top).abs() <= 8 * 2.0 ** -24 * top).all()


def test_rope_far_positions(oracle_lib):
    """Positions to 2^31 - 1 keep the angle (an fp32 product would be off by whole turns)."""
    _check_rope(64, 2, 1, 128, 128, 0, B, far=2 ** 31 - 1, seed=9)
    _check_rope(64, 2, 1, 128, 128, 1, H, far=2 ** 31 - 1, seed=10, theta=10.0)


def test_rope_bad_slot_sets_status_and_skips(oracle_lib):
    gen = torch.Generator().manual_seed(5)
    kc, vc = _cache(3, 16, 2, 64, "nhd", B, gen)
    k0, v0 = kc.clone(), vc.clone()
    T = 4
    k = torch.randn(T, 2, 64, generator=gen).to(B).cuda()
    slots = torch.tensor([48, 2 ** 40, 5, -7], device="cuda")    # 48 cells: 0 .. 47
    ws = lily.alloc_workspace(256)
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    freq = torch.ones(32, dtype=torch.float64, device="cuda")
    dims = lily.make_rope_dims(None, k, k, None, 64)
    lily.lily_attn_rope_append(dims, lily.PagedCache(kc, vc), None, k, k, pos, slots, freq, None, ws)
    torch.cuda.synchronize()
    assert lily.lily_moe_status(ws) == lily.LILY_STATUS_BAD_SLOT
    assert lily.lily_moe_status(ws) == 0
    k0.view(48, 2, 64)[5] = k[2]
    v0.view(48, 2, 64)[5] = k[2]
    assert torch.equal(kc, k0) and torch.equal(vc, v0)


def test_rope_in_place_and_rotate_only(oracle_lib):
    gen = torch.Generator().manual_seed(6)
    q = torch.randn(9, 3, 128, generator=gen).to(B).cuda()
    kc, vc = _cache(2, 16, 1, 128, "nhd", B, gen)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    freq = 1e4 ** (-torch.arange(0, 128, 2, dtype=torch.float64, device="cuda") / 128)
    ws = lily.alloc_workspace(256)
    out = torch.empty_like(q)
    cache = lily.PagedCache(kc, vc)
    lily.lily_attn_rope_append(lily.make_rope_dims(q, None, None, out, 128), cache, q, None, None,
                               pos, None, freq, out, ws)
    lily.lily_attn_rope_append(lily.make_rope_dims(q, None, None, q, 128), cache, q, None, None,
                               pos, None, freq, q, ws)
    torch.cuda.synchronize()
    assert torch.equal(q, out)


def test_kv_pair_in_one_allocation(oracle_lib):
    """K and V as the two halves of one [pages][2][page][heads][D] tensor."""
    gen = torch.Generator().manual_seed(7)
    kv = torch.zeros(3, 2, 16, 2, 64, dtype=B, device="cuda")
    k = torch.randn(20, 2, 64, generator=gen).to(B).cuda()
    v = torch.randn(20, 2, 64, generator=gen).to(B).cuda()
    ws = lily.alloc_workspace(256)
    pos = torch.zeros(20, dtype=torch.int32, device="cuda")
    freq = torch.ones(32, dtype=torch.float64, device="cuda")
    slots = torch.arange(20, device="cuda") + 11
    lily.lily_attn_rope_append(lily.make_rope_dims(None, k, v, None, 64),
                               lily.PagedCache(kv[:, 0], kv[:, 1]), None, k, v, pos, slots, freq,
                               None, ws)
    torch.cuda.synchronize()
    assert torch.equal(kv[:, 0].reshape(48, 2, 64)[11:31], k)     # position 0 turns nothing
    assert torch.equal(kv[:, 1].reshape(48, 2, 64)[11:31], v)
