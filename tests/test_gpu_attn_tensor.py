"""The shared prefix on the tensor cores (many rows and keys) against a 64-bit reference: every case
asserts that the call's plan takes that kernel."""
import pytest
import torch

import w4_grouped_gemm_gb300 as lily

from test_gpu_attn import Batch

pytestmark = pytest.mark.gpu
B, H = torch.bfloat16, torch.float16


def keys_for(rows, hkv, D, less=0):
    """Keys that make the fewest tiles of 64 rows and 64 keys which go to the tensor cores, less up to
    63 of the last tile's."""
    blocks = hkv * -(-rows // 64)
    return 64 * -(-(256 if D <= 128 else 512) // blocks) - less


def tensor_batch(seqs, hq, hkv, D, less=0, prefix=None, page=16, **kw):
    rows = seqs * hq // hkv
    prefix = keys_for(rows, hkv, D, less) if prefix is None else prefix
    b = Batch(hq=hq, hkv=hkv, D=D, own=kw.pop("own", [1 + i % 3 for i in range(seqs)]), prefix=prefix,
              page=page, **kw)
    dims = lily.make_attn_dims(b.q, b.q, seqs, b.max_q, prefix, b.max_own, b.table.shape[1], b.scale)
    assert lily.lily_attn_prefix_kernel(dims, b.cache()) == lily.LILY_PREFIX_TENSOR
    return b


def go(b, some=4, **kw):
    """The call, and a few of its sequences, the first and last among them, against the reference."""
    out, lse = b.run(**kw)
    check(b, out, lse, some)


def check(b, out, lse, some=4):
    n = len(b.own)
    keep = {round(i * (n - 1) / (some - 1)) for i in range(some)}
    b.check(out, lse, skip=[s for s in range(n) if s not in keep])
    assert bool(out.float().isfinite().all()) and bool(lse.isfinite().all())


# 128 rows a block (two streams of alternate tiles), 256 (two row blocks, the last of which may be
# empty), several units
@pytest.mark.parametrize("seqs,hq,hkv", [(65, 1, 1), (13, 5, 1), (128, 1, 1), (129, 2, 2), (64, 4, 1),
                                         (43, 12, 2), (100, 7, 1), (97, 8, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rows(oracle_lib, seqs, hq, hkv, D):
    go(tensor_batch(seqs, hq, hkv, D, less=seqs % 64, page=32, seed=seqs))


@pytest.mark.parametrize("less", [0, 1, 15, 16, 47, 63])
@pytest.mark.parametrize("seqs", [10, 40])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_ends(oracle_lib, less, seqs, D):
    """The last tile of 128 keys, its pages and its second half anywhere between full and empty."""
    go(tensor_batch(seqs, 8, 1, D, less=less, dtype=H, seed=less))
    rows = 8 * seqs
    go(tensor_batch(seqs, 8, 1, D, prefix=keys_for(rows, 1, D) + 64 - less, dtype=B, seed=less))


@pytest.mark.parametrize("D", [8, 40, 72, 80, 96, 136, 192, 200])
@pytest.mark.parametrize("dtype", [B, H])
@pytest.mark.parametrize("seqs", [12, 25])
def test_head_dims(oracle_lib, D, dtype, seqs):
    go(tensor_batch(seqs, 6, 1, D, less=5, dtype=dtype, seed=D))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128, 200, 256])
def test_pages(oracle_lib, page, layout, D):
    go(tensor_batch(60, 8, 2, D, less=13, page=page, layout=layout, seed=page))
    go(tensor_batch(20, 8, 2, D, less=50, page=page, layout=layout, dtype=H, seed=page))


@pytest.mark.parametrize("D,dtype", [(64, B), (128, H), (128, B), (192, B), (256, H)])
@pytest.mark.parametrize("seqs", [10, 40])
def test_growing_maximum(oracle_lib, D, dtype, seqs):
    """Keys in the order of their size, large scores: the maximum keeps growing and the output is
    rescaled again and again."""
    b = tensor_batch(seqs, 8, 1, D, less=9, dtype=dtype, q_scale=12.0, seed=17)
    order = b.keys[b.prefix_cells, 0].float().norm(dim=-1).argsort()
    for c in (b.keys, b.values):
        c[b.prefix_cells] = c[b.prefix_cells[order]]
    go(b)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("seqs", [10, 40])
def test_bad_pages(oracle_lib, page, D, seqs):
    """Indices outside the cache, below and above: parts of a tile, whole tiles and whole runs of tiles
    without a page, the first and the last page; the rest counts."""
    b = tensor_batch(seqs, 8, 1, D, less=7, page=page, seed=18)
    n = len(b.prefix_pages)
    bad = {0, n - 1, *range(1, n, 7), *range(n // 3, n // 3 + max(1, 640 // page))}
    for i in bad:
        b.prefix_pages[i] = (-1, 10 ** 7, -(2 ** 31), len(b.keys) // page)[i % 4]
    out, lse = b.run(status=lily.LILY_STATUS_BAD_PAGE)
    keep = torch.tensor([i // page not in bad for i in range(b.prefix)])
    b.prefix_cells = b.prefix_cells[keep]
    check(b, out, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqs", [10, 40])
def test_no_page_at_all(oracle_lib, D, seqs):
    """A prefix without one good page: rows see their own keys, rows without any are 0."""
    b = tensor_batch(seqs, 8, 1, D, own=[i % 2 for i in range(seqs)], seed=19)
    b.prefix_pages.fill_(-5)
    out, lse = b.run(status=lily.LILY_STATUS_BAD_PAGE)
    b.prefix_cells = b.prefix_cells[:0]
    b.check(out, lse)
    assert bool((out[0::2] == 0).all())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_non_finite_prefix_keys(oracle_lib, D):
    """An infinity in V of a key that all rows see reaches all rows, in its column alone; a NaN in Q its
    own row alone."""
    b = tensor_batch(40, 8, 1, D, less=3, seed=20)
    clean, clean_lse = b.run()
    b.values[b.prefix_cells[700], 0, 5] = float("inf")
    q0 = b.q[3, 2].clone()
    b.q[3, 2, 1] = float("nan")
    out, lse = b.run()
    rest = torch.ones(out.shape, dtype=torch.bool)
    rest[..., 5] = False
    rest[3, 2] = False
    assert torch.equal(out[rest], clean[rest])
    assert bool(out[3, 2].isnan().all()) and bool(lse[3, 2].isnan())
    b.q[3, 2] = q0
    hit = out[..., 5].clone()
    hit[3, 2] = float("inf")
    assert bool((hit == float("inf")).all())
    lse[3, 2] = clean_lse[3, 2]
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("D", [128, 256])
def test_same_bits_every_time(oracle_lib, D):
    b = tensor_batch(97, 8, 2, D, less=11, seed=21)
    out, lse = b.run()
    for _ in range(3):
        again, lse2 = b.run(repeat=4)
        assert torch.equal(out, again) and torch.equal(lse, lse2)
