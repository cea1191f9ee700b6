"""Shared-prefix attention over a paged cache against a 64-bit reference: head sizes and groups,
page sizes and layouts, lengths that end anywhere in a page or tile, empty rows, and what masked
places may hold."""
import math

import pytest
import torch

import w4_grouped_gemm_gb300 as lily

from attn_ref import attn_ref

pytestmark = pytest.mark.gpu
B, H = torch.bfloat16, torch.float16


class Batch:
    """A batch in a paged cache.  Cells that no sequence owns hold NaN, table entries past a
    sequence's pages hold indices far outside the cache."""

    def __init__(self, dtype=B, hq=4, hkv=2, D=64, page=16, layout="nhd", prefix=0, own=(5,),
                 q_lens=None, q_start=True, max_q=None, spare=0, seed=0, q_scale=1.0):
        gen = torch.Generator().manual_seed(seed)
        q_lens = [1] * len(own) if q_lens is None else list(q_lens)
        self.prefix, self.own, self.q_lens = prefix, list(own), q_lens
        self.hq, self.hkv, self.D, self.page, self.layout = hq, hkv, D, page, layout
        T = sum(q_lens)
        self.max_own = max(own) + spare
        width = -(-self.max_own // page) if self.max_own else 0
        n_pre = -(-prefix // page)
        need = [-(-n // page) for n in own]
        pages = n_pre + sum(need) + 2
        perm = torch.randperm(pages, generator=gen)
        keys = torch.full((pages * page, hkv, D), math.nan)
        values = keys.clone()
        self.prefix_pages = perm[:n_pre].to(torch.int32)
        table = torch.full((len(own), max(width, 1)), 10 ** 9, dtype=torch.int32)
        at = n_pre

        def fill(page_list, n):
            k, v = torch.randn(n, hkv, D, generator=gen), torch.randn(n, hkv, D, generator=gen)
            cells = torch.tensor([int(page_list[i // page]) * page + i % page for i in range(n)],
                                 dtype=torch.long)
            keys[cells], values[cells] = k.to(dtype).float(), v.to(dtype).float()
            return cells

        self.prefix_cells = fill(self.prefix_pages, prefix)
        self.own_cells = []
        for s, n in enumerate(own):
            mine = perm[at:at + need[s]]
            at += need[s]
            table[s, :need[s]] = mine.to(torch.int32)
            self.own_cells.append(fill(mine, n))
        self.keys, self.values = keys.to(dtype), values.to(dtype)
        self.table = table
        self.q = (q_scale * torch.randn(T, hq, D, generator=gen)).to(dtype)
        starts = [0]
        for n in q_lens:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q_start = torch.tensor(starts, dtype=torch.int32) if q_start else None
        self.max_q = max_q or max(1, max(q_lens))
        self.scale = 1.3 / math.sqrt(D)

    def cache(self):
        k, v = (c.view(-1, self.page, self.hkv, self.D) for c in (self.keys, self.values))
        if self.layout == "hnd":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        return lily.PagedCache(k.contiguous().cuda(), v.contiguous().cuda(), self.layout)

    def run(self, want_lse=True, lens=None, status=0, out=None, q=None, ws=None, repeat=1):
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda") if out is None else out
        lse = torch.full(q.shape[:2], 9.0, device="cuda") if want_lse else None
        dims = lily.make_attn_dims(q, out, len(self.own), self.max_q, self.prefix, self.max_own,
                                   self.table.shape[1], self.scale)
        cache = self.cache()
        if ws is None:
            ws = lily.alloc_workspace(lily.lily_attn_workspace_bytes(dims, cache))
        lens = self.own if lens is None else lens
        args = (q, self.prefix_pages.cuda() if self.prefix else None,
                self.q_start.cuda() if self.q_start is not None else None,
                torch.tensor(lens, dtype=torch.int32).cuda(), self.table.cuda(), out, lse, ws)
        for _ in range(repeat):
            lily.lily_attn_shared_prefix(dims, cache, *args)
        torch.cuda.synchronize()
        assert lily.lily_moe_status(ws) == status
        return out.cpu(), lse.cpu() if want_lse else None

    def check(self, out, lse, own_cells=None, skip=()):
        """Every row against the reference; own_cells: the cells of each sequence that count."""
        own_cells = self.own_cells if own_cells is None else own_cells
        G = self.hq // self.hkv
        for s, n_q in enumerate(self.q_lens):
            if n_q == 0 or s in skip:
                continue
            cells = torch.cat([self.prefix_cells, own_cells[s]])
            n, p = self.own[s], len(self.prefix_cells)
            seen = torch.zeros(n_q, len(cells), dtype=torch.bool)
            for j in range(n_q):
                seen[j, :p] = True
                seen[j, p:p + max(0, n - n_q + 1 + j)] = True
            t0 = self.starts[s]
            for h in range(self.hkv):
                q = self.q[t0:t0 + n_q, h * G:(h + 1) * G]
                ref, l64, tol, tol_l = attn_ref(q.reshape(n_q * G, -1), self.keys[cells, h],
                                                self.values[cells, h], self.scale,
                                                seen.repeat_interleave(G, 0))
                got = out[t0:t0 + n_q, h * G:(h + 1) * G].reshape(n_q * G, -1).double()
                err = (got - ref).abs()
                assert bool((err <= tol).all()), (s, h, float((err - tol).max()))
                if lse is not None:
                    gl = lse[t0:t0 + n_q, h * G:(h + 1) * G].reshape(-1).double()
                    none = l64 == -math.inf
                    assert torch.equal(gl == -math.inf, none)
                    assert bool(((gl - l64).abs()[~none] <= tol_l[~none]).all())

    def go(self, **kw):
        self.check(*self.run(**kw))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 200, 1000])
@pytest.mark.parametrize("prefix", [0, 37])
def test_lengths(oracle_lib, n, prefix):
    Batch(own=(n, 1, max(1, n // 2)), prefix=prefix, seed=n).go()


@pytest.mark.parametrize("prefix", [1, 16, 63, 64, 65, 500, 1023, 4097])
def test_prefix_lengths(oracle_lib, prefix):
    Batch(own=(3, 70), prefix=prefix, D=128, seed=prefix).go()


@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 96, 128, 136, 192, 200, 256])
@pytest.mark.parametrize("dtype", [B, H])
def test_head_dims(oracle_lib, D, dtype):
    Batch(dtype=dtype, D=D, own=(130, 33), prefix=150, seed=D).go()


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (8, 1), (7, 1), (10, 2), (24, 1), (48, 1),
                                    (64, 1), (15, 3), (128, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups(oracle_lib, hq, hkv, D):
    Batch(hq=hq, hkv=hkv, D=D, own=(100, 5, 64), prefix=90, seed=hq).go()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_pages_and_layouts(oracle_lib, page, layout, D):
    Batch(page=page, layout=layout, D=D, own=(page, page + 1, page - 1, 2 * page + 7),
          prefix=3 * page - 5, seed=page).go()


@pytest.mark.parametrize("q_lens", [(3, 1, 5), (5, 5, 5), (1, 0, 8), (40, 1, 70)])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (6, 2)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_query_tokens(oracle_lib, q_lens, hq, hkv, D):
    Batch(hq=hq, hkv=hkv, D=D, own=(64, 100, 70), q_lens=q_lens, prefix=100, seed=D).go()


def test_uniform_query_tokens_without_q_start(oracle_lib):
    Batch(own=(50, 9, 64), q_lens=(4, 4, 4), q_start=False, prefix=20).go()
    Batch(own=(50, 9), q_start=False).go()


@pytest.mark.parametrize("seqs,D", [(40, 64), (100, 128), (300, 128), (70, 256)])
def test_many_sequences_and_rows(oracle_lib, seqs, D):
    """Row counts of the prefix past one and several blocks; lengths from one to many tiles."""
    Batch(hq=8, hkv=2, D=D, own=[1 + (37 * i) % 150 for i in range(seqs)], prefix=700, page=32,
          seed=seqs).go()


# more than 64 rows per KV head: the tensor-core kernel of the prefix, whose CTAs take 128 rows (two
# streams of alternate tiles) or 256 (two row blocks, the last of which may be empty)
@pytest.mark.parametrize("seqs,hq,hkv", [(65, 1, 1), (13, 5, 1), (128, 1, 1), (129, 2, 2),
                                         (64, 4, 1), (43, 12, 2), (100, 7, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_rows(oracle_lib, seqs, hq, hkv, D):
    Batch(hq=hq, hkv=hkv, D=D, own=[1 + i % 3 for i in range(seqs)], prefix=300, page=32,
          seed=seqs).go()


@pytest.mark.parametrize("prefix", [1, 64, 127, 128, 129, 255, 257, 1000, 6001])
@pytest.mark.parametrize("seqs", [10, 30])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_rows_prefix_lengths(oracle_lib, prefix, seqs, D):
    Batch(hq=8, hkv=1, D=D, own=[1 + i % 3 for i in range(seqs)], prefix=prefix, dtype=H,
          seed=prefix).go()


@pytest.mark.parametrize("D", [8, 40, 72, 80, 96, 136, 192, 200])
@pytest.mark.parametrize("dtype", [B, H])
def test_wide_rows_head_dims(oracle_lib, D, dtype):
    Batch(dtype=dtype, hq=6, hkv=1, D=D, own=[2] * 25, prefix=700, seed=D).go()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_rows_pages(oracle_lib, page, layout, D):
    Batch(page=page, layout=layout, D=D, hq=8, hkv=2, own=[1] * 20, prefix=3 * page + 77,
          seed=page).go()
    Batch(page=page, layout=layout, D=D, hq=8, hkv=2, own=[1] * 60, prefix=2000, seed=page).go()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_rows_peaked_and_bad_pages(oracle_lib, D):
    """A maximum that keeps growing rescales the output; pages outside the cache are skipped, whole
    tiles of them too."""
    for seqs in (10, 40):
        b = Batch(hq=8, hkv=1, D=D, own=[3] * seqs, prefix=900, q_scale=12.0, seed=17)
        order = b.keys[b.prefix_cells, 0].float().norm(dim=-1).argsort()
        for c in (b.keys, b.values):
            c[b.prefix_cells] = c[b.prefix_cells[order]]
        b.go()
        b = Batch(hq=8, hkv=1, D=D, own=[3] * seqs, prefix=900, seed=18)
        bad = [0, 3, 5, *range(16, 32), 56]
        for i in bad:
            b.prefix_pages[i] = -1 if i % 2 else 10 ** 7
        out, lse = b.run(status=lily.LILY_STATUS_BAD_PAGE)
        keep = torch.tensor([i // 16 not in bad for i in range(900)])
        b.prefix_cells = b.prefix_cells[keep]
        b.check(out, lse)


# CTAs that go on from one unit to the next: from a unit with one row block to one with two, from few
# tiles to many, with both streams, one, or one that alternates
@pytest.mark.parametrize("D,hq,hkv,seqs,prefix", [(96, 28, 4, 44, 5000), (128, 15, 3, 100, 4000),
                                                  (64, 6, 3, 50, 9000), (128, 4, 2, 30, 30000),
                                                  (256, 8, 4, 45, 5000), (192, 1, 1, 360, 9000),
                                                  (256, 8, 1, 40, 20000)])
def test_units_in_a_row(oracle_lib, D, hq, hkv, seqs, prefix):
    b = Batch(hq=hq, hkv=hkv, D=D, own=[1 + i % 3 for i in range(seqs)], prefix=prefix, page=128,
              dtype=H, seed=seqs)
    out, lse = b.run()
    again, lse2 = b.run(repeat=8)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    b.check(out, lse, skip=[s for s in range(seqs) if s % 6])    # every sixth, to keep the CPU's part short


def test_batch_that_fills_the_gpu(oracle_lib):
    """More units than CTAs, cut at other places than their ends."""
    Batch(hq=2, hkv=2, D=64, own=[(97 * i) % 700 + 1 for i in range(350)], seed=8).go()


def test_long_own_sequence_split_over_ctas(oracle_lib):
    Batch(hq=8, hkv=1, D=128, own=(9000, 4), page=64, seed=11).go()
    Batch(hq=2, hkv=2, D=256, own=(3000,), page=128, dtype=H, seed=12).go()


def test_empty_rows(oracle_lib):
    """No prefix and no own keys, more new tokens than keys, sequences without tokens: rows that see
    nothing are 0 with lse -inf."""
    b = Batch(own=(0, 5, 0), seed=1)
    out, lse = b.run()
    b.check(out, lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    Batch(own=(2, 3), q_lens=(6, 3), seed=2).go()      # four of six tokens see nothing
    b = Batch(own=(0,), seed=3)                        # max_seq_len 0: nothing at all
    out, lse = b.run()
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    Batch(own=(0, 0), prefix=30, seed=4).go()


def test_query_bound_above_the_tokens(oracle_lib):
    """max_q_len is a bound: it may pass the call's number of tokens."""
    Batch(own=(9,), q_lens=(1,), max_q=5, prefix=20).go()
    Batch(own=(9, 70), q_lens=(3, 2), max_q=100, hq=8, hkv=1).go()


def test_spare_capacity_and_no_lse(oracle_lib):
    b = Batch(own=(5, 70), spare=1000, prefix=10, seed=5)
    out, _ = b.run(want_lse=False)
    b.check(out, None)


def test_strided_q_and_out(oracle_lib):
    """q as a slice of a fused projection's rows, out as a slice of wider rows."""
    b = Batch(own=(40, 7), prefix=33, hq=4, hkv=2, D=128, seed=6)
    T = b.q.shape[0]
    fused = torch.zeros(T, 4 * 128 + 512, dtype=B, device="cuda")
    q = fused[:, :512].view(T, 4, 128)
    q.copy_(b.q)
    wide = torch.full((T, 8, 256), 5.0, dtype=B, device="cuda")
    out = wide[:, 2:6, 64:192]
    got, lse = b.run(q=q, out=out)
    b.check(got, lse)
    wide[:, 2:6, 64:192] = 5.0
    assert bool((wide == 5.0).all())


def test_peaked_scores(oracle_lib):
    """Large scores, so that the running maximum moves and most weights vanish."""
    for D in (64, 128, 256):
        Batch(own=(500, 3), prefix=400, D=D, q_scale=12.0, seed=7).go()
        Batch(own=(500, 3), prefix=400, D=D, q_scale=12.0, dtype=H, seed=7).go()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_bad_pages_are_skipped(oracle_lib, D):
    """Indices outside the cache, below and above: their keys do not count, and the status says so."""
    b = Batch(own=(64, 200), prefix=160, D=D, seed=9)
    b.table[1, 3], b.table[1, 5] = -1, 10 ** 6
    b.prefix_pages[2] = 2 ** 30
    out, lse = b.run(status=lily.LILY_STATUS_BAD_PAGE)
    cells = b.own_cells[1]
    keep = torch.ones(200, dtype=torch.bool)
    keep[48:64] = keep[80:96] = False
    b.prefix_cells = torch.cat([b.prefix_cells[:32], b.prefix_cells[48:]])
    b.own[1] = int(keep.sum())
    b.check(out, lse, own_cells=[b.own_cells[0], cells[keep]])


def test_bad_lengths_are_clamped(oracle_lib):
    b = Batch(own=(30, 48, 0), prefix=20, seed=10)
    out, lse = b.run(lens=[30, 10 ** 6, -4], status=lily.LILY_STATUS_BAD_LEN)
    b.check(out, lse)


def test_bad_lengths_among_many_sequences(oracle_lib):
    """The same where the sequences are summed by groups, and the bad one's group has no keys."""
    n = 70
    b = Batch(own=[5] * 32 + [0] * (n - 32), prefix=20, seed=19)
    out, lse = b.run(lens=[5] * 32 + [0] * (n - 33) + [-1], status=lily.LILY_STATUS_BAD_LEN)
    b.check(out, lse)


def test_non_finite_values_of_unseen_tokens(oracle_lib):
    """A later token's K and V hold NaN and infinities: the rows before it do not see them, its own
    row and those after do."""
    for D, hq, hkv in ((64, 4, 2), (128, 8, 1), (256, 4, 4), (128, 32, 1)):
        for own in (70, 64, 5):
            b = Batch(own=(own, 40), q_lens=(5, 2), D=D, hq=hq, hkv=hkv, prefix=9, seed=own)
            clean, clean_lse = b.run()
            cell = b.own_cells[0][own - 2]                     # that of query token 3 of 5
            b.values[cell, :, 3] = math.nan
            b.values[cell, :, 4] = math.inf
            out, lse = b.run()
            assert torch.equal(out[:3], clean[:3]) and torch.equal(out[5:], clean[5:])
            assert bool(out[3:5, :, 3].isnan().all()) and bool((out[3:5, :, 4] == math.inf).all())
            assert torch.equal(lse, clean_lse)
            b.keys[cell] = math.nan
            out, lse = b.run()
            assert torch.equal(out[:3], clean[:3]) and torch.equal(out[5:], clean[5:])
            assert torch.equal(lse[:3], clean_lse[:3])
            assert bool(out[3:5].isnan().all()) and bool(lse[3:5].isnan().all())


def test_same_bits_every_time_and_on_other_streams(oracle_lib):
    b = Batch(hq=8, hkv=2, D=128, own=[1 + (91 * i) % 333 for i in range(60)], prefix=900, seed=13)
    out, lse = b.run(repeat=3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out2, lse2 = b.run()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_graph_capture(oracle_lib):
    """Append and attention of one decode step captured in a graph and replayed."""
    b = Batch(own=(40, 41), prefix=50, hq=4, hkv=2, D=64, seed=14)
    want, _ = b.run()
    q, cache = b.q.cuda(), b.cache()
    out = torch.zeros_like(q)
    dims = lily.make_attn_dims(q, out, 2, 1, 50, b.max_own, b.table.shape[1], b.scale)
    ws = lily.alloc_workspace(lily.lily_attn_workspace_bytes(dims, cache))
    pre, qs, lens, table = (t.cuda() for t in (b.prefix_pages, b.q_start,
                                               torch.tensor(b.own, dtype=torch.int32), b.table))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lily.lily_attn_shared_prefix(dims, cache, q, pre, qs, lens, table, out, None, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_cache_past_32_bits(oracle_lib):
    """Pages whose element offsets pass 2^32, and 2^31 tokens' worth of slots never touched."""
    D, page = 256, 64
    n_pages = (2 ** 32 // (page * D)) + 8                        # 8.6 GB of K and of V
    k = torch.empty(n_pages, page, 1, D, dtype=B, device="cuda")
    v = torch.empty(n_pages, page, 1, D, dtype=B, device="cuda")
    gen = torch.Generator().manual_seed(15)
    n = 100
    kk, vv = (torch.randn(n, 1, D, generator=gen).to(B) for _ in range(2))
    pages = torch.tensor([n_pages - 1, n_pages - 3], dtype=torch.int32)
    slots = torch.tensor([int(pages[i // page]) * page + i % page for i in range(n)]).cuda()
    ws = lily.alloc_workspace(256)
    cache = lily.PagedCache(k, v)
    lily.lily_attn_rope_append(lily.make_rope_dims(None, kk.cuda(), vv.cuda(), None, 0), cache,
                               None, kk.cuda(), vv.cuda(), None, slots, None, None, ws)
    q = torch.randn(1, 2, D, generator=gen).to(B)
    out = torch.empty(1, 2, D, dtype=B, device="cuda")
    dims = lily.make_attn_dims(q, out, 1, 1, 0, n, 2, 0.05)
    ws = lily.alloc_workspace(lily.lily_attn_workspace_bytes(dims, cache))
    lily.lily_attn_shared_prefix(dims, cache, q.cuda(), None, None,
                                 torch.tensor([n], dtype=torch.int32).cuda(), pages[None].cuda(),
                                 out, None, ws)
    torch.cuda.synchronize()
    ref, _, tol, _ = attn_ref(q[0], kk[:, 0], vv[:, 0], 0.05, torch.ones(2, n, dtype=torch.bool))
    assert bool(((out[0].double().cpu() - ref).abs() <= tol).all())
