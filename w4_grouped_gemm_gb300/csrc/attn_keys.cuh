// attn_keys.cuh -- attention over a paged cache for a batch that shares a prefix:
// partial outputs over runs of keys (lily_attn_shared_prefix), included once per
// element type.
//
//   out = sum_k softmax_k(scale q.k) v_k.  Over any part of the keys, with
//   m = max s, l = sum 2^(c (s - m)), o = sum 2^(c (s - m)) v / l, c = scale log2(e),
//   the part's weight is 2^(c m + log2 l); parts add up with those weights.  (Any z
//   near c m serves in its place; see softmax_z.)
//
// The shared prefix is one "sequence" whose query rows are the whole batch's,
// so its keys and values are read once for all; each sequence's own pages are
// a sequence of few rows (its new tokens times the query heads per KV head).
// Both run here as a set of units (AttnSet): the units' 64-key tiles form one
// list that the CTAs share out evenly, whatever the lengths, and a unit cut
// between CTAs leaves one partial per CTA for the merge.  Few rows and long
// lengths so fill the GPU as well as many rows and short ones.
//
// Per CTA one producer warp and four warps of mma.sync (16 rows each).  Up to
// 64 rows meet each key, so a byte of K or V brings at most 64 flop: HBM
// bounds these units, not the tensor cores, and mma.sync keeps the softmax in
// registers.  The producer brings K, V (TMA, one box per page and 64
// dimensions) and the rows of Q into a ring of stages; the warps split a
// tile's keys when rows are few (16 rows: 16 keys each; 64 rows: a row block
// each).  Two CTAs per SM (heads of up to 128) hide one's softmax and merges
// behind the other's loads.
//
// Measured, in a graph, with the merge: 4 sequences behind 131072 keys (16 query
// heads on 2, D = 256): 58 us, 270 MB, 4.7 TB/s; 96 sequences with up to 2500
// own keys behind 2051 (32 heads on 8, D = 128): 120 us, 540 MB, 4.5 TB/s; one
// sequence of 301 keys: 8.9 us, of which the two launches and the merge are some
// 6.  A CTA spends some 2 us on a unit besides its tiles (rows of Q, the warps'
// sums, the partial), which bounds batches of short sequences: 300 of up to 60
// keys take 34 us.
#pragma once
#include "attn.cuh"

namespace lily {
namespace {

constexpr int kWarps = 4;                       // compute warps
constexpr int kThreads = 32 * (kWarps + 1);     // and the producer
constexpr int kTile = kAttnTile;

// DP: head dimension rounded up to 64, 128 or 256 (the rest reads as zero);
// ROWS: query rows of a unit, 8, 16, 32 or 64 (8 fill both halves of an mma's 16).
template <int DP, int ROWS>
struct Cfg {
  static constexpr int kRows = ROWS;
  static constexpr int WR = ROWS <= 16 ? 1 : ROWS / 16;  // blocks of 16 rows
  static constexpr int kWK = kWarps / WR;        // warps that split a tile's keys
  static constexpr int kKeys = kTile / kWK;      // keys of a warp
  static constexpr int kOcc = DP <= 128 ? 2 : 1;
  // (two at 128 dimensions: a third brought nothing and cost 3 to 12 percent
  // through the L1 cache that it took, 39 sequences of up to 2900 keys, 21 rows a
  // unit, 39.1 us against 36.4)
  static constexpr int kStages = DP == 64 ? 6 : DP == 128 ? 2 : 3;
  static constexpr int kHalfBytes = kTile * 128;             // 64 keys x 64 dimensions
  static constexpr int kTileBytes = kHalfBytes * (DP / 64);  // K or V of a tile
  static constexpr int kStageBytes = 2 * kTileBytes;
  // Q: up to 128 dimensions live in registers during a unit; 256 stay in shared
  // memory (rows padded by 16 bytes).  Several units' rows are brought ahead
  // where units are short: with one buffer the next unit's K and V waited for
  // its Q, and a unit of one key took 7 us.
  static constexpr bool kQRegs = DP <= 128;
  static constexpr int kQPitch = kQRegs ? DP * 2 : DP * 2 + 16;
  static constexpr int kQBufs = ROWS == 8 ? (DP == 256 ? 3 : 4) : ROWS == 16 ? 2 : 1;
  static constexpr int kQBytes = kRows * kQPitch;
  // columns of O that the warps of a row block exchange at a time
  static constexpr int kRedRows = ROWS < 16 ? ROWS : 16;
  static constexpr int kRedCols = ROWS == 8 ? 64 : ROWS == 16 ? 32 : 16;
  static constexpr int kRedBytes = kWK > 1 ? kWarps * kRedRows * kRedCols * 4 : 0;
  static constexpr int kQOff = kStages * kStageBytes;
  static constexpr int kRedOff = kQOff + kQBufs * kQBytes;
  static constexpr int kBytes = kRedOff + kRedBytes;
};

struct alignas(16) Desc {
  int part, head, q0, row0;   // partial index (-1: no more); KV head; first token; first row
  int nrows, qn, len, key0;   // rows; tokens and keys of the sequence; first key
  int tiles, pad[3];
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte piece c (0..7) of row r in a tile of 128-byte rows
// with the 128-byte swizzle (tile base 1024-byte aligned).
__device__ __forceinline__ uint32_t swz(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Units and tiles of a sequence: row blocks per KV head, and tiles per unit.
__device__ __forceinline__ int blocks_of(const AttnSet& s, int G, int qn) {
  return (qn * G + s.rows - 1) / s.rows;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// Shared memory of any of the variants beside stages, Q and the exchange.
struct Fixed {
  static constexpr int kMaxStages = 6, kMaxQBufs = 4;
  uint64_t bars[2 * kMaxStages + 2 * kMaxQBufs];
  Desc desc[kMaxQBufs];
  unsigned long long mask[kMaxStages];  // valid keys of a stage
  float red_z[kWarps][16], red_l[kWarps][16];
  int abort;
  int dead[2];  // compute warps agree at each unit whether to go on
};

// Partials of one set: CTA `cta` of its `set.grid`.
template <int DP, int ROWS, bool F16>
__device__ __forceinline__ void keys_body(const AttnArgs& a, const AttnSet& set, const CUtensorMap& mk,
                                          const CUtensorMap& mv, bool first, int cta,
                                          uint8_t* smem, Fixed& fx) {
  using C = Cfg<DP, ROWS>;
  constexpr int WR = C::WR;
  static_assert(C::kStages <= Fixed::kMaxStages && C::kQBufs <= Fixed::kMaxQBufs, "shared memory");
  auto& bars = fx.bars;
  auto& desc = fx.desc;
  auto& mask_s = fx.mask;
  auto& red_z = fx.red_z;
  auto& red_l = fx.red_l;
  auto& abort_s = fx.abort;
  auto& dead_s = fx.dead;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (C::kStages + i); };
  auto qfull = [&](int i) { return bar0 + 8 * (2 * C::kStages + i); };
  auto qempty = [&](int i) { return bar0 + 8 * (2 * C::kStages + C::kQBufs + i); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kWarps);
    }
    for (int i = 0; i < C::kQBufs; ++i) {
      mbar_init(qfull(i), 1);
      mbar_init(qempty(i), kWarps);
    }
    fence_mbar_init();
    abort_s = 0;
    dead_s[0] = dead_s[1] = 0;
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  // Q rows start as zeros: dimensions past D are never written and meet K's
  // zero fill, rows past a unit's last hold numbers
  for (int i = threadIdx.x; i < C::kQBufs * C::kQBytes / 16; i += kThreads)
    reinterpret_cast<uint4*>(smem + C::kQOff)[i] = make_uint4(0, 0, 0, 0);
  // and blocks of 64 dimensions past D, which no copy writes
  const int halves = (a.D + 63) / 64;
  if (halves < DP / 64)
    for (int i = threadIdx.x; i < C::kStages * 2 * C::kTileBytes / 16; i += kThreads)
      if (i % (C::kTileBytes / 16) >= halves * (C::kHalfBytes / 16))
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncthreads();
  if (first) pdl_wait();
  pdl_trigger();

  // The set's tiles (31 bits: checked on the host).  Up to 32 sequences: the
  // producer has them in its lanes.  More: 32 at a time by all warps, which
  // leave the groups' sums in the first stage.
  auto cost_of = [&](const SeqInfo& q) { return a.hkv * blocks_of(set, a.G, q.qn) * tiles_of(q.len); };
  const int groups = (set.n_seqs + 31) / 32;
  int* sums = reinterpret_cast<int*>(smem);
  if (groups > 1) {
    for (int g = warp; g < groups; g += kWarps + 1) {
      const int i = g * 32 + lane;
      SeqInfo q = {};
      if (i < set.n_seqs) q = seq_info(set, a.T, i);
      if (q.bad && cta == 0) set_status(a.status, LILY_STATUS_BAD_LEN);
      const int c = __reduce_add_sync(0xffffffffu, cost_of(q));
      if (lane == 0) sums[g] = c;
    }
    fence_proxy_async_smem();
    __syncthreads();
  }

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    // Short sequences make this warp the bottleneck, so it keeps global memory
    // latency off its path: 32 sequences' lengths lie in the lanes, the next
    // sequence's first pages are requested a sequence ahead.
    int stage = 0, phase = 0, seg = 0;
    bool ok = true;
    uint32_t used = 0;  // stages filled at least once
    const int ps = a.page_shift;
    const int box_rows = min(kTile, 1 << ps);
    const int pages_per_tile = kTile / box_rows;
    const uint32_t box_bytes = box_rows * 128;
    // lane l: page l / (2 halves) of a tile, K or V, half of the head
    const int i = lane / (2 * halves), rest = lane - i * 2 * halves;
    const bool is_v = rest >= halves;
    const int hf = rest - (is_v ? halves : 0);
    const uint32_t at_stage = (is_v ? C::kTileBytes : 0) + hf * C::kHalfBytes + i * box_bytes;

    int s0 = -1, s = 0;       // sequences s0 .. s0 + 31 lie in the lanes; current one
    int s_base = 0;           // first tile of sequence s
    SeqInfo mine = {};        // of sequence s0 + lane
    int my_cost = 0, my_base = 0;
    auto load32 = [&](int first_seq, int base_tile) {
      s0 = first_seq;
      mine = SeqInfo{};
      if (s0 + lane < set.n_seqs) mine = seq_info(set, a.T, s0 + lane);
      if (mine.bad && groups == 1 && cta == 0) set_status(a.status, LILY_STATUS_BAD_LEN);
      my_cost = s0 + lane < set.n_seqs ? cost_of(mine) : 0;
      int inc = my_cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      my_base = base_tile + inc - my_cost;
    };
    // total tiles, and the group that holds this CTA's first
    int total = 0, group = 0, group_base = 0;
    if (groups == 1) {
      load32(0, 0);
      total = __reduce_add_sync(0xffffffffu, my_cost);
    } else {
      for (int g = lane; g < groups; g += 32) total += sums[g];
      total = __reduce_add_sync(0xffffffffu, total);
    }
    const int share = max((total + set.grid - 1) / set.grid, set.min_share);  // tiles per CTA
    const int begin = (int)min((int64_t)share * cta, (int64_t)total);
    const int end = min(begin + share, total);
    int at = begin;
    if (groups > 1) {
      for (int g0 = 0; g0 < groups; g0 += 32) {
        const int c = g0 + lane < groups ? sums[g0 + lane] : 0;
        int inc = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, group_base + inc > begin);
        if (past) {
          const int l = __ffs(past) - 1;
          group = g0 + l;
          group_base += __shfl_sync(0xffffffffu, inc - c, l);
          break;
        }
        group_base += __shfl_sync(0xffffffffu, inc, 31);
      }
      __syncwarp();
      fence_proxy_async_smem();
    }
    // the sequence that holds tile t, from the current group on; false past the last
    auto find = [&](int t) {
      for (;;) {
        const uint32_t in = __ballot_sync(0xffffffffu, my_cost > 0 && my_base + my_cost > t);
        if (in) {
          s = s0 + __ffs(in) - 1;
          s_base = __shfl_sync(0xffffffffu, my_base, s - s0);
          return true;
        }
        if (s0 + 32 >= set.n_seqs) return false;
        load32(s0 + 32, __shfl_sync(0xffffffffu, my_base + my_cost, 31));
      }
    };
    // page indices of the current sequence from page pbase on, and of the next one
    auto first_pages = [&](int seq, int page) {
      const int n = seq < s0 + 32 && seq < set.n_seqs ? __shfl_sync(0xffffffffu, mine.len, seq - s0) : 0;
      const int p = page + lane;
      return n > 0 && p <= (n - 1) >> ps ? set.table[(int64_t)seq * set.table_stride + p] : -1;
    };
    int pseq = -1, pbase = 0, pcache = 0, next_cache = 0;
    if (at < end) {
      if (groups > 1) load32(group * 32, group_base);
      ok = find(at);
    }
    while (ok && at < end) {
      SeqInfo q;
      q.q0 = __shfl_sync(0xffffffffu, mine.q0, s - s0);
      q.qn = __shfl_sync(0xffffffffu, mine.qn, s - s0);
      q.len = __shfl_sync(0xffffffffu, mine.len, s - s0);
      const int nt = tiles_of(q.len), nb = blocks_of(set, a.G, q.qn);
      const int in_seq = (at - s_base) / nt;  // unit of the sequence
      const int t0 = (at - s_base) - in_seq * nt;
      const int nseg = min(nt - t0, end - at);
      const int h = in_seq / nb, blk = in_seq - h * nb;
      const int unit = (s * a.hkv + h) * set.row_blocks + blk;
      const int row0 = blk * C::kRows;
      const int nrows = min(C::kRows, q.qn * a.G - row0);
      const int last = (q.len - 1) >> ps;
      if (s != pseq) {
        // a sequence's first pages came with the one before it, if it was that
        // one's neighbour and starts here
        const bool have = pseq >= 0 && s == pseq + 1 && t0 == 0 && s > s0;
        pbase = (t0 * kTile) >> ps;
        pcache = have ? next_cache : first_pages(s, pbase);
        next_cache = first_pages(s + 1, 0);
        pseq = s;
      }

      const int qb = seg % C::kQBufs;
      ok = wait_warp(qempty(qb), ((seg / C::kQBufs) & 1) ^ 1, &abort_s, a.wait_feed, a.status);
      if (!ok) break;
      if (lane == 0) {
        Desc d;
        d.part = unit + cta;
        d.head = h;
        d.q0 = q.q0;
        d.row0 = row0;
        d.nrows = nrows;
        d.qn = q.qn;
        d.len = q.len;
        d.key0 = t0 * kTile;
        d.tiles = nseg;
        desc[qb] = d;
        mbar_arrive_expect_tx(qfull(qb), nrows * a.D * 2);
      }
      __syncwarp();
      for (int r = lane; r < nrows; r += 32) {
        const int rr = row0 + r;
        const int j = rr / a.G, g = rr - j * a.G;
        const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(q.q0 + j) * a.q_tok +
                              (int64_t)(h * a.G + g) * a.q_head;
        bulk_load(base + C::kQOff + qb * C::kQBytes + r * C::kQPitch, src, a.D * 2, qfull(qb));
        if (t0 == 0 && set.rows_at) {
          // where the merge finds this row's partials: the unit's first, and how many
          const int u0 = s_base + in_seq * nt;
          set.rows_at[(int64_t)(q.q0 + j) * a.hq + h * a.G + g] =
              make_int4(unit + cta, r, (u0 + nt - 1) / share - cta + 1, s);
        }
      }
      ++seg;

      for (int t = 0; t < nseg; ++t) {
        const int k0 = (t0 + t) * kTile;
        const int p0 = k0 >> ps;
        if (p0 < pbase || p0 + pages_per_tile > pbase + 32) {
          pbase = p0;
          pcache = first_pages(s, pbase);
        }
        const int pg = __shfl_sync(0xffffffffu, pcache, min(p0 + min(i, pages_per_tile - 1) - pbase, 31));
        const bool there = i < pages_per_tile && p0 + i <= last;
        const bool good = there && pg >= 0 && pg < a.n_pages;
        const uint32_t good_m = __ballot_sync(0xffffffffu, good);
        if (there && !good) set_status(a.status, LILY_STATUS_BAD_PAGE);
        ok = wait_warp(empty(stage), phase ^ 1, &abort_s, a.wait_feed, a.status);
        if (!ok) break;
        if (lane == 0) {
          unsigned long long m = 0;
          for (int p = 0; p < pages_per_tile; ++p)
            if (good_m >> (p * 2 * halves) & 1u)
              m |= (box_rows == 64 ? ~0ull : ((1ull << box_rows) - 1)) << (p * box_rows);
          if (q.len - k0 < kTile) m &= (1ull << (q.len - k0)) - 1;
          mask_s[stage] = m;
          mbar_arrive_expect_tx(full(stage), __popc(good_m) * box_bytes);
        }
        __syncwarp();
        if (good) {
          const uint32_t dst = base + stage * C::kStageBytes + at_stage;
          const int row = pages_per_tile > 1 ? 0 : k0 & ((1 << ps) - 1);
          if (is_v) tma_load_4d(dst, &mv, hf * 64, row, h, pg, full(stage));
          else tma_load_4d(dst, &mk, hf * 64, row, h, pg, full(stage));
        }
        __syncwarp();
        used |= 1u << stage;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      at += nseg;
      if (ok && at < end && at >= s_base + a.hkv * nb * nt) ok = find(at);
    }
    // no more units
    if (ok) {
      const int qb = seg % C::kQBufs;
      ok = wait_warp(qempty(qb), ((seg / C::kQBufs) & 1) ^ 1, &abort_s, a.wait_feed, a.status);
      if (ok && lane == 0) {
        desc[qb].part = -1;
        mbar_arrive(qfull(qb));
      }
      seg += ok;
    }
    named_sync(2, kThreads);  // all roles have ended
    if (*static_cast<volatile int*>(&abort_s) && lane == 0) {
      // one gave up: this CTA's copies must have landed before its memory goes
      int dead = 0;
      for (int k = max(seg - C::kQBufs, 0); k < seg; ++k)
        mbar_wait(qfull(k % C::kQBufs), (k / C::kQBufs) & 1, &dead, a.status);
      for (int j = 0; j < C::kStages; ++j)
        if (used >> j & 1u) mbar_wait(full(j), j < stage ? phase : phase ^ 1, &dead, a.status);
    }
  } else {
    // ------------------------------------------------------------- compute
    const int wr = warp % WR, wk = warp / WR;
    const int g8 = lane >> 2, c2 = (lane & 3) * 2;
    constexpr int kNT = C::kKeys / 8;  // n-tiles of scores
    const int key_w = wk * C::kKeys;   // this warp's first key in a tile
    const float c = a.scale_log2;
    int stage = 0, phase = 0;
    bool ok = true;
    for (int seg = 0;; ++seg) {
      const int qb = seg % C::kQBufs;
      if (ok) ok = wait_warp(qfull(qb), (seg / C::kQBufs) & 1, &abort_s, a.wait_use, a.status);
      // a warp whose wait gave up takes the others with it, so that none is
      // left at a barrier
      if (!ok && lane == 0) dead_s[seg & 1] = 1;
      named_sync(1, 32 * kWarps);
      if (*reinterpret_cast<volatile int*>(&dead_s[seg & 1])) break;
      const Desc d = desc[qb];
      if (d.part < 0) break;
      const uint32_t qaddr = base + C::kQOff + qb * C::kQBytes +
                             (wr * 16 + (lane & 7) + (ROWS > 8 ? ((lane >> 3) & 1) * 8 : 0)) * C::kQPitch +
                             (lane >> 4) * 16;
      uint32_t qf[C::kQRegs ? DP / 16 : 1][4];
      if (C::kQRegs) {
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks) ldsm4(qaddr + ks * 32, qf[ks]);
      }
      const bool busy = wr * 16 < d.nrows;
      // keys that each of the thread's two rows sees
      const int ra = wr * 16 + g8, rb = ra + 8;
      int lim_a = d.len, lim_b = d.len;
      if (set.causal) {
        lim_a = d.len - d.qn + 1 + (d.row0 + ra) / a.G;
        lim_b = d.len - d.qn + 1 + (d.row0 + rb) / a.G;
      }
      const int lim_all = set.causal ? d.len - d.qn + 1 + d.row0 / a.G : d.len;  // least of the unit
      // largest score, z = c * largest score less softmax_z's powers of two (a
      // rounded number: every exponent and the final log use the same z), sum
      float m_a = -INFINITY, m_b = -INFINITY, z_a = 0.f, z_b = 0.f, l_a = 0.f, l_b = 0.f;
      float o[DP / 8][4];
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

      for (int t = 0; t < d.tiles; ++t) {
        ok = wait_warp(full(stage), phase, &abort_s, a.wait_use, a.status);
        if (!ok) break;
        if (busy) {
          const uint32_t ks_base = base + stage * C::kStageBytes;
          const uint32_t vs_base = ks_base + C::kTileBytes;
          const int k0 = d.key0 + t * kTile;
          const unsigned long long mask = mask_s[stage];
          const bool masked = mask != ~0ull || k0 + kTile > lim_all;

          float sc[kNT][4];
#pragma unroll
          for (int n = 0; n < kNT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
          const int krow = key_w + (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t qt[4];
            if (C::kQRegs) {
#pragma unroll
              for (int e = 0; e < 4; ++e) qt[e] = qf[C::kQRegs ? ks : 0][e];
            } else {
              ldsm4(qaddr + ks * 32, qt);
            }
#pragma unroll
            for (int n = 0; n < kNT; n += 2) {
              uint32_t b[4];
              ldsm4(ks_base + (ks >> 2) * C::kHalfBytes + swz(krow + n * 8, (ks & 3) * 2 + kch), b);
              mma16816<F16>(sc[n], qt, b[0], b[1]);
              mma16816<F16>(sc[n + 1], qt, b[2], b[3]);
            }
          }
          if (masked) {
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = key_w + n * 8 + c2 + e;
                const bool there = mask >> k & 1ull;
                if (!there || k0 + k >= lim_a) sc[n][e] = -INFINITY;
                if (!there || k0 + k >= lim_b) sc[n][2 + e] = -INFINITY;
              }
          }
          float x_a = m_a, x_b = m_b;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            x_a = fmaxf(x_a, fmaxf(sc[n][0], sc[n][1]));
            x_b = fmaxf(x_b, fmaxf(sc[n][2], sc[n][3]));
          }
          x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, 1));
          x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, 1));
          x_a = fmaxf(x_a, __shfl_xor_sync(0xffffffffu, x_a, 2));
          x_b = fmaxf(x_b, __shfl_xor_sync(0xffffffffu, x_b, 2));
          if (__any_sync(0xffffffffu, x_a != m_a || x_b != m_b)) {
            // (a row that has seen nothing keeps z = 0 and has nothing to scale)
            const float y_a = x_a == -INFINITY ? 0.f : softmax_z<F16>(__fmul_rn(x_a, c), 14.f);
            const float y_b = x_b == -INFINITY ? 0.f : softmax_z<F16>(__fmul_rn(x_b, c), 14.f);
            const float f_a = m_a == -INFINITY ? 0.f : ex2(z_a - y_a);
            const float f_b = m_b == -INFINITY ? 0.f : ex2(z_b - y_b);
            l_a *= f_a;
            l_b *= f_b;
#pragma unroll
            for (int i = 0; i < DP / 8; ++i) {
              o[i][0] *= f_a;
              o[i][1] *= f_a;
              o[i][2] *= f_b;
              o[i][3] *= f_b;
            }
            m_a = x_a;
            m_b = x_b;
            z_a = y_a;
            z_b = y_b;
          }
          uint32_t pf[kNT / 2][4];
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            const float p0 = ex2(fmaf(sc[n][0], c, -z_a)), p1 = ex2(fmaf(sc[n][1], c, -z_a));
            const float p2 = ex2(fmaf(sc[n][2], c, -z_b)), p3 = ex2(fmaf(sc[n][3], c, -z_b));
            l_a += p0 + p1;
            l_b += p2 + p3;
            pf[n / 2][(n & 1) * 2] = pack16(p0, p1, F16);
            pf[n / 2][(n & 1) * 2 + 1] = pack16(p2, p3, F16);
          }
          const int vrow = key_w + (lane & 7) + ((lane >> 3) & 1) * 8, vch = lane >> 4;
          auto v_frag = [&](int kb, int i, uint32_t(&b)[4]) {
            ldsm4_t(vs_base + (i >> 2) * C::kHalfBytes + swz(vrow + kb * 16, (i & 3) * 2 + vch), b);
          };
          // the thread's keys of block kb that are in m, as masks of V's two words
          auto v_masks = [&](unsigned long long m, int kb, uint32_t& v0, uint32_t& v1) {
            const uint32_t mb = (uint32_t)(m >> (key_w + kb * 16 + c2));
            v0 = (mb & 1u ? 0xffffu : 0u) | (mb & 2u ? 0xffff0000u : 0u);
            v1 = (mb & 0x100u ? 0xffffu : 0u) | (mb & 0x200u ? 0xffff0000u : 0u);
          };
          // V of keys that a row does not see may hold anything, and 0 * NaN
          // would reach its sum.  Keys that are not there are cut to zero for
          // all rows.  Where a new token's V holds an infinity or NaN that
          // some rows of the tile see and others do not, the tile's product
          // is taken token by token with that token's keys alone.
          bool split = false;
          if (masked && set.causal && k0 + kTile > lim_all) {
            const int seen = max(lim_all - k0, 0);  // keys every row sees
            const unsigned long long some = mask & (seen < kTile ? ~0ull << seen : 0ull);
            constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
#pragma unroll
            for (int kb = 0; kb < kNT / 2; ++kb) {
              uint32_t v0, v1;
              v_masks(some, kb, v0, v1);
              if (!__any_sync(0xffffffffu, (v0 | v1) != 0)) continue;
              for (int i = 0; i < DP / 16; ++i) {
                uint32_t b[4];
                v_frag(kb, i, b);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint32_t w = b[e] & (e & 1 ? v1 : v0);
                  split |= (w & kExp) == kExp || (w >> 16 & kExp) == kExp;
                }
              }
            }
            split = __any_sync(0xffffffffu, split);
          }
          if (!split) {
#pragma unroll
            for (int kb = 0; kb < kNT / 2; ++kb) {
              uint32_t v0 = 0xffffffffu, v1 = 0xffffffffu;
              if (masked) v_masks(mask, kb, v0, v1);
#pragma unroll
              for (int i = 0; i < DP / 16; ++i) {
                uint32_t b[4];
                v_frag(kb, i, b);
                if (masked) {
                  b[0] &= v0;
                  b[1] &= v1;
                  b[2] &= v0;
                  b[3] &= v1;
                }
                mma16816<F16>(o[2 * i], pf[kb], b[0], b[1]);
                mma16816<F16>(o[2 * i + 1], pf[kb], b[2], b[3]);
              }
            }
          } else {
            const int j1 = (d.row0 + wr * 16 + 15) / a.G;
            for (int j = (d.row0 + wr * 16) / a.G; j <= j1; ++j) {
              const int seen = d.len - d.qn + 1 + j - k0;
              const unsigned long long m =
                  mask & (seen <= 0 ? 0ull : seen < kTile ? (1ull << seen) - 1 : ~0ull);
              const bool keep_a = (d.row0 + ra) / a.G == j, keep_b = (d.row0 + rb) / a.G == j;
#pragma unroll
              for (int i = 0; i < DP / 16; ++i) {
                float x[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                  for (int e = 0; e < 4; ++e) x[n][e] = o[2 * i + n][e];
#pragma unroll
                for (int kb = 0; kb < kNT / 2; ++kb) {
                  uint32_t b[4], v0, v1;
                  v_masks(m, kb, v0, v1);
                  v_frag(kb, i, b);
                  mma16816<F16>(x[0], pf[kb], b[0] & v0, b[1] & v1);
                  mma16816<F16>(x[1], pf[kb], b[2] & v0, b[3] & v1);
                }
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  if (keep_a) o[2 * i + n][0] = x[n][0];
                  if (keep_a) o[2 * i + n][1] = x[n][1];
                  if (keep_b) o[2 * i + n][2] = x[n][2];
                  if (keep_b) o[2 * i + n][3] = x[n][3];
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(empty(stage));
          // The first tile's products have used the fragments of Q: only now is
          // the buffer free.  (Released right after the loads were issued, the
          // next rows could land before these were read.)
          if (C::kQRegs && t == 0) mbar_arrive(qempty(qb));
        }
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!C::kQRegs) {
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty(qb));
      }

      l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
      l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
      l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
      float* part_o = set.part_o + (int64_t)d.part * C::kRows * a.D;
      float* part_lse = set.part_lse + (int64_t)d.part * C::kRows;
      auto lse2 = [&](float z, float l) { return l == 0.f ? -INFINITY : z + log2f(l); };
      auto inverse = [](float l) { return l == 0.f ? 0.f : 1.f / l; };
      if constexpr (C::kWK == 1) {
        const float i_a = inverse(l_a), i_b = inverse(l_b);
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          const int col = i * 8 + c2;
          if (col < a.D) {
            if (ra < d.nrows)
              *reinterpret_cast<float2*>(part_o + (int64_t)ra * a.D + col) =
                  make_float2(o[i][0] * i_a, o[i][1] * i_a);
            if (rb < d.nrows)
              *reinterpret_cast<float2*>(part_o + (int64_t)rb * a.D + col) =
                  make_float2(o[i][2] * i_b, o[i][3] * i_b);
          }
        }
        if ((lane & 3) == 0) {
          if (ra < d.nrows) part_lse[ra] = lse2(z_a, l_a);
          if (rb < d.nrows) part_lse[rb] = lse2(z_b, l_b);
        }
      } else {
        // the warps that split the keys put their rows together
        float* red = reinterpret_cast<float*>(smem + C::kRedOff);
        if ((lane & 3) == 0) {
          red_z[warp][g8] = m_a == -INFINITY ? -INFINITY : z_a;
          red_z[warp][g8 + 8] = m_b == -INFINITY ? -INFINITY : z_b;
          red_l[warp][g8] = l_a;
          red_l[warp][g8 + 8] = l_b;
        }
        named_sync(1, 32 * kWarps);
        float M_a = -INFINITY, M_b = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::kWK; ++w) {
          M_a = fmaxf(M_a, red_z[w * WR + wr][g8]);
          M_b = fmaxf(M_b, red_z[w * WR + wr][g8 + 8]);
        }
        const float f_a = M_a == -INFINITY ? 0.f : ex2(red_z[warp][g8] - M_a);
        const float f_b = M_b == -INFINITY ? 0.f : ex2(red_z[warp][g8 + 8] - M_b);
        // this thread's share of the sums: four columns of one row
        constexpr int kQuads = C::kRedCols / 4;
        // (word of a row's column: pieces of 8 columns swizzled by the row)
        auto word = [&](int w, int r, int col) {
          return (w * C::kRedRows + r) * C::kRedCols + (col ^ ((r & (C::kRedCols / 8 - 1)) << 3));
        };
        static_assert(C::kRows * kQuads == 32 * kWarps, "one quad of columns per thread");
        const int orow = threadIdx.x / kQuads, oq = threadIdx.x % kQuads;
        const int ob = orow >> 4, oi = orow & 15;  // row block, row in it
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < C::kWK; ++w) M = fmaxf(M, red_z[w * WR + ob][oi]);
#pragma unroll
        for (int w = 0; w < C::kWK; ++w)
          if (M != -INFINITY) L += red_l[w * WR + ob][oi] * ex2(red_z[w * WR + ob][oi] - M);
          else L += red_l[w * WR + ob][oi];  // 0, or NaN
        const float inv = inverse(L);
        if (oq == 0 && orow < d.nrows) part_lse[orow] = lse2(M == -INFINITY ? 0.f : M, L);
#pragma unroll
        for (int cb = 0; cb < DP / C::kRedCols; ++cb) {
#pragma unroll
          for (int n = 0; n < C::kRedCols / 8; ++n) {
            const int i = cb * (C::kRedCols / 8) + n;
            *reinterpret_cast<float2*>(red + word(warp, g8, n * 8 + c2)) =
                make_float2(o[i][0] * f_a, o[i][1] * f_a);
            if (ROWS > 8)
              *reinterpret_cast<float2*>(red + word(warp, g8 + 8, n * 8 + c2)) =
                  make_float2(o[i][2] * f_b, o[i][3] * f_b);
          }
          named_sync(1, 32 * kWarps);
          const int col = cb * C::kRedCols + oq * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < C::kWK; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(red + word(w * WR + ob, oi, oq * 4));
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          if (orow < d.nrows && col < a.D)
            *reinterpret_cast<float4*>(part_o + (int64_t)orow * a.D + col) =
                make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          named_sync(1, 32 * kWarps);
        }
      }
    }
    named_sync(2, kThreads);  // (see the producer's end)
  }
}

// One launch for the prefix (set pa: the first pa.grid CTAs) and the batch's own
// pages (pb), or for one set alone (pb.grid 0).  first: it follows the call's
// predecessor and waits for it; else it follows the prefix's launch on the
// tensor cores, which has waited, and only ends after it (so that the merge,
// which waits for this launch, sees both).
template <int DP, int RA, int RB, bool F16>
__global__ void __launch_bounds__(kThreads, Cfg<DP, RA>::kOcc)
    attn_keys_kernel(const AttnArgs a, const AttnSet pa, const AttnSet pb,
                     const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                     bool first) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Fixed fx;
  const int cta = (int)blockIdx.x;
  if (RA == RB) {
    const bool second = cta >= pa.grid;
    keys_body<DP, RA, F16>(a, second ? pb : pa, mk, mv, first, second ? cta - pa.grid : cta, smem, fx);
  } else if (cta < pa.grid) {
    keys_body<DP, RA, F16>(a, pa, mk, mv, first, cta, smem, fx);
  } else {
    keys_body<DP, RB, F16>(a, pb, mk, mv, first, cta - pa.grid, smem, fx);
  }
  if (!first) pdl_wait();
}

struct KeysLaunch {
  const AttnArgs& a;
  const AttnSet &pa, &pb;
  const CUtensorMap &mk, &mv;
  bool first;
  cudaStream_t s;
};
template <int DP, int RA, int RB, bool F16>
cudaError_t launch_keys_as(const KeysLaunch& l) {
  auto kern = attn_keys_kernel<DP, RA, RB, F16>;
  constexpr int kBytes =
      Cfg<DP, RA>::kBytes > Cfg<DP, RB>::kBytes ? Cfg<DP, RA>::kBytes : Cfg<DP, RB>::kBytes;
  const cudaError_t e = ensure_smem_attr((const void*)kern, kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(l.pa.grid + l.pb.grid), dim3(kThreads), kBytes, l.s, l.a, l.pa, l.pb,
                    l.mk, l.mv, l.first);
}
template <int DP, bool F16>
cudaError_t launch_keys_dp(const KeysLaunch& l) {
  // (the pairs of rows that attn_api.cu plans)
  const int ra = l.pa.rows, rb = l.pb.grid ? l.pb.rows : ra;
  if (ra == 8) return launch_keys_as<DP, 8, 8, F16>(l);
  if (ra == 16) return rb == 8 ? launch_keys_as<DP, 16, 8, F16>(l) : launch_keys_as<DP, 16, 16, F16>(l);
  if (ra == 32) return rb == 8 ? launch_keys_as<DP, 32, 8, F16>(l) : launch_keys_as<DP, 32, 32, F16>(l);
  return rb == 8    ? launch_keys_as<DP, 64, 8, F16>(l)
         : rb == 16 ? launch_keys_as<DP, 64, 16, F16>(l)
                    : launch_keys_as<DP, 64, 64, F16>(l);
}

template <bool F16>
cudaError_t launch_keys_type(const KeysLaunch& l) {
  const int dp = padded_dim(l.a.D);
  return dp == 64    ? launch_keys_dp<64, F16>(l)
         : dp == 128 ? launch_keys_dp<128, F16>(l)
                     : launch_keys_dp<256, F16>(l);
}

}  // namespace
}  // namespace lily
