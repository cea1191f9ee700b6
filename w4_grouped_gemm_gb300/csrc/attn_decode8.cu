// attn_decode8.cu -- attention of new tokens over an 8-bit paged cache
// (lily_attn_decode8): e4m3 codes with a scale for each token and head.
//
//   z = c (q . k_code) k_scale,  out = sum 2^(z - m) v_scale v_code / sum 2^(z - m)
// HBM bounds it: a key and value of D dimensions are 2 D + 8 bytes and meet the few
// rows of their KV head.  A code is exact in fp16, so codes become operands of
// mma.sync by a conversion alone and the scales meet the products: k_scale the
// score, v_scale the probability (fp32, then rounded to fp16 for its product).
//
// A unit is a sequence, a KV head and up to 8 query rows (row r = token
// r / G, head h*G + r % G).  The units' tiles of keys form one list in which every CTA
// takes an equal run, found by adding up the lengths on the device; a unit that two CTAs
// share leaves partials, which a second kernel joins.  A warp of each CTA brings tiles by
// TMA across the ends of units; in a tile each of four others has keys of its own and a
// softmax state of its own, and the four are joined at a unit's end.  (128 sequences of
// up to 4096 keys: 127 us where each warp brought its keys by cp.async of 16 bytes, whose
// instructions were a third of all and waited for one another; 121 by TMA of its own,
// half of each step then being addresses and page indices.)
//
// Keys and dimensions are the MMAs' 16 rows and query rows their 8 columns (scores
// [keys][rows], outputs [dimensions][rows]), since a KV head often has eight query
// heads or fewer: with the query as 16 rows half of all products, registers and
// exponentials were of rows that do not exist (950 instructions per 32 keys, 150 us for
// 128 sequences of up to 4096 keys).  Nothing is transposed in shared memory: an MMA's
// k index may be any order of the dimensions (scores) or keys (output) as long as both
// operands agree.  For scores a lane reads 16 consecutive dimensions of two keys and
// q's lanes hold the same; for outputs it reads 8 or 16 consecutive dimensions of four
// keys and pairs the keys' bytes; the probabilities change sides by movmatrix.
//
// The exponentials' reference is a row's maximum at the time when a score last passed
// it by 4: most steps then need neither the maximum nor a rescaling, and a vote tells.
// fp16 for the probabilities: 2^(z - m) v_scale, at most 2^4 times the largest v_scale,
// is held 2^(10 - e) times as large, e the exponent of the largest v_scale so far, so
// that it ends below 2^15 and all bits are kept from 2^-24 of the reference on.  e may be
// that of any fp32 number: powers of two by it are taken in two factors where one would
// leave fp32's range, and partial outputs are divided by their sums.  The rounding is what
// an operand of 16 bits costs (a second product with what it took off would be half of all
// MMAs more): with fp16 outputs the error against 64 bits is 2.9e-4, where fp32 throughout
// gives 2.1e-4, and bf16 outputs round away more.  q is brought to fp16's range by a power of
// two for each row.
//
// Measured: 4 sequences of up to 131072 keys, 2 KV heads of 256, 84 us, 5.9 TB/s; 128 of
// up to 4096, 98 us, 5.9 TB/s; one of 301 keys 8.3 us, half of it the look-ups before
// the first tile (lengths, pages, keys one after another) and the joining.  A tile is some
// 1800 cycles of a CTA, a unit's end and next beginning some 4000, which bounds short
// sequences (256 of up to 300 keys: 40 us).
#include <algorithm>
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "decode8.cuh"
#include "stream.cuh"

namespace lily {
namespace {

constexpr int kWarps = 4;              // that compute
constexpr int kUsers = 32 * kWarps;    // their threads
constexpr int kThreads = kUsers + 32;  // and the warp that brings tiles
constexpr int kRows = kDecode8Rows;    // query rows of a unit
constexpr float kAhead = 4.f;          // log2 of how far a score may be ahead of the reference

// Per padded head size: keys of a warp in a tile, CTAs on an SM, stages.
template <int DP>
struct Cfg {
  static constexpr int kKeys = DP == 256 ? 16 : 32;
  static constexpr int kBlocks = kKeys / 16;
  static constexpr int kTile = kKeys * kWarps;
  static constexpr int kCtas = DP == 64 ? 3 : 2;
  static constexpr int kStages = DP == 64 ? 4 : 3;
  static constexpr int kWide = DP == 64 ? 64 : 128;  // bytes of a row in a box
  static constexpr int kKV = kTile * DP;             // bytes of K, and of V, in a stage
  static constexpr int kStage = 2 * kKV;
  // beside a stage: scales of K and V, q (in a unit's first stage), which blocks are there
  static constexpr int kQ = 2 * kTile * 4, kThere = kQ + kRows * DP * 2, kSide = kThere + 16;
  static constexpr int kMT = DP / 16;  // row tiles of the output
  static constexpr size_t kSmem = 1024 + (size_t)kStages * (kStage + kSide);
  static_assert(kStage >= kWarps * kMT * 512 && 2 * kKeys * DP >= kMT * 512, "a warp's keys hold its outputs, for joining");
  static_assert((kSmem + 1024 + 128 + 16 * kStages + 128 * kRows) * kCtas <= 228 * 1024, "the CTAs fit on an SM");
};

// Where 16-byte piece c (of D) of a key's row lies among a stage's K or V, as the
// copies' 128- or 64-byte swizzle puts it.
template <int DP, int TILE>
__device__ __forceinline__ int place(int key, int c) {
  if (DP == 64) return key * 64 + (c ^ (key >> 1 & 3)) * 16;
  return (c >> 3) * (TILE * 128) + key * 128 + ((c ^ key) & 7) * 16;
}
// Row i of an MMA's 16 keys is key in_block(i) of a block: rows 2j and 2j + 1 are four
// keys apart, and those of the four j differ by the swizzle's upper bits, so that both
// the reads of K (two keys' four pieces) and of V (four keys' two pieces) meet every
// bank once.
__device__ __forceinline__ int in_block(int i) {
  const int j = i >> 1 & 3;
  return ((2 * j + (j >> 1)) ^ (i & 1) << 2) + (i & 8);
}

// Two e4m3 codes as a pair of fp16.
__device__ __forceinline__ uint32_t codes_f16(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// An 8 x 8 tile of 16-bit elements, lane 4 i + j with row i's 2 j and 2 j + 1, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

struct Cursor {
  int seq, h, rb, tile;         // of the next tile (h: of the KV heads that are this CTA's)
  int q0, qn, len, rbs, tiles;  // the sequence's
  int3 ahead;                   // the next one's start, end and length, looked up while this one is gone through
  __device__ __forceinline__ int3 look(const AttnSet& s, int i) const {
    if (i >= s.n_seqs) return make_int3(0, 0, 0);
    return s.q_start ? make_int3(s.q_start[i], s.q_start[i + 1], s.lens[i])
                     : make_int3(i * s.max_q_len, (i + 1) * s.max_q_len, s.lens[i]);
  }
  __device__ __forceinline__ void load(const AttnSet& s, const Decode8Args& a, int tile_keys, int3 is) {
    SeqInfo i = {is.x, 0, is.z, false};
    hold_tokens(i, s, a.T, is.y);
    hold_len(i, s);
    q0 = i.q0;
    qn = i.qn;
    len = i.len;
    rbs = (qn * a.G + kRows - 1) / kRows;
    tiles = max(1, (len + tile_keys - 1) / tile_keys);
    ahead = look(s, seq + 1);
  }
  // To the next tile of the list; true where a new unit begins.
  __device__ __forceinline__ bool next(const AttnSet& s, const Decode8Args& a, int tile_keys) {
    if (++tile < tiles) return false;
    tile = 0;
    if (++rb < rbs) return true;
    rb = 0;
    if ((h += a.side) < a.hkv) return true;
    h = blockIdx.x % a.side;
    do {
      if (++seq >= s.n_seqs) return true;
      load(s, a, tile_keys, ahead);
    } while (rbs == 0);
    return true;
  }
};

// The token of row r of a unit in its sequence, and its head.
__device__ __forceinline__ void row_at(const Decode8Args& a, const Cursor& c, int r, int& j, int& head) {
  const int rr = c.rb * kRows + r;
  j = a.G == 1 ? rr : __umulhi(rr, a.G_inverse);  // rr / G
  head = c.h * a.G + rr - j * a.G;
}

// Of `total` tiles in equal runs, total i / grid (as two products that 32 bits hold).
__device__ __forceinline__ int first_tile(int total, int grid, int i) {
  const uint32_t each = (uint32_t)total / grid, rest = total - each * grid;
  return (int)(each * i + rest * i / grid);
}

// 2^e in two factors, for e of -252 to 254.
__device__ __forceinline__ float2 power2(int e) {
  const int half = e >> 1;
  return make_float2(__uint_as_float((uint32_t)(127 + half) << 23), __uint_as_float((uint32_t)(127 + e - half) << 23));
}

// Tries of the wait for the last copies: 2 s.
constexpr uint32_t kDrainTries = (uint32_t)(2000000000ull / kTryNs);

template <int DP>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kCtas)
    decode8_kernel(const Decode8Args a, const AttnSet s, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<DP>;
  constexpr int kMT = C::kMT;
  extern __shared__ uint8_t smem_any[];
  uint8_t* smem = smem_any + (-(int)smem_u32(smem_any) & 1023);
  __shared__ int scan[kWarps];
  __shared__ int gave_up;
  __shared__ int4 found;
  __shared__ float4 stat[2][kWarps][kRows];  // of a unit and of the next
  __shared__ uint64_t full_bars[C::kStages], empty_bars[C::kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem), sides = ring + C::kStages * C::kStage;
  const uint32_t full = smem_u32(full_bars), empty = smem_u32(empty_bars);
  if (threadIdx.x == 0) {
    gave_up = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full + 8 * i, 33);  // the bytes' sender, and the 32 lanes' smaller copies
      mbar_init(empty + 8 * i, kWarps);
    }
    fence_mbar_init();
  }
  pdl_wait();
  pdl_trigger();

  // ---- this CTA's run of the list
  int total, grid, start, end;  // tiles of a head; groups of CTAs with a tile or more; this one's
  Cursor in;
  {
    const int per = (s.n_seqs + kUsers - 1) / kUsers;  // (none for the last warp)
    const int s0 = min(s.n_seqs, threadIdx.x * per), s1 = min(s.n_seqs, s0 + per);
    auto weight = [&](int i) {
      const SeqInfo q = seq_info(s, a.T, i);
      if (q.bad && blockIdx.x == 0) set_status(a.status, LILY_STATUS_BAD_LEN);
      return a.hkv / a.side * ((q.qn * a.G + kRows - 1) / kRows) * max(1, (q.len + C::kTile - 1) / C::kTile);
    };
    const int first = s0 < s1 ? weight(s0) : 0;
    int own = first;
    for (int i = s0 + 1; i < s1; ++i) own += weight(i);
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31 && warp < kWarps) scan[warp] = upto;
    __syncthreads();
    total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += scan[w];
      total += scan[w];
    }
    const int group = blockIdx.x / a.side;
    grid = min((int)gridDim.x / a.side, total);
    start = end = 0;
    if (group < grid) {
      start = first_tile(total, grid, group);
      end = first_tile(total, grid, group + 1);
    }
    if (start < end && start >= upto - own && start < upto) {
      int at = upto - own, i = s0;
      for (;; ++i) {
        const int w = i == s0 ? first : weight(i);
        if (start < at + w) break;
        at += w;
      }
      found = make_int4(i, start - at, 0, 0);
    }
    __syncthreads();
    if (threadIdx.x == 0 && start >= end) a.split[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
    if (start >= end) return;
    in.seq = found.x;
    in.load(s, a, C::kTile, in.look(s, in.seq));
    const int unit = found.y / in.tiles;
    in.tile = found.y - unit * in.tiles;
    in.h = unit / in.rbs;
    in.rb = unit - in.h * in.rbs;
    in.h = in.h * a.side + blockIdx.x % a.side;
  }

  if (warp == kWarps) {
    // ---- bringing tiles
    // Page indices lie in registers, a lane each, 32 at a time: those at hand, the 32
    // after them, the sequence's first and the next sequence's first.  All are looked up
    // long before they are needed.
    int window, pages, pages_after, first_pages, next_pages;
    auto pages_of = [&](int seq, int len, int from) {
      const int p = from + lane;
      return seq < s.n_seqs && p < (len + (1 << a.page_shift) - 1) >> a.page_shift
                 ? s.table[(int64_t)seq * s.table_stride + p]
                 : 0;
    };
    auto next_first = [&]() {  // of the sequence after this one, whose length is known (held to what it may be)
      return pages_of(in.seq + 1, min(max(in.ahead.z, 0), s.max_len), 0);
    };
    window = (in.tile * C::kTile >> a.page_shift) & ~31;
    pages = pages_of(in.seq, in.len, window);
    pages_after = pages_of(in.seq, in.len, window + 32);
    first_pages = window ? pages_of(in.seq, in.len, 0) : pages;
    next_pages = next_first();

    // a lane's block of 16 keys of the tile, and its box of box_keys if it begins one
    const int box_keys = min(1 << a.page_shift, C::kTile);
    const bool boxes = lane < C::kTile / 16 && 16 * lane % box_keys == 0;
    bool fresh = true;       // the next tile is its unit's first in this CTA
    uint32_t used = 0, bit = 0;  // stages filled so far; the parity of the last filling
    int slot = 0;
    for (int j = end - start; j > 0; --j) {
      if (used >> slot & 1) {
        if (!wait_warp(empty + 8 * slot, bit >> slot & 1, &gave_up, a.wait_feed, a.status)) break;
        bit ^= 1u << slot;
      }
      used |= 1u << slot;
      const uint32_t st = ring + slot * C::kStage, side = sides + slot * C::kSide, bar = full + 8 * slot;
      const int k0 = in.tile * C::kTile;
      int page;
      {
        const int p = ((k0 + 16 * lane) >> a.page_shift) - window;
        const int p1 = __shfl_sync(0xffffffffu, pages, p & 31), p2 = __shfl_sync(0xffffffffu, pages_after, p & 31);
        page = p < 32 ? p1 : p2;
      }
      const bool held = lane < C::kTile / 16 && k0 + 16 * lane < in.len;
      const bool is = held && (uint32_t)page < (uint32_t)a.n_pages;
      if (held && !is) set_status(a.status, LILY_STATUS_BAD_PAGE);
      const uint32_t there = __ballot_sync(0xffffffffu, is), sent = __popc(__ballot_sync(0xffffffffu, is && boxes));
      if (lane == 0) {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(side + C::kThere), "r"(there) : "memory");
        mbar_arrive_expect_tx(bar, sent * box_keys * 2 * DP);
      }
      __syncwarp();
      if (is && boxes) {
        const int row0 = (k0 + 16 * lane) & ((1 << a.page_shift) - 1);
        const uint32_t to = st + 16 * lane * C::kWide;
#pragma unroll
        for (int w = 0; w < DP / C::kWide; ++w) {
          tma_load_4d(to + w * C::kTile * C::kWide, &mk, w * C::kWide, row0, in.h, page, bar);
          tma_load_4d(to + w * C::kTile * C::kWide + C::kKV, &mv, w * C::kWide, row0, in.h, page, bar);
        }
      }
      // scales: a key a lane
#pragma unroll
      for (int i = 0; i < C::kTile / 32; ++i) {
        const int key = lane + 32 * i, block = key >> 4;
        const int64_t at = (int64_t)__shfl_sync(0xffffffffu, page, block) * a.s_page + in.h * a.s_head +
                           ((k0 + key) & ((1 << a.page_shift) - 1)) * a.s_tok;
        const bool one = (there >> block & 1) && k0 + key < in.len;
        cp_async4(side + key * 4, one ? a.ks + at : a.ks, one ? 4 : 0);
        cp_async4(side + C::kTile * 4 + key * 4, one ? a.vs + at : a.vs, one ? 4 : 0);
      }
      if (fresh) {
        constexpr int kOfRow = DP / 8, kAll = kRows * kOfRow;  // pieces of 16 bytes
        const int rows = in.qn * a.G - in.rb * kRows;
#pragma unroll
        for (int i = 0; i < kAll / 32; ++i) {
          const int at = lane + 32 * i, piece = at % kOfRow, r = at / kOfRow;
          int jt, head;
          row_at(a, in, r, jt, head);
          const bool row = r < rows && piece * 8 < a.D;
          const uint16_t* src = static_cast<const uint16_t*>(a.q);
          if (row) src += (int64_t)(in.q0 + jt) * a.q_tok + (int64_t)head * a.q_head + piece * 8;
          cp_async16(side + C::kQ + at * 16, src, row ? 16 : 0);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
      const int from = in.seq;
      fresh = in.next(s, a, C::kTile);
      if (fresh) {
        if (in.seq != from) {
          // (sequences without query tokens are passed over)
          first_pages = in.seq == from + 1 ? next_pages : pages_of(in.seq, in.len, 0);
          next_pages = next_first();
        }
        window = 0;
        pages = first_pages;
        pages_after = pages_of(in.seq, in.len, 32);
      } else if ((in.tile * C::kTile) >> a.page_shift >= window + 32) {
        window += 32;
        pages = pages_after;
        pages_after = pages_of(in.seq, in.len, window + 32);
      }
      if (++slot == C::kStages) slot = 0;
    }
    // until all copies have landed: nothing ends before them, whichever wait ran out
    for (int i = 0; i < C::kStages; ++i)
      if (used >> i & 1) wait_warp(full + 8 * i, bit >> i & 1, &gave_up, kDrainTries, a.status);
    return;
  }
  Cursor out = in;
  const int g = lane >> 2, t = lane & 3;

  // ---- units
  // keys of a lane in a block: rows g and g + 8 of an MMA of scores, and of the outputs'
  // k index 2t, 2t + 1 and 8 on
  const int key_of_lane = in_block(g), v_key = in_block(2 * t);
  uint32_t phase = 0;  // of the stages' barriers, one bit each
  bool dead = false;   // a wait ran out: this warp computes no more
  const int my_keys = warp * C::kKeys;  // of a tile, from here on
  int slot = 0, left = end - start;
  bool whole = out.tile == 0;  // this CTA has the unit from its first tile on
  int odd = 0;                 // units gone through, mod 2
  int head_split = 0;          // the unit that goes on in the next CTA began here
  while (left > 0) {
    const int rows = min(kRows, out.qn * a.G - out.rb * kRows);
    auto wait_tile = [&]() {
      if (!dead && !wait_warp(full + 8 * slot, phase >> slot & 1, &gave_up, a.wait_use, a.status)) dead = true;
    };
    wait_tile();
    // q, as fp16 in the order in which a lane reads a key's dimensions: row g of each block
    uint32_t q[DP / 64][4][2];
    float qs[2];   // what takes the products of rows 2t and 2t + 1 to z
    int limit[2];  // keys that they see
    {
      const uint32_t from = sides + slot * C::kSide + C::kQ + g * DP * 2;
      uint32_t sizes = 0;
#pragma unroll
      for (int d = 0; d < DP / 64; ++d)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 v = lds128(from + (64 * d + 16 * t + 8 * p) * 2);
          q[d][2 * p][0] = v.x, q[d][2 * p][1] = v.y, q[d][2 * p + 1][0] = v.z, q[d][2 * p + 1][1] = v.w;
        }
#pragma unroll
      for (int d = 0; d < DP / 64; ++d)
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const uint32_t w = q[d][p >> 1][p & 1];
          sizes = __vmaxu2(sizes, w & 0x7FFF7FFFu);  // (of either type: the bits' order is the sizes')
        }
      uint32_t most = __float_as_uint(lo16_f32(max(sizes & 0xFFFFu, sizes >> 16), a.f16));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // its largest size to 2^14 .. 2^15 (a row that is no number: as it is)
      const int e = (int)(most >> 23);
      const int up = e == 0 || e == 255 ? 0 : min(14 - (e - 127), 126);
      const float f = __uint_as_float((uint32_t)(127 + up) << 23);
      const float to_z = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
      for (int d = 0; d < DP / 64; ++d)
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          uint32_t& w = q[d][p >> 1][p & 1];
          w = pack16(lo16_f32(w, a.f16) * f, hi16_f32(w, a.f16) * f, true);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qs[i] = __shfl_sync(0xffffffffu, to_z, (2 * t + i) * 4);
        int j, head;
        row_at(a, out, 2 * t + i, j, head);
        // (rows that do not exist see all: nothing of them is stored)
        limit[i] = 2 * t + i < rows ? max(0, out.len - out.qn + j + 1) : INT_MAX;
      }
    }
    int first, first_head;
    row_at(a, out, 0, first, first_head);
    const int seen_by_all = max(0, out.len - out.qn + first + 1);
    float o[kMT][4];
    float m[2], l[2];  // rows 2t and 2t + 1: the reference, and this lane's part of the sum
#pragma unroll
    for (int n = 0; n < kMT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    int ev = -127;                 // exponent of the largest v_scale so far
    float2 fv = power2(10 - ev);
    float next_v = 0x1p-126f;      // 2^(ev + 1): a scale of that size moves ev

    const int n_tiles = min(left, out.tiles - out.tile);
#pragma unroll 1
    for (int it = 0; it < n_tiles; ++it) {
      if (it) {
        // (the unit's last stage is kept for the joining)
        __syncwarp();
        if (lane == 0 && !dead) mbar_arrive(empty + 8 * slot);
        phase ^= 1u << slot;
        if (++slot == C::kStages) slot = 0;
        wait_tile();
      }
      const uint32_t st = ring + slot * C::kStage, side = sides + slot * C::kSide + my_keys * 4;
      const int k0 = (out.tile + it) * C::kTile + my_keys;
      const uint32_t there = lds32(sides + slot * C::kSide + C::kThere) >> (my_keys / 16) & ((1u << C::kBlocks) - 1);
      if (there == 0 || dead) continue;
      const uint32_t kst = st + my_keys * C::kWide;
      if (k0 + C::kKeys > out.len) {
        // V past the last key, whatever lies there: zeros (a probability of 0 takes no NaN)
        const int held = out.len - k0;
        for (int i = lane; i < (C::kKeys - held) * (DP / 16); i += 32)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                           kst + C::kKV + place<DP, C::kTile>(held + i / (DP / 16), i % (DP / 16))),
                       "r"(0)
                       : "memory");
        fence_proxy_async_smem();
        __syncwarp();
      }
      auto step = [&](auto all_seen) {
      constexpr bool plain = decltype(all_seen)::value;  // all keys are there and seen by every row
      float z[C::kBlocks][4];  // key key_of_lane: rows 2t, 2t + 1; key + 8: the same
      float vs[C::kBlocks][2];
      bool ahead = false;
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b) {
        z[b][0] = z[b][1] = z[b][2] = z[b][3] = 0.f;
#pragma unroll
        for (int d = 0; d < DP / 64; ++d) {
          const uint32_t at = kst + 16 * b * C::kWide;
          const uint4 k1 = lds128(at + place<DP, C::kTile>(key_of_lane, 4 * d + t));
          const uint4 k2 = lds128(at + place<DP, C::kTile>(key_of_lane + 8, 4 * d + t));
          const uint32_t w1[4] = {k1.x, k1.y, k1.z, k1.w}, w2[4] = {k2.x, k2.y, k2.z, k2.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = codes_f16((uint16_t)w1[i]), a1 = codes_f16((uint16_t)w2[i]);
            const uint32_t a2 = codes_f16((uint16_t)(w1[i] >> 16)), a3 = codes_f16((uint16_t)(w2[i] >> 16));
            mma16816<true>(z[b], a0, a1, a2, a3, q[d][i][0], q[d][i][1]);
          }
        }
        const uint32_t ks_at = side + (16 * b + key_of_lane) * 4;
        const float ks[2] = {__uint_as_float(lds32(ks_at)), __uint_as_float(lds32(ks_at + 32))};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float& v = z[b][i];
          v *= ks[i >> 1] * qs[i & 1];
          if (!plain) {
            const int key = k0 + 16 * b + key_of_lane + (i >> 1) * 8;
            if (!(there >> b & 1) || key >= limit[i & 1]) v = -INFINITY;
          }
          ahead |= v > m[i & 1] + kAhead;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          vs[b][i] = __uint_as_float(lds32(side + C::kTile * 4 + (16 * b + key_of_lane + 8 * i) * 4));
          ahead |= (plain || (there >> b & 1)) && fabsf(vs[b][i]) >= next_v;
        }
      }
      if (__any_sync(0xffffffffu, ahead)) {
        // the largest v_scale that is a number (lanes past the keys: their own again)
        const int key = lane % C::kKeys;
        uint32_t vmax = lds32(side + C::kTile * 4 + key * 4) & 0x7FFFFFFFu;
        vmax = __reduce_max_sync(0xffffffffu, (there >> (key >> 4) & 1) && vmax < 0x7F800000u ? vmax : 0u);
        const int e_new = max(ev, (int)(vmax >> 23) - 127);
        const float down = __uint_as_float((uint32_t)max(127 - (e_new - ev), 0) << 23);
        ev = e_new;
        fv = power2(10 - ev);
        next_v = __uint_as_float((uint32_t)(ev + 128) << 23);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = m[i];
#pragma unroll
          for (int b = 0; b < C::kBlocks; ++b) top = fmaxf(top, fmaxf(z[b][i], z[b][i + 2]));
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
          const float f = top == -INFINITY ? 1.f : ex2(m[i] - top);
          m[i] = top;
          l[i] *= f;
#pragma unroll
          for (int n = 0; n < kMT; ++n) {
            o[n][i] *= f * down;
            o[n][i + 2] *= f * down;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < C::kBlocks; ++b) {
        if (!plain && !(there >> b & 1)) continue;  // (what lies there is another tile's)
        vs[b][0] = vs[b][0] * fv.x * fv.y;
        vs[b][1] = vs[b][1] * fv.x * fv.y;
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = ex2(z[b][i] - m[i & 1]);
          if (plain) {
            l[i & 1] += e[i];
            e[i] *= vs[b][i >> 1];
          } else {
            // (a key that the row does not see has no part in it, whatever its scale)
            const bool seen = z[b][i] != -INFINITY;
            l[i & 1] += seen ? e[i] : 0.f;
            e[i] = seen ? e[i] * vs[b][i >> 1] : 0.f;
          }
        }
        const uint32_t p0 = transposed(pack16(e[0], e[1], true)), p1 = transposed(pack16(e[2], e[3], true));
        // four keys' words of the same dimensions: pairs of keys for each dimension
        auto four = [&](int n, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
          const uint32_t x0 = prmt(v0, v1, 0x5140), x1 = prmt(v2, v3, 0x5140);
          const uint32_t y0 = prmt(v0, v1, 0x7362), y1 = prmt(v2, v3, 0x7362);
          const uint32_t a0 = codes_f16((uint16_t)x0), a1 = codes_f16((uint16_t)(x0 >> 16));
          const uint32_t a2 = codes_f16((uint16_t)x1), a3 = codes_f16((uint16_t)(x1 >> 16));
          const uint32_t b0 = codes_f16((uint16_t)y0), b1 = codes_f16((uint16_t)(y0 >> 16));
          const uint32_t b2 = codes_f16((uint16_t)y1), b3 = codes_f16((uint16_t)(y1 >> 16));
          mma16816<true>(o[n], a0, a1, a2, a3, p0, p1);
          mma16816<true>(o[n + 1], b0, b1, b2, b3, p0, p1);
        };
        const uint32_t vb = kst + C::kKV + 16 * b * C::kWide;
        const int v_keys[4] = {v_key, v_key ^ 4, v_key + 8, (v_key ^ 4) + 8};
        if (DP == 64) {
          uint2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = lds64(vb + place<DP, C::kTile>(v_keys[i], g >> 1) + (g & 1) * 8);
          four(0, v[0].x, v[1].x, v[2].x, v[3].x);
          four(2, v[0].y, v[1].y, v[2].y, v[3].y);
        } else {
#pragma unroll
          for (int h = 0; h < DP / 128; ++h) {
            uint4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lds128(vb + place<DP, C::kTile>(v_keys[i], 8 * h + g));
            four(8 * h, v[0].x, v[1].x, v[2].x, v[3].x);
            four(8 * h + 2, v[0].y, v[1].y, v[2].y, v[3].y);
            four(8 * h + 4, v[0].z, v[1].z, v[2].z, v[3].z);
            four(8 * h + 6, v[0].w, v[1].w, v[2].w, v[3].w);
          }
        }
      }
      };
      if (there == (1u << C::kBlocks) - 1 && k0 + C::kKeys <= seen_by_all)
        step(std::true_type{});
      else
        step(std::false_type{});
    }

    // ---- the four warps' states into one: references, sums and the outputs' factors, and
    // the outputs as they are, each warp's where its own keys of the unit's last tile were
    // (a warp that is ahead may be at the next unit's end: its states lie beside these)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
      if (g == 0) stat[odd][warp][2 * t + i] = make_float4(m[i], l[i], __int_as_float(ev), 0.f);
    }
    auto join = [&](int w, int n) {
      constexpr int kPer = C::kKeys * C::kWide / 512, kAcross = DP / C::kWide;  // tiles of 512 bytes; halves of a row
      const int part = n / kPer;
      return reinterpret_cast<float4*>(smem + slot * C::kStage + part % kAcross * (C::kTile * C::kWide) + part / kAcross * C::kKV +
                                       w * (C::kKeys * C::kWide) + n % kPer * 512) + lane;
    };
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kMT; ++n) *join(warp, n) = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
    named_sync(1, kUsers);
    float to[2], sum[2], by_warp[kWarps][2];
    int e_all = -127;  // the largest of the warps' exponents, which the outputs' sum is held by
#pragma unroll
    for (int k = 0; k < kWarps; ++k) e_all = max(e_all, __float_as_int(stat[odd][k][0].z));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float4 w[kWarps];
      to[i] = -INFINITY;
      sum[i] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        w[k] = stat[odd][k][2 * t + i];
        to[i] = fmaxf(to[i], w[k].x);
      }
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        // (a maximum of -infinity with a sum: a NaN)
        const float f = w[k].x == -INFINITY ? (w[k].y == 0.f ? 0.f : 1.f) : ex2(w[k].x - to[i]);
        sum[i] += w[k].y * f;
        const float down = __uint_as_float((uint32_t)max(127 - (e_all - __float_as_int(w[k].z)), 0) << 23);
        by_warp[k][i] = w[k].x == -INFINITY ? (w[k].y == 0.f ? 0.f : w[k].y) : f * down;
      }
    }
    odd ^= 1;
    const bool ends = out.tile + n_tiles == out.tiles;
    const bool done = whole && ends;
    const int part = 2 * blockIdx.x + (whole ? 1 : 0);
    uint16_t* dst[2];  // of rows 2t and 2t + 1
    const float2 held = power2(e_all - 10);
    float by[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int j, head;
      row_at(a, out, 2 * t + i, j, head);
      dst[i] = static_cast<uint16_t*>(a.out) + (int64_t)(out.q0 + j) * a.out_tok + (int64_t)head * a.out_head;
      by[i] = sum[i] == 0.f ? 0.f : held.x / sum[i];
    }
#pragma unroll
    for (int n = warp; n < kMT; n += kWarps) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *join(w, n);
        v.x += x.x * by_warp[w][0], v.y += x.y * by_warp[w][1], v.z += x.z * by_warp[w][0], v.w += x.w * by_warp[w][1];
      }
      v.x = v.x * by[0] * held.y, v.y = v.y * by[1] * held.y, v.z = v.z * by[0] * held.y, v.w = v.w * by[1] * held.y;
      // dimensions d and d + 1 of both rows
      const int d = DP == 64 ? 8 * g + 2 * n : 128 * (n >> 3) + 16 * g + 2 * (n & 7);
      if (!done) {
        a.part_o[((size_t)part * kMT + n) * 32 + lane] = v;
      } else if (d < a.D) {
        if (2 * t < rows) *reinterpret_cast<uint32_t*>(dst[0] + d) = pack16(v.x, v.z, a.f16);
        if (2 * t + 1 < rows) *reinterpret_cast<uint32_t*>(dst[1] + d) = pack16(v.y, v.w, a.f16);
      }
    }
    if (warp == 0 && g == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 2 * t + i;
        if (!done) {
          a.part_ml[part * kRows + row] = make_float2(to[i], sum[i]);
        } else if (a.lse && row < rows) {
          int j, head;
          row_at(a, out, row, j, head);
          a.lse[(int64_t)(out.q0 + j) * a.hq + head] =
              sum[i] == 0.f ? -INFINITY : (to[i] + log2f(sum[i])) * 0.6931471805599453f;
        }
      }
      if (whole && !ends && t == 0) {
        // the CTAs that the unit's other tiles lie in
        const int last = start + (end - start - left) + out.tiles - 1;
        const int64_t c = (((int64_t)last + 1) * grid - 1) / total;
        a.split[2 * blockIdx.x] = make_int4((int)c - (int)(blockIdx.x / a.side) + 1, out.q0, rows, out.rb);
        a.split[2 * blockIdx.x + 1] = make_int4(out.h, 0, 0, 0);
      }
    }
    if (whole && !ends) head_split = 1;
    left -= n_tiles;
    out.tile += n_tiles - 1;
    out.next(s, a, C::kTile);
    whole = true;
    // the stage goes back once every warp has read its share
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && !dead) mbar_arrive(empty + 8 * slot);
    phase ^= 1u << slot;
    if (++slot == C::kStages) slot = 0;
  }
  if (threadIdx.x == 0 && !head_split) a.split[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
}

// The partials of the units that CTAs share.  Block (c, y): the unit that began in
// CTA c and went on, its tile y (32 lanes of float4, as the kernel above holds them),
// whose partials the block's warps take in turn.  It lets the kernel after it start only
// at its end: where the next call's CTAs of the kernel above came to SMs one by one, while
// merges still ran there, they no longer read neighbouring heads at the same time (64
// sequences of up to 8192 keys, 8 KV heads of 64: 86 us, so 58).
template <int DP, int kMergeWarps>
__global__ void __launch_bounds__(32 * kMergeWarps) decode8_merge_kernel(const Decode8Args a) {
  constexpr int kMT = DP / 16, kAcross = 32 * kMergeWarps / kRows;
  extern __shared__ float weight[];  // [parts][rows]
  __shared__ float4 acc[kMergeWarps][32];
  __shared__ float part_max[kMergeWarps][kRows], part_sum[kMergeWarps][kRows];
  pdl_wait();
  const int4 s0 = a.split[2 * blockIdx.x];
  const int parts = min(s0.x, ((int)gridDim.x - (int)blockIdx.x - 1) / a.side + 1);
  if (parts < 1) return;
  const int h = a.split[2 * blockIdx.x + 1].x, q0 = s0.y, rows = s0.z, rb = s0.w;
  auto part_of = [&](int p) { return 2 * (blockIdx.x + p * a.side) + (p == 0 ? 1 : 0); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this thread's share of the outputs, on the way while the weights are found
  constexpr int kFirst = 4;
  float4 x[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i)
    if (warp + i * kMergeWarps < parts)
      x[i] = a.part_o[((size_t)part_of(warp + i * kMergeWarps) * kMT + blockIdx.y) * 32 + lane];
  // a thread per row and every kAcross-th partial: the references' maximum, then weights
  const int row = threadIdx.x % kRows;
  float to = -INFINITY;
  for (int p = threadIdx.x / kRows; p < parts; p += kAcross) to = fmaxf(to, a.part_ml[part_of(p) * kRows + row].x);
#pragma unroll
  for (int o = kRows; o < 32; o <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
  if (lane < kRows) part_max[warp][row] = to;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) to = fmaxf(to, part_max[w][row]);
  float sum = 0.f;
  for (int p = threadIdx.x / kRows; p < parts; p += kAcross) {
    const float2 ml = a.part_ml[part_of(p) * kRows + row];
    // (a maximum of -infinity with a sum: a NaN, and so is the weight)
    const float w = ml.x == -INFINITY ? ml.y : ex2(ml.x - to) * ml.y;
    weight[p * kRows + row] = w;
    sum += w;
  }
#pragma unroll
  for (int o = kRows; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < kRows) part_sum[warp][row] = sum;
  __syncthreads();
  const int n = blockIdx.y, g = lane >> 2, t = lane & 3;
  const float* w0 = weight + 2 * t;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  // (shares of rows 2t and 2t + 1: a sum of values near fp32's largest would not fit it)
  float total[2] = {0.f, 0.f}, by[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) total[i] += part_sum[w][2 * t + i];
    by[i] = total[i] == 0.f ? 0.f : 1.f / total[i];
  }
  auto add = [&](const float4& y, int p) {
    float2 w = *reinterpret_cast<const float2*>(w0 + p * kRows);
    w.x *= by[0], w.y *= by[1];
    v.x += w.x * y.x, v.y += w.y * y.y, v.z += w.x * y.z, v.w += w.y * y.w;
  };
#pragma unroll
  for (int i = 0; i < kFirst; ++i)
    if (warp + i * kMergeWarps < parts) add(x[i], warp + i * kMergeWarps);
#pragma unroll 4
  for (int p = warp + kFirst * kMergeWarps; p < parts; p += kMergeWarps)
    add(a.part_o[((size_t)part_of(p) * kMT + blockIdx.y) * 32 + lane], p);
  acc[warp][lane] = v;
  __syncthreads();
  if (warp) return;
#pragma unroll
  for (int i = 1; i < kMergeWarps; ++i) {
    const float4 y = acc[i][lane];
    v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
  }
  const int d = DP == 64 ? 8 * g + 2 * n : 128 * (n >> 3) + 16 * g + 2 * (n & 7);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = 2 * t + i;
    if (at >= rows) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) top = fmaxf(top, part_max[w][at]);
    const int rr = rb * kRows + at, j = rr / a.G, head = h * a.G + rr - j * a.G;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + (int64_t)(q0 + j) * a.out_tok + (int64_t)head * a.out_head;
    if (d < a.D)
      *reinterpret_cast<uint32_t*>(dst + d) = i ? pack16(v.y, v.w, a.f16) : pack16(v.x, v.z, a.f16);
    if (a.lse && n == 0 && g == 0)
      a.lse[(int64_t)(q0 + j) * a.hq + head] = total[i] == 0.f ? -INFINITY : (top + log2f(total[i])) * 0.6931471805599453f;
  }
}

}  // namespace

int decode8_tile(int D) {
  const int dp = padded_dim(D);
  return dp == 64 ? Cfg<64>::kTile : dp == 128 ? Cfg<128>::kTile : Cfg<256>::kTile;
}

// Bytes of a row and tokens of the copies' boxes.
void decode8_box(int D, int page, uint32_t& bytes, uint32_t& tokens) {
  bytes = padded_dim(D) == 64 ? 64 : 128;
  tokens = std::min(page, decode8_tile(D));
}

// KV heads side by side: all of them up to 16, else the most that divide them.
int decode8_side(int hkv) {
  int side = std::min(hkv, 16);
  while (hkv % side) --side;
  return side;
}

cudaError_t launch_decode8(const Decode8Args& a, const AttnSet& s, const CUtensorMap& mk, const CUtensorMap& mv,
                           int64_t units, int64_t tiles, int sms, cudaStream_t st) {
  auto launch = [&](auto dp) {
    constexpr int DP = decltype(dp)::value;
    using C = Cfg<DP>;
    // whole groups of `side` CTAs
    const int most = std::min(sms * C::kCtas, kDecode8Grid) / a.side * a.side;
    const int grid = (int)std::min<int64_t>(tiles, most);
    auto kern = decode8_kernel<DP>;
    prof_begin(K_ATTN_KEYS, st);
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), C::kSmem);
    if (e == cudaSuccess) e = launch_pdl(kern, dim3(grid), dim3(kThreads), C::kSmem, st, a, s, mk, mv);
    prof_end(K_ATTN_KEYS, st);
    if (e != cudaSuccess || grid == a.side) return e;
    prof_begin(K_ATTN_MERGE, st);
    // Eight warps a block where a unit may lie in more than 32 CTAs (one sequence of 131072
    // keys, 2 KV heads of 128: 23.7 us, by four 26.3), else four (128 sequences of up to
    // 4096 keys: 98.9, by eight 101.9, by sixteen 111)
    const dim3 blocks(grid, C::kMT);
    const size_t weights = (size_t)grid * kRows * 4;
    e = grid > 32 * units ? launch_pdl(decode8_merge_kernel<DP, 8>, blocks, dim3(256), weights, st, a)
                          : launch_pdl(decode8_merge_kernel<DP, 4>, blocks, dim3(128), weights, st, a);
    prof_end(K_ATTN_MERGE, st);
    return e;
  };
  const int dp = padded_dim(a.D);
  return dp == 64    ? launch(std::integral_constant<int, 64>{})
         : dp == 128 ? launch(std::integral_constant<int, 128>{})
                     : launch(std::integral_constant<int, 256>{});
}

}  // namespace lily
