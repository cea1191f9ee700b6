// attn_tc.cu -- partial outputs over the shared prefix on the 5th-generation
// tensor cores, for batches with more than 64 query rows per KV head.
//
// Every key of the prefix meets all rows = tokens x query heads per KV head,
// 4 D flop per key and row against 4 D bytes per key: past some 290 rows the
// tensor cores bound the prefix, and mma.sync reaches a fraction of their
// rate.  A CTA takes 256 rows (two streams of 128) or 128, and a run of
// 128-key tiles:
//   S = Q K^T      A = Q, B = K from shared memory, S in tensor memory
//   P = 2^(c S - z) one thread per row: 128 scores in registers, no shuffles;
//                  P overwrites S in tensor memory, rounded to the cache's 16
//                  bits, which the MMA takes (a wider type has half its rate);
//                  its sum is of the unrounded ones
//   O += P V       A = P from tensor memory, B = V from shared memory as it
//                  lies (keys x dimensions: the N-major operand layout)
// z follows the row's largest score, but O is rescaled only when it grew by
// more than 2^8 (a published way of attention on this generation): until then P is
// at most 256 times larger, which costs no precision, and the rescale (a pass over
// O in tensor memory) stays rare.
//
// Warps 0 and 2 bring K and V (TMA boxes of 64 dimensions and one page) into a
// ring of slots; warps 1 and 3 issue the MMAs of a stream each; two groups of
// four warps take the softmax of one stream each, so that one stream's softmax
// runs under the other's MMAs.  Rows over 128: the streams are the two row
// blocks and share every K and V tile ("paired"; L2 feeds 32 bytes per clock
// and SM at D = 128).  Up to 128 rows: the streams take alternate tiles of the
// same rows and leave two partials.  Heads over 128 fill tensor memory with
// one stream's output (256 columns) and two score buffers; one softmax group
// alternates between them.
//
// Measured: 256 sequences of 8 rows on each of 4 KV heads behind 32768 keys,
// D = 128 (137 GFLOP): 139 us with the own pages and the merge, 0.99 PFLOP/s.  A
// tile of 256 rows takes some 3000 cycles, 2200 of which the MMAs need; the rest
// is the chain from a score to its probability (wait, load, exponentials, store,
// arrive), which two streams cover in part.
#include "attn.cuh"

namespace lily {
namespace {

constexpr int kKeys = 128;           // keys of a tile
constexpr int kMasks = 16;           // tiles whose key masks are kept
constexpr int kCtrlWarps = 4;        // K, MMAs of stream 0, V, MMAs of stream 1
constexpr float kLag = 8.f;          // powers of two by which z may be behind the largest score
constexpr float kUp = 7.f;           // of softmax_z: kLag + kUp and a rounding stay within fp16

// DP: head dimension rounded up to 64, 128 or 256.
template <int DP>
struct Tc {
  static constexpr int kGroups = DP <= 128 ? 2 : 1;           // softmax groups = streams
  static constexpr int kThreads = 32 * (kCtrlWarps + 4 * kGroups);
  // ring slots of 128 keys x 64 or 128 dimensions of K, or as many bytes of
  // whole keys of V: a tile is one slot of each, or two where D > 128.  (With
  // slots of 16 KB the MMA warp spent as long on their barriers as on the MMAs.)
  static constexpr int kSlot = DP == 64 ? 16384 : 32768;
  static constexpr int kSlots = DP == 64 ? 11 : 5;
  static constexpr int kSlotBlocks = DP == 64 ? 1 : 2;        // blocks of 64 dimensions of K
  static constexpr int kVKeys = kSlot / (DP * 2);             // keys of a V slot
  static constexpr int kVSlots = kKeys / kVKeys;              // V slots of a tile
  static constexpr int kQTile = 128 * DP * 2;                 // 128 rows, blocks of 64 dimensions
  static constexpr int kQBytes = kGroups * kQTile;
  static constexpr int kBytes = kQBytes + kSlots * kSlot;
  // tensor memory columns
  static constexpr int kS = 0;        // + 128 * buffer; P in the first 64 columns
  static constexpr int kO = 256;      // + DP * stream
  static_assert(kO + kGroups * DP <= 512, "tensor memory");
};

// Shared-memory descriptors with the 128-byte swizzle, as a constant high word
// (stride offset 1024 between groups of 8 rows, version, swizzle) and a low
// word (address, leading offset) that advances by adding bytes / 16.
//   K-major (Q, K): rows of 64 elements along K; the leading offset is unused.
//   N-major (V as it lies): rows of 64 elements of N, one row per key; blocks
//   of 64 N are `block` bytes apart.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_n(uint32_t saddr, uint32_t block) {
  return saddr >> 4 | (block >> 4) << 16;
}
// D (+)= A B^T with A in shared memory / in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescHi), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two floats in a 64-bit register, and packed arithmetic on them.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// Keeps every use of r after the point (the wait of the load that filled it).
__device__ __forceinline__ void tie(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// A CTA's run of the units' tiles, unit by unit (every role walks it alike).
struct Run {
  int at, end, nt;
  int unit, t0, n;  // current unit, its first tile here and their number
  int before;       // tiles of the CTA's earlier units
  __device__ bool next() {
    if (at >= end) return false;
    before += n;
    unit = at / nt;
    t0 = at - unit * nt;
    n = min(nt - t0, end - at);
    at += n;
    return true;
  }
};

template <int DP, bool F16>
__global__ void __launch_bounds__(Tc<DP>::kThreads, 1)
    attn_prefix_tc_kernel(const AttnArgs a, const TcArgs p, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv) {
  using C = Tc<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * C::kSlots + 11];
  __shared__ __align__(16) uint32_t mask_s[kMasks][4];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;
  // 2 | parity of the last filling of a slot that copies were sent to, and of
  // `land`: what a CTA that gives up waits for before its memory goes
  __shared__ uint32_t armed_s[C::kSlots + 1];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t slots = base + C::kQBytes;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (C::kSlots + i); };
  const uint32_t bar1 = bar0 + 8 * 2 * C::kSlots;
  auto q_full = [&](int g) { return bar1 + 8 * g; };        // rows of Q in place
  auto s_full = [&](int b) { return bar1 + 8 * (2 + b); };  // scores in buffer b
  // probabilities in buffer b (four softmax warps), and the turn to use them
  auto p_full = [&](int b) { return bar1 + 8 * (4 + b); };
  // product added to the output: one barrier per stream; where one stream
  // alternates between two buffers, one per buffer.  (A wait names a phase by
  // its parity alone, so it must never be two phases off.  A stream with a
  // buffer to itself has its scores after the product before; an alternating
  // one hands P over while the product before may still run.)
  auto o_full = [&](int i) { return bar1 + 8 * (6 + i); };
  const uint32_t land = bar1 + 8 * 8;
  auto drain = [&](int g) { return bar1 + 8 * (9 + g); };  // a stream's MMAs are done

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < C::kSlots; ++i) {
        mbar_init(full(i), 1);
        mbar_init(empty(i), C::kGroups);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(q_full(i), 4);
        mbar_init(s_full(i), 1);
        mbar_init(p_full(i), 5);
        mbar_init(o_full(i), 1);
      }
      mbar_init(land, 1);
      for (int i = 0; i < 2; ++i) mbar_init(drain(i), 1);
      for (int i = 0; i <= C::kSlots; ++i) armed_s[i] = 0;
      fence_mbar_init();
      abort_s = 0;
      prefetch_tensormap(&mk);
      prefetch_tensormap(&mv);
    }
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_s), 512);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;

  // ring position: slot and the parity of its current filling
  struct Pos {
    int slot, par;
    __device__ void skip(int n) {
      slot += n;
      if (slot >= C::kSlots) {
        slot -= C::kSlots;
        par ^= 1;
      }
    }
  };
  Run run;
  run.nt = p.tiles;
  run.n = run.before = 0;
  run.at = (int)min((long long)p.share * blockIdx.x, (long long)p.total);
  run.end = (int)min((long long)p.share * (blockIdx.x + 1), (long long)p.total);
  const int rows_all = a.T * a.G;
  const int blocks = (a.D + 63) / 64;  // of 64 dimensions
  const int k_slots = (blocks + C::kSlotBlocks - 1) / C::kSlotBlocks;  // K slots of a tile
  const bool paired = p.paired != 0;

  if (warp < kCtrlWarps) {
    if (C::kGroups == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == 0 || warp == 2) {
      // --------------------------------------------------------- producers
      // One warp for K, one for V: a tile's boxes go out from one lane each
      // (lane -> slot c of the tile, first key, first dimension), all lanes
      // polling their own slot.  One warp for both, slot by slot, took 3800
      // cycles a tile and held the MMAs up.
      const bool is_v = warp == 2;
      const int ps = a.page_shift;
      const int n_slots = is_v ? C::kVSlots : k_slots;
      const int slot_keys = is_v ? C::kVKeys : kKeys;
      const int box_rows = min(slot_keys, 1 << ps);
      const int per_block = slot_keys / box_rows;      // boxes of 64 dimensions
      const int wide = is_v ? blocks : C::kSlotBlocks;  // blocks of a slot
      const int per_slot = per_block * wide;            // boxes; at most 32 of a tile
      const int c = lane / per_slot, in_slot = lane - c * per_slot;
      const int box = in_slot / wide, blk = in_slot - box * wide;
      const int dim = 64 * (blk + (is_v ? 0 : c * wide));
      const int key = (is_v ? c * slot_keys : 0) + box * box_rows;
      const uint32_t at_slot = (blk * slot_keys + box * box_rows) * 128;
      const bool active = c < n_slots && dim < a.D;
      const uint32_t all_boxes = __ballot_sync(0xffffffffu, active);
      const uint32_t slot_boxes = per_slot == 32 ? ~0u : (1u << per_slot) - 1;  // of slot 0
      const int last = (p.len - 1) >> ps;
      const int span = (kKeys + (1 << ps) - 1) >> ps;  // pages of a tile
      int c_base = -1, c_page = 0;                     // page indices, 32 at a time
      int land_par = 0;
      bool ok = true;
      Pos cur = {0, 0};
      auto load = [&](int h, int t) {
        const int k0 = t * kKeys, first = k0 >> ps;
        if (c_base < 0 || first < c_base || first + span > c_base + 32) {
          c_base = first;
          c_page = first + lane <= last ? p.pages[first + lane] : -1;
        }
        const int idx = (k0 + min(key, kKeys - 1)) >> ps;
        const int pg = __shfl_sync(0xffffffffu, c_page, idx - c_base);
        const bool there = active && idx <= last;
        const bool good = there && pg >= 0 && pg < a.n_pages;
        const uint32_t good_m = __ballot_sync(0xffffffffu, good);
        const bool whole = good_m == all_boxes && k0 + kKeys <= p.len;
        uint32_t* mask = mask_s[(run.before + t - run.t0) & (kMasks - 1)];
        uint32_t w = 0xffffffffu;
        if (!whole) {
          // valid keys: lane l answers for keys 4l .. 4l+3 (of one page)
          if (there && !good) set_status(a.status, LILY_STATUS_BAD_PAGE);
          const int kl = k0 + 4 * lane;
          const int pl = __shfl_sync(0xffffffffu, c_page, (kl >> ps) - c_base);
          const int left = pl < 0 || pl >= a.n_pages ? 0 : p.len - kl;
          w = (left <= 0 ? 0u : left >= 4 ? 15u : (1u << left) - 1) << (4 * (lane & 7));
          w |= __shfl_xor_sync(0xffffffffu, w, 1);
          w |= __shfl_xor_sync(0xffffffffu, w, 2);
          w |= __shfl_xor_sync(0xffffffffu, w, 4);
        }
        if (!is_v && (lane & 7) == 0) mask[lane >> 3] = w;
        __syncwarp();
        Pos mine = cur;
        mine.skip(min(c, n_slots - 1));
        const uint32_t slot = slots + mine.slot * C::kSlot;
        // (slot by slot: a warp's slots are up to a whole ring apart, and a wait
        // for a slot holds only once the filling before is known to be done)
        if (C::kVSlots > 1) ok = wait_warp(empty(cur.slot), cur.par ^ 1, &abort_s, a.wait_feed, a.status);
        if (!ok || !(ok = wait_warp(empty(mine.slot), mine.par ^ 1, &abort_s, a.wait_feed, a.status))) return;
        const bool cut = is_v && !whole;
        const uint32_t bar = cut ? land : full(mine.slot);
        if (cut ? lane == 0 : active && in_slot == 0) {
          mbar_arrive_expect_tx(bar, __popc(cut ? good_m : good_m >> lane & slot_boxes) * box_rows * 128);
          armed_s[cut ? C::kSlots : mine.slot] = 2u | (cut ? land_par : mine.par);
        }
        __syncwarp();
        if (good) {
          const int row = (k0 + key) & ((1 << ps) - 1);
          if (is_v) tma_load_4d(slot + at_slot, &mv, dim, row, h, pg, bar);
          else tma_load_4d(slot + at_slot, &mk, dim, row, h, pg, bar);
        }
        __syncwarp();
        if (cut) {
          // V of keys that are not there may hold anything, and 0 * NaN
          // would reach every row: it is set to zero before the MMAs see it
          if (!(ok = wait_warp(land, land_par, &abort_s, a.wait_feed, a.status))) return;
          land_par ^= 1;
          // (a key per lane, its pieces in an order that spreads the lanes over
          // the banks; key after key by the whole warp took 11 us of a short
          // prefix's 25)
#pragma unroll
          for (int i = 0; i < kKeys / 32; ++i) {
            const int k = 32 * i + lane;
            if (__shfl_sync(0xffffffffu, w, 8 * i) >> lane & 1u) continue;
            Pos z = cur;
            z.skip(k / C::kVKeys);
            const uint32_t at = slots + z.slot * C::kSlot + k % C::kVKeys * 128;
            for (int x = 0; x < blocks * 8; ++x)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               at + (x >> 3) * (C::kVKeys * 128) + ((x + lane) & 7) * 16),
                           "r"(0)
                           : "memory");
          }
          __syncwarp();
          fence_proxy_async_smem();
          __syncwarp();
          if (active && in_slot == 0) {
            armed_s[mine.slot] = 2u | mine.par;
            mbar_arrive(full(mine.slot));
          }
        }
      };
      // in the order in which the MMAs take the slots
      auto step = [&](bool v, int h, int t) {
        if (!ok) return;
        if (v == is_v) load(h, t);
        cur.skip(v ? C::kVSlots : k_slots);
      };
      while (ok && run.next()) {
        const int h = run.unit / p.row_blocks;
        const int ahead = paired ? 1 : 2;
        for (int t = 0; t < min(ahead, run.n); ++t) step(false, h, run.t0 + t);
        for (int t = 0; t < run.n && ok; ++t) {
          step(true, h, run.t0 + t);
          if (t + ahead < run.n) step(false, h, run.t0 + t + ahead);
        }
      }
    } else if (warp == 1 || C::kGroups == 2) {
      // ------------------------------------- MMA issuers: one warp per stream
      // (Issuing blocks until the tensor pipe takes the MMA, and each barrier
      // costs some 180 cycles; with one warp for both streams the pipe idled a
      // third of the time.)
      const int g = warp >> 1;
      const uint32_t id_qk = F16 ? idesc_f16_f32(128, 128) : idesc_bf16_f32(128, 128);
      const uint32_t id_pv = (F16 ? idesc_f16_f32(128, blocks * 64) : idesc_bf16_f32(128, blocks * 64)) |
                             1u << 16;  // B is N-major
      Pos cur = {0, 0};    // slot of the current step
      uint32_t p_par = 0;  // parity of buffer b's P: bit b
      int q_par = 0;
      bool ok = true;
      auto take = [&](Pos x, int n) {  // the n slots from x on have arrived
        for (int j = 0; j < n && ok; ++j, x.skip(1))
          ok = wait_warp(full(x.slot), x.par, &abort_s, a.wait_feed, a.status);
      };
      // Two streams issue by turns, P V of a tile and Q K of the next together:
      // their MMAs and softmaxes so stay out of step, each under the other's.
      // (Left alone they fall into step and the pipe idles during both
      // softmaxes.)  The turn is the fifth arrival on p_full, from the warp that
      // issued before, sent before its last MMAs; a first product, or a stream
      // alone, gives it to itself.  (On a barrier of its own it cost 250 cycles
      // more of each product's way.)
      bool turns = false;
      int next_buf = -1;  // buffer whose product follows, -1: none
      // (the next three: by one elected thread)
      // the n slots from x on are free once this stream's MMAs so far are done
      // and the other stream's warp has let them go too
      auto release = [&](Pos x, int n) {
        for (int j = 0; j < n; ++j, x.skip(1)) mma_commit(empty(x.slot));
      };
      // S[buf] = Q K^T with K in the slots from x on; passes the turn
      auto qk = [&](int buf, Pos x) {
        const Pos k_pos = x;
        const uint32_t q = desc_k(base + g * C::kQTile), d = tmem + C::kS + 128 * buf;
        uint32_t k = desc_k(slots + x.slot * C::kSlot);
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
          if (c < blocks) {
            if (c && c % C::kSlotBlocks == 0) {
              x.skip(1);
              k = desc_k(slots + x.slot * C::kSlot);
            }
            if (next_buf >= 0 && c == blocks - 1) mbar_arrive(p_full(next_buf));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_ss(d, q + c * (128 * 128 / 16) + 2 * i,
                     k + c % C::kSlotBlocks * (128 * 128 / 16) + 2 * i, id_qk, (c | i) != 0);
          }
        mma_commit(s_full(buf));
        release(k_pos, k_slots);
      };
      // O (+)= P[buf] V with V in the slots from x on
      auto pv = [&](int buf, Pos x, bool fresh) {
        const Pos v_pos = x;
        const uint32_t d = tmem + C::kO + DP * g, pt = tmem + C::kS + 128 * buf;
        uint32_t v = desc_n(slots + x.slot * C::kSlot, C::kVKeys * 128);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k && k % (C::kVKeys / 16) == 0) {
            x.skip(1);
            v = desc_n(slots + x.slot * C::kSlot, C::kVKeys * 128);
          }
          mma_ts(d, pt + k * 8, v + k % (C::kVKeys / 16) * (16 * 128 / 16), id_pv, k != 0 || !fresh);
        }
        mma_commit(o_full(C::kGroups == 2 ? g : buf));
        release(v_pos, C::kVSlots);
      };
      while (ok && run.next()) {
        const int left = rows_all - run.unit % p.row_blocks * p.block_rows;
        const int n = run.n;
        const bool shared = paired && left > 128;
        turns = C::kGroups == 2 && (paired ? shared : n > 1);
        if (!(ok = wait_warp(q_full(g), q_par, &abort_s, a.wait_feed, a.status))) break;
        q_par ^= 1;
        // the ring's order: K of the first `ahead` tiles, then V of a tile and K
        // of the tile `ahead` after it; alternating streams take every other tile
        const int ahead = paired ? 1 : 2;
        // A warp follows the ring over the tiles that are not its stream's, too:
        // running ahead it would take an old filling of a slot for a later one.
        // (It lets them go behind its own MMAs: the producers count on slots
        // becoming free in the ring's order.)
        auto pass = [&](int m) {
          take(cur, m);
          if (ok && elect_one()) release(cur, m);
          __syncwarp();
          cur.skip(m);
        };
        if (g == 1 && !turns) {
          // nothing here for this stream: its softmax warps wait for this, so
          // that they do not run ahead either
          for (int t = 0; t < min(ahead, n) && ok; ++t) pass(k_slots);
          for (int t = 0; t < n && ok; ++t) {
            pass(C::kVSlots);
            if (t + ahead < n) pass(k_slots);
          }
          if (lane == 0) mbar_arrive(s_full(1));
          continue;
        }
        const bool every = paired || C::kGroups == 1;
        for (int t = 0; t < min(ahead, n) && ok; ++t) {
          if (!every && t != g) {
            pass(k_slots);
            continue;
          }
          take(cur, k_slots);
          if (!ok) break;
          tc_fence_after();
          next_buf = -1;
          if (elect_one()) qk(paired ? g : t, cur);
          __syncwarp();
          cur.skip(k_slots);
        }
        for (int t = 0; t < n && ok; ++t) {
          const bool more = t + ahead < n;
          if (!every && (t & 1) != g) {
            pass(C::kVSlots);
            if (more) pass(k_slots);
            continue;
          }
          Pos nk = cur;
          nk.skip(C::kVSlots);
          const int buf = paired ? g : t & 1;
          // the first product of all, and every one of a stream alone
          if ((!turns || (t == 0 && g == 0)) && lane == 0) mbar_arrive(p_full(buf));
          next_buf = !turns ? -1 : paired ? (g == 0 ? 1 : more ? 0 : -1) : t + 1 < n ? buf ^ 1 : -1;
          take(cur, C::kVSlots);
          if (more && C::kGroups == 2) take(nk, k_slots);
          ok = ok && wait_warp(p_full(buf), p_par >> buf & 1u, &abort_s, a.wait_feed, a.status);
          p_par ^= 1u << buf;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            pv(buf, cur, paired || C::kGroups == 1 ? t == 0 : t < 2);
            if (more && C::kGroups == 2) qk(buf, nk);
            else if (next_buf >= 0) mbar_arrive(p_full(next_buf));
          }
          __syncwarp();
          if (more && C::kGroups == 1) {  // (the ring holds less than two tiles)
            take(nk, k_slots);
            if (!ok) break;
            tc_fence_after();
            next_buf = -1;
            if (elect_one()) qk(buf, nk);
            __syncwarp();
          }
          cur = nk;
          if (more) cur.skip(k_slots);
        }
      }
      // The MMAs must be done before tensor memory goes: the softmax warps see to
      // that, but not where they have given up.
      if (elect_one()) mma_commit(drain(g));
      __syncwarp();
      int dead = 0;
      if (lane == 0) mbar_wait(drain(g), 0, &dead, a.status);
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------------- softmax
    if (C::kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int g = (warp - kCtrlWarps) >> 2;          // stream
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;  // tensor memory lane field
    const float c = a.scale_log2;
    uint32_t s_par = 0;  // parity of buffer b's scores: bit b
    uint32_t o_par = 0;  // parity of the next product's phase on o_full(i): bit i
    int o_last = 0;      // barrier of the last product
    bool ok = true;
    while (ok && run.next()) {
      const int h = run.unit / p.row_blocks;
      const int row0 = run.unit % p.row_blocks * p.block_rows + (paired ? g * 128 : 0);
      const int nrows = min(128, rows_all - row0);  // may be 0 or less
      // rows of Q, 16 bytes at a time, swizzled; zeros past the rows and past D
      // (a warp brings its own 32 rows, eight per thread, whose loads of two blocks
      // are in flight together)
      {
        const int e = lane & 7;
        int64_t at[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = quad * 32 + i * 4 + (lane >> 3);
          const int rr = row0 + r, j = rr / a.G, gg = rr - j * a.G;
          at[i] = r < nrows ? (int64_t)j * a.q_tok + (int64_t)(h * a.G + gg) * a.q_head : -1;
        }
        for (int k = 0; k < blocks; k += 2) {
          uint4 v[2][8];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int col = (k + m) * 64 + e * 8;
              v[m][i] = make_uint4(0, 0, 0, 0);
              if (at[i] >= 0 && col < a.D)
                v[m][i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at[i] + col);
            }
#pragma unroll
          for (int m = 0; m < 2; ++m)
            if (k + m < blocks)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = quad * 32 + i * 4 + (lane >> 3);
                *reinterpret_cast<uint4*>(smem + g * C::kQTile + (k + m) * 128 * 128 + r * 128 +
                                          ((e ^ (r & 7)) << 4)) = v[m][i];
              }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(g));

      float z = 0.f, l = 0.f;
      bool have = false;  // z follows a score
      bool any = false;  // a product has been started
      const bool idle = paired && nrows <= 0;
      const int step = !paired && C::kGroups == 2 ? 2 : 1;
      for (int t = step == 2 ? g : 0; t < run.n && !idle; t += step) {
        const int b = paired ? g : t & 1;
        ok = wait_warp(s_full(b), s_par >> b & 1u, &abort_s, a.wait_use, a.status);
        if (!ok) break;
        s_par ^= 1u << b;
        const uint4 mw = *reinterpret_cast<const uint4*>(mask_s[(run.before + t) & (kMasks - 1)]);
        tc_fence_after();
        uint32_t s[4][32];
        const uint32_t st = tmem + lanes + C::kS + 128 * b;
        const uint32_t mask[4] = {mw.x, mw.y, mw.z, mw.w};
        const bool masked = (mw.x & mw.y & mw.z & mw.w) != 0xffffffffu;
        auto cut = [&](int i) {  // keys that are not there
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!(mask[i] >> j & 1u)) s[i][j] = 0xff800000u;  // -inf
        };
        const uint64_t c2 = pair(c, c);
        uint64_t z2, sum[4];
        uint32_t w[32];
        // P of one half (packed arithmetic) and its sums
        auto exps = [&](int half) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const uint32_t* v = s[2 * half + i];
              float p0, p1;
              unpair(fma2(pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), c2, z2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[(j / 2) & 3] = add2(sum[(j / 2) & 3], pair(p0, p1));
              w[16 * i + j / 2] = pack16(p0, p1, F16);
            }
        };
        tmem_ld32(st, s[0]);
        tmem_ld32(st + 32, s[1]);
        tmem_ld_wait();
        tie(s[0]);
        tie(s[1]);
        tmem_ld32(st + 64, s[2]);
        tmem_ld32(st + 96, s[3]);
        if (masked) {
          cut(0);
          cut(1);
        }
        // The first half is taken with the z of the tiles before, under which
        // the tile's maximum is found; only where that shows z to be more than
        // 2^8 behind (always at first) z moves, O is rescaled and the half taken
        // again.
        for (int pass = 0;; ++pass) {
          z2 = pair(-z, -z);
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] = 0;
          exps(0);
          if (pass) break;
          tmem_ld_wait();
          tie(s[2]);
          tie(s[3]);
          if (masked) {
            cut(2);
            cut(3);
          }
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              y[i] = max3(y[i], __uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1]));
              y[4 + i] = max3(y[4 + i], __uint_as_float(s[i][j + 2]), __uint_as_float(s[i][j + 3]));
            }
          const float zx =
              __fmul_rn(max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), fmaxf(y[6], y[7])), c);
          // (!(<=): infinities and NaN too)
          const float most = F16 && fabsf(z) < kFineZ ? kLag + kUp : kLag;
          const bool grow = have ? !(zx - z <= most) : zx != -INFINITY;
          if (!__any_sync(0xffffffffu, grow)) break;
          const float z_new = softmax_z<F16>(zx, kUp);
          const float f = grow && have ? ex2(z - z_new) : 1.f;
          if (grow) {
            z = z_new;
            have = true;
          }
          if (any) {
            // O *= f, after the product that is under way
            ok = wait_warp(o_full(o_last), (o_par >> o_last & 1u) ^ 1u, &abort_s, a.wait_use, a.status);
            if (!ok) break;
            tc_fence_after();
            l *= f;
            for (int i = 0; i < blocks * 2; ++i) {
              uint32_t o[32];
              tmem_ld32(tmem + lanes + C::kO + DP * g + 32 * i, o);
              tmem_ld_wait();
              tie(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(tmem + lanes + C::kO + DP * g + 32 * i, o);
            }
            tmem_st_wait();
          }
        }
        if (!ok) break;
        tmem_st32(st, w);
        exps(1);
        tmem_st32(st + 32, w);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(b));
        {
          float u, v;
          unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), u, v);
          l += u + v;
        }
        any = true;
        o_last = C::kGroups == 2 ? g : b;
        o_par ^= 1u << o_last;
      }
      if (ok && C::kGroups == 2 && g == 1 && (idle || (!paired && run.n < 2))) {
        ok = wait_warp(s_full(1), s_par >> 1 & 1u, &abort_s, a.wait_use, a.status);
        s_par ^= 2u;
      }
      if (!ok) break;

      // the unit's partial: O / l and the log of its weight
      if (any) {
        ok = wait_warp(o_full(o_last), (o_par >> o_last & 1u) ^ 1u, &abort_s, a.wait_use, a.status);
        if (!ok) break;
        tc_fence_after();
      }
      const int64_t slot0 =
          ((int64_t)run.unit + blockIdx.x) * (128 * C::kGroups) + 128 * g + quad * 32;
      const int64_t slot_row = slot0 + lane;
      const bool live = row < nrows;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      // 32 columns at a time through the first block of the warp's own rows of Q
      // (whose last product is done), so that rows leave in whole 128-byte lines
      if (any) {
        uint8_t* stage = smem + g * C::kQTile + quad * 4096;
        for (int i = 0; i < blocks * 2; ++i) {
          uint32_t o[32];
          tmem_ld32(tmem + lanes + C::kO + DP * g + 32 * i, o);
          tmem_ld_wait();
          tie(o);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<float4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = make_float4(
                __uint_as_float(o[4 * j]) * inv, __uint_as_float(o[4 * j + 1]) * inv,
                __uint_as_float(o[4 * j + 2]) * inv, __uint_as_float(o[4 * j + 3]) * inv);
          __syncwarp();
          const int piece = lane & 7, col = 32 * i + 4 * piece;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int r = j * 4 + (lane >> 3);
            if (quad * 32 + r < nrows && col < a.D)
              *reinterpret_cast<float4*>(p.part_o + (slot0 + r) * a.D + col) =
                  *reinterpret_cast<const float4*>(stage + r * 128 + ((piece ^ (r & 7)) << 4));
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      if (live) p.part_lse[slot_row] = l == 0.f ? -INFINITY : z + log2f(l);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*static_cast<volatile int*>(&abort_s) && threadIdx.x <= C::kSlots && armed_s[threadIdx.x]) {
    // a role has given up, nothing is sent any more: copies in flight must land
    // before this memory goes
    int dead = 0;
    mbar_wait(threadIdx.x < C::kSlots ? full(threadIdx.x) : land, armed_s[threadIdx.x] & 1u, &dead, a.status);
  }
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int DP, bool F16>
cudaError_t launch_tc_as(const AttnArgs& a, const TcArgs& p, const CUtensorMap& mk,
                         const CUtensorMap& mv, cudaStream_t s) {
  auto kern = attn_prefix_tc_kernel<DP, F16>;
  const cudaError_t e = ensure_smem_attr((const void*)kern, Tc<DP>::kBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.grid), dim3(Tc<DP>::kThreads), Tc<DP>::kBytes, s, a, p, mk, mv);
}

}  // namespace

// Keys of a V slot: the largest box of V.
int attn_tc_v_keys(int D) { return D <= 128 ? 128 : 64; }
// Rows of a partial: two streams of 128, or one.
int attn_tc_rows(int D) { return D <= 128 ? 256 : 128; }

cudaError_t launch_attn_prefix_tc(const AttnArgs& a, const TcArgs& p, const CUtensorMap& mk,
                                  const CUtensorMap& mv, cudaStream_t s) {
  prof_begin(K_ATTN_KEYS, s);
  cudaError_t e;
  if (a.D <= 64)
    e = a.f16 ? launch_tc_as<64, true>(a, p, mk, mv, s) : launch_tc_as<64, false>(a, p, mk, mv, s);
  else if (a.D <= 128)
    e = a.f16 ? launch_tc_as<128, true>(a, p, mk, mv, s) : launch_tc_as<128, false>(a, p, mk, mv, s);
  else
    e = a.f16 ? launch_tc_as<256, true>(a, p, mk, mv, s) : launch_tc_as<256, false>(a, p, mk, mv, s);
  prof_end(K_ATTN_KEYS, s);
  return e;
}

}  // namespace lily
