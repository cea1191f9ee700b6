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
//                  P overwrites S in tensor memory (16 bits)
//   O += P V       A = P from tensor memory, B = V from shared memory as it
//                  lies (keys x dimensions: the N-major operand layout)
// z follows the row's largest score, but O is rescaled only when it grew by
// more than 2^8: until then P is at most 256 instead of 1, which costs no
// precision, and the rescale (a pass over O in tensor memory) stays rare.
//
// Warp 0 brings K and V (TMA boxes of 64 dimensions and one page) into a ring
// of 16 KB slots; warp 1 issues the MMAs (one elected thread); two groups of
// four warps take the softmax of one stream each, so that one stream's softmax
// runs under the other's MMAs.  Rows over 128: the streams are the two row
// blocks and share every K and V tile ("paired"; L2 feeds 32 bytes per clock
// and SM at D = 128).  Up to 128 rows: the streams take alternate tiles of the
// same rows and leave two partials.  Heads over 128 fill tensor memory with
// one stream's output (256 columns) and two score buffers; one softmax group
// alternates between them.
#include "attn.cuh"

namespace lily {
namespace {

constexpr int kKeys = 128;           // keys of a tile
constexpr int kSlot = 16384;         // bytes of a ring slot
constexpr int kMasks = 16;           // tiles whose key masks are kept
constexpr int kCtrlWarps = 4;        // producer, MMA issuer, two that only balance the registers

// DP: head dimension rounded up to 64, 128 or 256.
template <int DP>
struct Tc {
  static constexpr int kGroups = DP <= 128 ? 2 : 1;           // softmax groups = streams
  static constexpr int kThreads = 32 * (kCtrlWarps + 4 * kGroups);
  static constexpr int kVKeys = 128 * 64 / DP;                // keys of a V slot
  static constexpr int kVSlots = kKeys / kVKeys;              // V slots of a tile
  static constexpr int kQTile = 128 * DP * 2;                 // 128 rows, blocks of 64 dimensions
  static constexpr int kQBytes = kGroups * kQTile;
  static constexpr int kSlots = DP == 64 ? 11 : 10;
  static constexpr int kBytes = kQBytes + kSlots * kSlot;
  // tensor memory columns
  static constexpr int kS = 0;        // + 128 * buffer; P in the first 64 columns
  static constexpr int kO = 256;      // + DP * stream
  static_assert(kO + kGroups * DP <= 512, "tensor memory");
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return warp_wait_all(bar, parity, abort, status);
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
  __shared__ __align__(8) uint64_t bars[2 * C::kSlots + 10];
  __shared__ uint32_t mask_s[kMasks][4];
  __shared__ uint32_t tmem_s;
  __shared__ int abort_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  const uint32_t slots = base + C::kQBytes;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (C::kSlots + i); };
  const uint32_t bar1 = bar0 + 8 * 2 * C::kSlots;
  auto q_full = [&](int g) { return bar1 + 8 * g; };        // rows of Q in place
  auto s_full = [&](int b) { return bar1 + 8 * (2 + b); };  // scores in buffer b
  auto p_full = [&](int b) { return bar1 + 8 * (4 + b); };  // probabilities in buffer b
  auto o_full = [&](int g) { return bar1 + 8 * (6 + g); };  // product added to stream g's output
  const uint32_t land = bar1 + 8 * 8, drain = bar1 + 8 * 9;

  if (warp == 0) {
    if (lane == 0) {
      for (int i = 0; i < 2 * C::kSlots; ++i) mbar_init(bar0 + 8 * i, 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(q_full(i), 4);
        mbar_init(s_full(i), 1);
        mbar_init(p_full(i), 4);
        mbar_init(o_full(i), 1);
      }
      mbar_init(land, 1);
      mbar_init(drain, 1);
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

  Run run;
  run.nt = p.tiles;
  run.n = run.before = 0;
  run.at = (int)min((long long)p.share * blockIdx.x, (long long)p.total);
  run.end = (int)min((long long)p.share * (blockIdx.x + 1), (long long)p.total);
  const int rows_all = a.T * a.G;
  const int blocks = (a.D + 63) / 64;  // of 64 dimensions
  const bool paired = p.paired != 0;

  if (warp < kCtrlWarps) {
    if (C::kGroups == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      const int ps = a.page_shift;
      const int k_rows = min(kKeys, 1 << ps), v_rows = min(C::kVKeys, 1 << ps);  // of a box
      const int k_boxes = kKeys / k_rows;                     // of a K slot
      const int v_pages = C::kVKeys / v_rows;                 // of a V slot, times `blocks`
      const int last = (p.len - 1) >> ps;
      int cnt = 0, land_phase = 0;
      bool ok = true;
      int c_base[2] = {-1, -1}, c_page[2] = {0, 0};  // page indices, 32 at a time, for K and V
      // the lane's page of a tile (key k of the prefix), -1 where there is none
      auto page_of = [&](int which, int k0, int k) {
        const int first = k0 >> ps, span = (kKeys + (1 << ps) - 1) >> ps;
        if (c_base[which] < 0 || first < c_base[which] || first + span > c_base[which] + 32) {
          c_base[which] = first;
          c_page[which] = first + lane <= last ? p.pages[first + lane] : -1;
        }
        const int i = k >> ps;
        const int pg = __shfl_sync(0xffffffffu, c_page[which], min(max(i - c_base[which], 0), 31));
        if (i > last) return -1;
        if (pg < 0 || pg >= a.n_pages) {
          set_status(a.status, LILY_STATUS_BAD_PAGE);
          return -1;
        }
        return pg;
      };
      auto load_k = [&](int h, int t) {
        const int k0 = t * kKeys;
        // valid keys of the tile: lane l answers for keys 4l .. 4l+3 (one page)
        const int kl = k0 + 4 * lane;
        const bool there = page_of(0, k0, kl) >= 0;
        const int left = p.len - kl;
        const uint32_t four = !there || left <= 0 ? 0u : left >= 4 ? 15u : (1u << left) - 1;
        uint32_t w = four << (4 * (lane & 7));
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        if ((lane & 7) == 0) mask_s[(run.before + t - run.t0) & (kMasks - 1)][lane >> 3] = w;
        const int c = lane / k_boxes, i = lane - c * k_boxes;
        const int pg = page_of(0, k0, k0 + i * k_rows);
        const bool mine = c < blocks && pg >= 0;
        const uint32_t all = __ballot_sync(0xffffffffu, mine);
        __syncwarp();
        for (int j = 0; j < blocks && ok; ++j) {
          const int slot = (cnt + j) % C::kSlots;
          ok = wait_warp(empty(slot), (((cnt + j) / C::kSlots) & 1) ^ 1, &abort_s, a.status);
          if (ok && lane == 0) {
            const uint32_t boxes = (k_boxes == 32 ? all : all >> (j * k_boxes) & ((1u << k_boxes) - 1));
            mbar_arrive_expect_tx(full(slot), __popc(boxes) * k_rows * 128);
          }
          __syncwarp();
          if (ok && mine && c == j)
            tma_load_4d(slots + slot * kSlot + i * k_rows * 128, &mk, c * 64,
                        k_boxes > 1 ? 0 : k0 & ((1 << ps) - 1), h, pg, full(slot));
          __syncwarp();
        }
        if (ok) cnt += blocks;
      };
      auto load_v = [&](int h, int t) {
        const int k0 = t * kKeys;
        const uint32_t* m = mask_s[(run.before + t - run.t0) & (kMasks - 1)];
        const bool whole = (m[0] & m[1] & m[2] & m[3]) == 0xffffffffu;
        const int per = v_pages * blocks;  // boxes of a slot
        const int c = lane / per, r = lane - c * per;
        const int i = r / blocks, b = r - i * blocks;
        const int kv = c * C::kVKeys + i * v_rows;  // first key of the lane's box in the tile
        const int pg = page_of(1, k0, k0 + min(kv, kKeys - 1));
        const bool mine = c < C::kVSlots && pg >= 0;
        const uint32_t all = __ballot_sync(0xffffffffu, mine);
        for (int j = 0; j < C::kVSlots && ok; ++j) {
          const int slot = (cnt + j) % C::kSlots;
          const uint32_t at = slots + slot * kSlot;
          ok = wait_warp(empty(slot), (((cnt + j) / C::kSlots) & 1) ^ 1, &abort_s, a.status);
          if (!ok) break;
          const uint32_t bar = whole ? full(slot) : land;
          if (lane == 0) {
            const uint32_t boxes = per == 32 ? all : all >> (j * per) & ((1u << per) - 1);
            mbar_arrive_expect_tx(bar, __popc(boxes) * v_rows * 128);
          }
          __syncwarp();
          if (mine && c == j)
            tma_load_4d(at + (b * C::kVKeys + i * v_rows) * 128, &mv, b * 64,
                        (k0 + kv) & ((1 << ps) - 1), h, pg, bar);
          __syncwarp();
          if (!whole) {
            // V of keys that are not there may hold anything, and 0 * NaN
            // would reach every row: it is set to zero before the MMAs see it
            ok = wait_warp(land, land_phase, &abort_s, a.status);
            land_phase ^= 1;
            if (!ok) break;
            for (int k = 0; k < C::kVKeys; ++k) {
              const int key = j * C::kVKeys + k;
              if (m[key >> 5] >> (key & 31) & 1u) continue;
              for (int x = lane; x < blocks * 8; x += 32)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                 at + ((x >> 3) * C::kVKeys + k) * 128 + (x & 7) * 16),
                             "r"(0)
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full(slot));
          }
        }
        if (ok) cnt += C::kVSlots;
      };
      // in the order in which the MMAs take them
      while (ok && run.next()) {
        const int h = run.unit / p.row_blocks;
        load_k(h, run.t0);
        if (!paired && run.n > 1 && ok) load_k(h, run.t0 + 1);
        const int ahead = paired ? 1 : 2;
        for (int t = 0; t < run.n && ok; ++t) {
          load_v(h, run.t0 + t);
          if (t + ahead < run.n && ok) load_k(h, run.t0 + t + ahead);
        }
      }
      if (!ok && lane == 0) {
        // given up: the copies in flight must land before the memory goes
        int dead = 0;
        for (int i = max(0, cnt - C::kSlots); i < cnt; ++i)
          mbar_wait(full(i % C::kSlots), (i / C::kSlots) & 1, &dead, a.status);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const uint32_t fmt = F16 ? idesc_f16_f32(128, 128) : idesc_bf16_f32(128, 128);
      const uint32_t id_qk = fmt;
      const uint32_t id_pv = (F16 ? idesc_f16_f32(128, blocks * 64) : idesc_bf16_f32(128, blocks * 64)) |
                             1u << 16;  // B is N-major
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
      Pos cur = {0, 0};    // next slot to take
      int p_par[2] = {0, 0};
      int q_par = 0;
      bool ok = true;
      // One converged poll for everything a group of MMAs needs: n slots from
      // x and m more from y on, and P of buffer buf (buf < 0: none).
      auto ready = [&](Pos x, int n, Pos y, int m, int buf) {
        for (uint32_t tries = 0;; ++tries) {
          bool r = buf < 0 || mbar_test_wait(p_full(buf), p_par[buf]);
          Pos i = x;
          for (int j = 0; j < n; ++j, i.skip(1)) r = r && mbar_test_wait(full(i.slot), i.par);
          i = y;
          for (int j = 0; j < m; ++j, i.skip(1)) r = r && mbar_test_wait(full(i.slot), i.par);
          if (__all_sync(0xffffffffu, r)) break;
          if ((tries & 255u) == 255u) {
            // the bounded wait takes over, one barrier after the other
            bool w = buf < 0 || warp_wait_all(p_full(buf), p_par[buf], &abort_s, a.status);
            for (int j = 0; j < n && w; ++j, x.skip(1))
              w = warp_wait_all(full(x.slot), x.par, &abort_s, a.status);
            for (int j = 0; j < m && w; ++j, y.skip(1))
              w = warp_wait_all(full(y.slot), y.par, &abort_s, a.status);
            if (!w) return false;
            break;
          }
        }
        if (buf >= 0) p_par[buf] ^= 1;
        tc_fence_after();
        return true;
      };
      // (the next four: by one elected thread)
      // S[buf] = Q[g] K^T with K in the slots from x on
      auto qk = [&](int g, int buf, Pos x) {
        const uint32_t q = desc_k(base + g * C::kQTile), d = tmem + C::kS + 128 * buf;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
          if (c < blocks) {
            const uint32_t k = desc_k(slots + x.slot * kSlot);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_ss(d, q + c * (128 * 128 / 16) + 2 * i, k + 2 * i, id_qk, (c | i) != 0);
            x.skip(1);
          }
        mma_commit(s_full(buf));
      };
      // O[g] (+)= P[buf] V with V in the slots from x on
      auto pv = [&](int g, int buf, Pos x, bool fresh) {
        const uint32_t d = tmem + C::kO + DP * g, pt = tmem + C::kS + 128 * buf;
#pragma unroll
        for (int c = 0; c < C::kVSlots; ++c) {
          const uint32_t v = desc_n(slots + x.slot * kSlot, C::kVKeys * 128);
#pragma unroll
          for (int i = 0; i < C::kVKeys / 16; ++i)
            mma_ts(d, pt + (c * (C::kVKeys / 16) + i) * 8, v + i * (2048 / 16), id_pv,
                   (c | i) != 0 || !fresh);
          x.skip(1);
        }
        mma_commit(o_full(g));
      };
      // the n slots from x on are free once the MMAs so far are done
      auto release = [&](Pos x, int n) {
        for (int j = 0; j < n; ++j, x.skip(1)) mma_commit(empty(x.slot));
      };
      auto q_ready = [&](int g) {
        ok = ok && warp_wait_all(q_full(g), q_par, &abort_s, a.status);
      };
      while (ok && run.next()) {
        const int left = rows_all - run.unit % p.row_blocks * p.block_rows;
        const int n = run.n;
        q_ready(0);
        if (C::kGroups == 2) q_ready(1);
        q_par ^= 1;
        if (paired) {
          const bool two = left > 128;
          if (!(ok = ok && ready(cur, blocks, cur, 0, -1))) break;
          if (elect_one()) {
            qk(0, 0, cur);
            if (two) qk(1, 1, cur);
            release(cur, blocks);
          }
          __syncwarp();
          cur.skip(blocks);
          for (int t = 0; t < n; ++t) {
            const bool more = t + 1 < n;
            Pos nk = cur;  // the next tile's K
            nk.skip(C::kVSlots);
            if (!(ok = ready(cur, C::kVSlots, nk, more ? blocks : 0, 0))) break;
            if (elect_one()) {
              pv(0, 0, cur, t == 0);
              if (more) qk(0, 0, nk);
            }
            __syncwarp();
            if (two && !(ok = ready(cur, 0, cur, 0, 1))) break;
            if (elect_one()) {
              if (two) pv(1, 1, cur, t == 0);
              release(cur, C::kVSlots);
              if (more) {
                if (two) qk(1, 1, nk);
                release(nk, blocks);
              }
            }
            __syncwarp();
            cur = nk;
            if (more) cur.skip(blocks);
          }
        } else {
          // alternate tiles: buffer t & 1, of stream t & 1 where there are two
          for (int t = 0; t < min(2, n); ++t) {
            if (!(ok = ok && ready(cur, blocks, cur, 0, -1))) break;
            if (elect_one()) {
              qk(C::kGroups == 2 ? t : 0, t, cur);
              release(cur, blocks);
            }
            __syncwarp();
            cur.skip(blocks);
          }
          for (int t = 0; t < n && ok; ++t) {
            const int b = t & 1, g = C::kGroups == 2 ? b : 0;
            const bool more = t + 2 < n;
            Pos nk = cur;
            nk.skip(C::kVSlots);
            if (!(ok = ready(cur, C::kVSlots, nk, more ? blocks : 0, b))) break;
            if (elect_one()) {
              pv(g, b, cur, C::kGroups == 2 ? t < 2 : t == 0);
              release(cur, C::kVSlots);
              if (more) {
                qk(g, b, nk);
                release(nk, blocks);
              }
            }
            __syncwarp();
            cur = nk;
            if (more) cur.skip(blocks);
          }
        }
        // a stream without a tile here still waits for the unit's end, so that
        // it does not run ahead of the others
        if (C::kGroups == 2 && ok && (paired ? left <= 128 : n < 2)) {
          if (elect_one()) mma_commit(s_full(1));
          __syncwarp();
        }
      }
      if (!ok) {
        // given up: the MMAs in flight must be done before tensor memory goes
        if (elect_one()) mma_commit(drain);
        __syncwarp();
        int dead = 0;
        if (lane == 0) mbar_wait(drain, 0, &dead, a.status);
        __syncwarp();
      }
    }
  } else {
    // --------------------------------------------------------------- softmax
    if (C::kGroups == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int g = (warp - kCtrlWarps) >> 2;          // stream
    const int quad = warp & 3, row = quad * 32 + lane;
    const int tid = threadIdx.x - 32 * kCtrlWarps - 128 * g;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;  // tensor memory lane field
    const float c = a.scale_log2;
    int s_cnt[2] = {0, 0}, o_cnt = 0;
    bool ok = true;
    while (ok && run.next()) {
      const int h = run.unit / p.row_blocks;
      const int row0 = run.unit % p.row_blocks * p.block_rows + (paired ? g * 128 : 0);
      const int nrows = min(128, rows_all - row0);  // may be 0 or less
      // rows of Q, 16 bytes at a time, swizzled; zeros past the rows and past D
      for (int x = tid; x < 128 * blocks * 8; x += 128) {
        const int r = x / (blocks * 8), e = x - r * blocks * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < nrows && e * 8 < a.D) {
          const int rr = row0 + r, j = rr / a.G, gg = rr - j * a.G;
          v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                              (int64_t)j * a.q_tok +
                                              (int64_t)(h * a.G + gg) * a.q_head + e * 8);
        }
        *reinterpret_cast<uint4*>(smem + g * C::kQTile + (e >> 3) * 128 * 128 + r * 128 +
                                  (((e & 7) ^ (r & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(g));

      float z = 0.f, m = -INFINITY, l = 0.f;
      bool any = false;  // a product has been started
      const bool idle = paired && nrows <= 0;
      const int step = !paired && C::kGroups == 2 ? 2 : 1;
      for (int t = step == 2 ? g : 0; t < run.n && !idle; t += step) {
        const int b = paired ? g : t & 1;
        ok = wait_warp(s_full(b), s_cnt[b] & 1, &abort_s, a.status);
        if (!ok) break;
        ++s_cnt[b];
        tc_fence_after();
        uint32_t s[4][32];
        const uint32_t st = tmem + lanes + C::kS + 128 * b;
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(st + 32 * i, s[i]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) tie(s[i]);
        const uint32_t* mw = mask_s[(run.before + t) & (kMasks - 1)];
        const uint32_t mask[4] = {mw[0], mw[1], mw[2], mw[3]};
        if ((mask[0] & mask[1] & mask[2] & mask[3]) != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(mask[i] >> j & 1u)) s[i][j] = 0xff800000u;  // -inf
        }
        float x = m;
        {
          float y[4] = {m, m, m, m};
#pragma unroll
          for (int j = 0; j < 32; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = fmaxf(y[i], __uint_as_float(s[i][j]));
          x = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
        }
        const float zx = x == -INFINITY ? 0.f : __fmul_rn(x, c);
        // a first maximum is taken as it is; a later one only where the
        // probabilities would pass 2^8 (!(<=): infinities and NaN too)
        const bool grow = m != -INFINITY && !(zx - z <= 8.f);
        float f = 1.f;
        if (m == -INFINITY) {
          z = zx;
          m = x;
        } else if (grow) {
          f = ex2(z - zx);
          z = zx;
          m = x;
        }
        if (__any_sync(0xffffffffu, grow) && any) {
          // O *= f, after the product that is under way
          ok = wait_warp(o_full(g), (o_cnt - 1) & 1, &abort_s, a.status);
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
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float a0 = ex2(fmaf(__uint_as_float(s[i][j]), c, -z));
            const float a1 = ex2(fmaf(__uint_as_float(s[i][j + 1]), c, -z));
            const float b0 = ex2(fmaf(__uint_as_float(s[i + 1][j]), c, -z));
            const float b1 = ex2(fmaf(__uint_as_float(s[i + 1][j + 1]), c, -z));
            sum[0] += a0;
            sum[1] += a1;
            sum[2] += b0;
            sum[3] += b1;
            w[j / 2] = pack16(a0, a1, F16);
            w[16 + j / 2] = pack16(b0, b1, F16);
          }
          tmem_st32(st + 16 * i, w);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(b));
        any = true;
        ++o_cnt;
      }
      if (ok && C::kGroups == 2 && g == 1 && (idle || (!paired && run.n < 2))) {
        ok = wait_warp(s_full(1), s_cnt[1] & 1, &abort_s, a.status);
        ++s_cnt[1];
      }
      if (!ok) break;

      // the segment's partial: O / l and the log of its weight
      if (any) {
        ok = wait_warp(o_full(g), (o_cnt - 1) & 1, &abort_s, a.status);
        if (!ok) break;
        tc_fence_after();
      }
      const int64_t slot_row =
          ((int64_t)run.unit + blockIdx.x) * (128 * C::kGroups) + 128 * g + row;
      const bool live = row < nrows;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float* out = p.part_o + slot_row * a.D;
      if (any)
        for (int i = 0; i < blocks * 2; ++i) {
          uint32_t o[32];
          tmem_ld32(tmem + lanes + C::kO + DP * g + 32 * i, o);
          tmem_ld_wait();
          tie(o);
          if (live)
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              if (32 * i + j < a.D)
                *reinterpret_cast<float4*>(out + 32 * i + j) = make_float4(
                    __uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv,
                    __uint_as_float(o[j + 2]) * inv, __uint_as_float(o[j + 3]) * inv);
        }
      tc_fence_before();
      if (live) p.part_lse[slot_row] = l == 0.f ? -INFINITY : z + log2f(l);
    }
  }
  tc_fence_before();
  __syncthreads();
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
int attn_tc_v_keys(int D) { return D <= 64 ? 128 : D <= 128 ? 64 : 32; }
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
