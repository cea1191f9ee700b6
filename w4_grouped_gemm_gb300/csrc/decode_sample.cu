// decode_sample.cu -- a token for each row of logits (lily_decode_sample):
// temperature, top-k, top-p, min-p and one uniform number.
//
// A row's logits are read from HBM once, by a cluster of CTAs that holds them in
// shared memory as fp32; all further passes run there.  No sort: what is kept is a
// run from the top of the order (logit descending, index ascending), so its end is
// found by descending through histograms, as in a radix selection.  An order number
// joins the logit's bits and the index (51 bits, all different); a pass counts the
// numbers of the range at hand, or adds up their masses, in 512 bins, the cluster
// joins its histograms, and the bin where the count or mass is reached is the next
// range, until it holds one token.  Before the first pass the range of the first k is cut
// to what is not below a floor, from the threads' maxima, that k logits or more reach (all
// filters: one row of 131072 24 -> 13.7 us, 128 rows 125 -> 67).  The draw needs no
// order: masses of consecutive pieces are added up, and the piece that holds u times the
// sum is looked through.
//
// Masses are whole numbers of 2^-44 (the largest is 2^44), so that sums are exact
// and need no order; a mass is right to 2^-23, about as a float can be: borders of up
// to 2^19 tokens lie between 0 and 1, and u must fall on the right side of each.  A
// plain fp32 exponential is off by 2^-19 where the logit is 30 temperatures from the
// largest.
//
// Instructions and barriers bound it, not HBM.  Measured: 128 rows of 131072 by top-p
// 142 us (0.47 TB/s; 180 instructions a logit, 61 percent of issue slots, four rounds of
// 38 clusters), by all filters 66, by none 55; one row with all filters 13.6; 17 rows of
// 50021 in bf16 20 to 24, by the inputs.  A first pass that only counts logits by step and
// a second that adds masses up exactly and lists the steps about p took 132 us, and no less
// for few rows.
#include <algorithm>
#include <cfloat>

#include "decode.cuh"

namespace lily {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;
constexpr int kMaxCluster = 16;
constexpr int kShort = 128;       // slots that a warp's short list holds
constexpr int kFew = kThreads / 2;  // tokens that one CTA puts in order by itself
constexpr uint64_t kOne = 1ull << 44;
constexpr int kIndexBits = 19;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Address of `p`, in this CTA's shared memory, in that of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t remote_ld32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void remote_st32(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void remote_st64(uint32_t a, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// A float's bits in an order that unsigned comparison follows, and back.
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <typename T>
__device__ __forceinline__ T warp_add(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// exp((l - m) / temperature) in units of 2^-44, for l <= m.  With c = log2(e) /
// temperature it is 2^(n + a), n whole and |a| <= 1/2: c and c m are held as two
// floats each, and the first of c m on a grid so coarse that its sum with n is exact,
// so that a = c l - (c m + n) is off by 2^-25 whatever the size of c l (up to 2^12,
// see shifted).
struct Mass {
  float c_hi, c_lo, k, k_hi, k_lo;  // k: c m; k_hi + k_lo: the same
  __device__ __forceinline__ void set(float temperature, float m) {
    constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500e-8f;  // log2(e)
    const float c = kHi / temperature;
    c_hi = fminf(c, 1e30f);
    c_lo = c < 1e30f && temperature < 1e30f ? (fmaf(-c, temperature, kHi) + kLo) / temperature : 0.f;
    k = m * c_hi;
    const float grid = 1.5f * __uint_as_float(__float_as_uint(fabsf(k) + 64.f) & 0x7F800000u);
    k_hi = __fsub_rn(__fadd_rn(k, grid), grid);
    k_lo = (k - k_hi) + fmaf(m, c_lo, fmaf(m, c_hi, -k));
  }
  __device__ __forceinline__ float units(float l) const {
    const float y = fmaf(l, c_hi, -k);
    const float whole = __fadd_rn(y, kRound), n = __fsub_rn(whole, kRound);
    const float a = fmaf(l, c_lo, fmaf(l, c_hi, -(k_hi + n)) - k_lo);
    // 2^a - 1 by the exponential series to the seventh power (2^-27 at the ends)
    float q = 1.52527338040598403e-5f;  // ln2^7 / 7!, then the lower ones
    q = fmaf(q, a, 1.54035303933816100e-4f);
    q = fmaf(q, a, 1.33335581464284434e-3f);
    q = fmaf(q, a, 9.61812910762847716e-3f);
    q = fmaf(q, a, 5.55041086648215800e-2f);
    q = fmaf(q, a, 2.40226506959100712e-1f);
    q = fmaf(q, a, 6.93147180559945309e-1f);
    // (n lies in the last bits of `whole`; those of kRound leave at the top)
    const float w = __uint_as_float(__float_as_uint(fmaf(q, a, 1.f)) + (__float_as_uint(whole) << 23) + (44u << 23));
    return y > -46.f ? w : 0.f;  // (not of -infinity)
  }
  // The same as a whole number: high 2^21 + low, each the last bits of a sum.  (A
  // conversion to 64 bits takes as long as the rest.)
  static constexpr float kRound = 12582912.f;          // 1.5 2^23
  static constexpr float kSplit = 17592186044416.f;    // 2^44
  static constexpr uint32_t kRoundBits = 0x4B400000u, kSplitBits = 0x55800000u;
  __device__ __forceinline__ void split(float l, uint32_t& high, uint32_t& low) const {
    const float w = units(l), h = __fadd_rn(w, kSplit), r = __fsub_rn(w, __fsub_rn(h, kSplit));
    high = __float_as_uint(h);
    low = __float_as_uint(__fadd_rn(r, kRound));
  }
  // of `n` logits' added up
  __device__ __forceinline__ static uint64_t joined(uint32_t high, uint32_t low, uint32_t n) {
    return ((uint64_t)(high - n * kSplitBits) << 21) + (uint64_t)(int64_t)(int32_t)(low - n * kRoundBits);
  }
  __device__ __forceinline__ uint64_t operator()(float l) const {
    uint32_t high, low;
    split(l, high, low);
    return joined(high, low, 1);
  }
};

// f times n, rounded down or up, for 0 <= f <= 1 and n below 2^63.
__device__ __forceinline__ uint64_t share_of(float f, uint64_t n, bool up) {
  const uint32_t bits = __float_as_uint(f), e = bits >> 23;
  const uint64_t sig = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
  const int sh = 150 - (int)(e ? e : 1);  // f = sig 2^-sh, 23 at least
  const uint64_t hi = __umul64hi(sig, n), lo = sig * n;
  uint64_t v, rest;  // what is shifted out
  if (sh >= 128) {
    v = 0;
    rest = hi | lo;
  } else if (sh >= 64) {
    v = sh == 64 ? hi : hi >> (sh - 64);
    rest = lo | (sh == 64 ? 0 : hi << (128 - sh));
  } else {
    v = hi << (64 - sh) | lo >> sh;
    rest = lo << (64 - sh);
  }
  return v + (up && rest ? 1 : 0);
}

struct Shared {
  uint32_t cnt[kBins], lo[kBins], hi[kBins];  // this CTA's histogram: counts, masses in two words
  uint32_t all_cnt[kBins];                    // the cluster's
  uint64_t all_mass[kBins];
  uint32_t part_cnt[kBins];                   // this CTA's bins, each CTA's counts and masses
  uint64_t part_mass[kBins];
  uint64_t list[kFew], weight[kFew];          // the leader's: order numbers of what may be kept, and their masses
  uint64_t sums[kFew];
  uint64_t warp64[kWarps];
  uint32_t warp32[kWarps];
  uint64_t cta64[kMaxCluster];
  uint32_t cta_max[kMaxCluster], cta_min[kMaxCluster], cta_least[kMaxCluster];
  uint32_t warp_max[kWarps], warp_min[kWarps], warp_least[kWarps];
  uint16_t shorts[kWarps][kShort];            // each warp's slots with a logit in a range
  uint32_t n_list[3];  // of each gather: the search by count's, the search by mass's, the last one's
  uint64_t cut_floor, cut_mass;
  uint32_t bin, found, bin_cnt, cnt_before;
  uint64_t mass_before, mass;
};

struct Row {
  const float* v;  // this CTA's slots
  int seg, at0;    // slots of a warp; slot 0's token (may be negative: before the row)
  uint32_t C, rank;
};

// f(four values, token of the first) over this warp's slots, those without a logit
// being -infinity; the warp's lanes are in f together.
template <typename F>
__device__ __forceinline__ void for_fours(const Row& r, F f) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float* v = r.v + warp * r.seg;
  for (int i0 = 0; i0 < r.seg; i0 += 128) {
    const int i = i0 + lane * 4;
    float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (i < r.seg) x = *reinterpret_cast<const float4*>(v + i);
    const float xs[4] = {x.x, x.y, x.z, x.w};
    f(xs, r.at0 + warp * r.seg + i);
  }
}
// f(value, token), one by one.
template <typename F>
__device__ __forceinline__ void for_slots(const Row& r, F f) {
  for_fours(r, [&](const float(&x)[4], int token) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f(x[e], token + e);
  });
}
__device__ __forceinline__ uint64_t order_of(float x, int token) {
  return (uint64_t)key_of(x) << kIndexBits | (kIndexMask - (uint32_t)token);
}

// The cluster's histograms into all_cnt and all_mass.  Each CTA joins kBins / C bins, and
// consecutive threads read and write consecutive ones of one CTA: 5000 cycles, half of
// them the slowest CTA's pass (7500 where a warp's lanes met 16 CTAs).
__device__ __forceinline__ void join_bins(Shared& s, const Row& r) {
  const uint32_t each = kBins / r.C, at = threadIdx.x & (each - 1), j = threadIdx.x / each;
  const uint32_t bin = r.rank * each + at;
  cluster_sync();
  s.part_cnt[threadIdx.x] = remote_ld32(remote(&s.cnt[bin], j));
  s.part_mass[threadIdx.x] = remote_ld32(remote(&s.lo[bin], j)) + ((uint64_t)remote_ld32(remote(&s.hi[bin], j)) << 32);
  __syncthreads();
  uint32_t n = 0;
  uint64_t w = 0;
  for (uint32_t c = 0; c < r.C; ++c) {
    n += s.part_cnt[c * each + at];
    w += s.part_mass[c * each + at];
  }
  remote_st32(remote(&s.all_cnt[bin], j), n);
  remote_st64(remote(&s.all_mass[bin], j), w);
  cluster_sync();
}

// The cluster's sum of a value per thread; every thread gets it, and the sum of
// the CTAs before this one.
__device__ __forceinline__ uint64_t cluster_sum(Shared& s, const Row& r, uint64_t v, uint64_t& before) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_add(v);
  if (lane == 0) s.warp64[warp] = v;
  __syncthreads();
  if (threadIdx.x < r.C) {
    uint64_t sum = 0;
    for (int w = 0; w < kWarps; ++w) sum += s.warp64[w];
    remote_st64(remote(&s.cta64[r.rank], threadIdx.x), sum);
  }
  cluster_sync();
  uint64_t all = 0;
  before = 0;
  for (uint32_t c = 0; c < r.C; ++c) {
    if (c < r.rank) before += s.cta64[c];
    all += s.cta64[c];
  }
  return all;
}

// n and w become the sums over the threads up to this one, n_all and w_all those of
// all; s32 and s64 of kWarps are scratch.
__device__ __forceinline__ void block_scan(uint32_t& n, uint64_t& w, uint32_t* s32, uint64_t* s64, uint32_t& n_all,
                                           uint64_t& w_all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, n, o);
    const uint64_t b = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) n += a, w += b;
  }
  if (lane == 31) s32[warp] = n, s64[warp] = w;
  __syncthreads();
  n_all = 0;
  w_all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const uint32_t a = s32[i];
    const uint64_t b = s64[i];
    if (i == warp) n += n_all, w += w_all;
    n_all += a;
    w_all += b;
  }
}

// The drawn token and the log of its share: (x - m) / temperature less the log of the
// sum, 2^e (1 + f).  Both are 0 or below, so that roundings of 2^-23 of either stay that
// of their sum; f as the float of a whole number, so that a sum near the largest mass
// keeps its bits.
__device__ void put(float m, float x, int token, uint64_t total, float temperature, int32_t* token_out,
                    float* logprob_out) {
  *token_out = token;
  if (logprob_out) {
    const float d = x - m, back = d - x, err = (x - (d - back)) + (-m - back);
    const float z = x == m ? 0.f : d / temperature + err / temperature;
    const int e = 63 - __clzll((long long)total);
    const float f = __ull2float_rn(total - (1ull << e)) * __uint_as_float((uint32_t)(127 - e) << 23);
    *logprob_out = z - ((e - 44) * 0.693147180559945309f + log1pf(f));
  }
}

// The run that is kept: the order numbers from `floor` on; while a search goes on, of
// these the ones in the even steps of the logit up to `last`.
struct Run {
  uint64_t floor;
  int last;     // -1: any step
  float scale;  // steps for a logit's distance of 1
  int listed;   // slots of this warp with a logit in the range at hand, in its short list; -1: not listed
  __device__ __forceinline__ int step(float m, float x) const { return min(kBins - 1, (int)((m - x) * scale)); }
};

enum Found {
  kAll,    // the target is not reached: the run is as it was
  kExact,  // the run ends with the token that reaches it
  kSmall,  // it holds kFew at most, and those that it takes are the first of them
};

// Lists each warp's slots with a logit of lo (no number: any) to hi, n of them; false
// where a warp's are too many.
__device__ __forceinline__ bool list_slots(Shared& s, const Row& r, float lo, float hi, int& n) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  n = 0;
  for_fours(r, [&](const float(&x)[4], int token) {
    bool in[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) in[e] = !(x[e] < lo) && x[e] <= hi && x[e] > -INFINITY;
    if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t all = __ballot_sync(0xffffffffu, in[e]);
      const int at = n + __popc(all & ((1u << lane) - 1));
      if (in[e] && at < kShort) s.shorts[warp][at] = (uint16_t)(token + e - r.at0);
      n += __popc(all);
    }
  });
  return !__syncthreads_or(n > kShort);
}
// f(value, token) over the slots listed, n of this warp, or (n < 0) all.
template <typename F>
__device__ __forceinline__ void for_some(const Shared& s, const Row& r, int n, F f) {
  if (n < 0) {
    for_slots(r, f);
    return;
  }
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < n; i += 32) {
    const int slot = s.shorts[threadIdx.x >> 5][i];
    f(r.v[slot], r.at0 + slot);
  }
}

// The cluster's tokens for which f(logit, token) is true, kFew at most, into the list
// of its first CTA, in any order, counted from 0 by n_list[which]; ends with a barrier of
// the cluster.
template <typename F>
__device__ __forceinline__ void gather(Shared& s, const Row& r, int which, int listed, F f) {
  for_some(s, r, listed, [&](float x, int token) {
    if (x > -INFINITY && f(x, token)) {
      uint32_t at;
      asm volatile("atom.shared::cluster.add.u32 %0, [%1], 1;"
                   : "=r"(at)
                   : "r"(remote(&s.n_list[which], 0))
                   : "memory");
      remote_st64(remote(&s.list[at & (kFew - 1)], 0), order_of(x, token));
    }
  });
  cluster_sync();
}

// In the first CTA: thread i takes the list's number i and finds its place in the
// order, half of the list, the other half being counted by thread i + kFew.  False for
// threads without one.
__device__ __forceinline__ bool in_order(Shared& s, int which, uint64_t& o, uint32_t& place) {
  const uint32_t n = min(s.n_list[which], (uint32_t)kFew), i = threadIdx.x % kFew, half = (n + 1) / 2;
  const bool upper = threadIdx.x >= kFew;
  o = i < n ? s.list[i] : 0;
  place = 0;
  if (i < n)
    for (uint32_t j = upper ? half : 0, end = upper ? n : half; j < end; ++j) place += s.list[j] > o;
  if (upper) s.cnt[i] = place;
  __syncthreads();
  if (!upper) place += s.cnt[i];
  return !upper && i < n;
}

// Cuts the run to where a number of tokens (by_mass: a mass, 0: p times that of all)
// is reached; `mass` becomes its mass (masses: whether that is wanted).  Each pass takes
// the range at hand in kBins bins, even steps of the logit in the first by mass, where
// masses of all tokens count and few logits share a step, else even steps of the order
// numbers, until the bin that it ends in holds kFew.
__device__ Found search(Shared& s, const Row& r, const Mass& weigh, float m, bool by_mass, bool masses, bool linear,
                        float p, uint64_t top, uint64_t& target, Run& run, uint64_t& mass) {
  const int b = threadIdx.x;
  uint64_t lo = run.floor, hi = top, mass_above = 0;
  uint32_t cnt_above = 0;
  bool tried = false;
  run.listed = -1;
  auto list = [&]() {
    int n;
    if (list_slots(s, r, of_key((uint32_t)(lo >> kIndexBits)), of_key((uint32_t)(hi >> kIndexBits)), n)) run.listed = n;
    tried = true;
  };
  for (;;) {
    const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 9);
    s.cnt[b] = s.lo[b] = s.hi[b] = 0;
    if (b == 0) s.found = 0;
    __syncthreads();
    auto add = [&](int bin, uint64_t w) {
      atomicAdd(&s.cnt[bin], 1u);
      if (!masses) return;
      const uint32_t w_lo = (uint32_t)w, old = atomicAdd(&s.lo[bin], w_lo);
      const uint32_t w_hi = (uint32_t)(w >> 32) + (old + w_lo < old);
      if (w_hi) atomicAdd(&s.hi[bin], w_hi);
    };
    if (linear) {
      for_fours(r, [&](const float(&x)[4], int token) {
        uint64_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = weigh(x[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (w[e] && (lo == 0 || order_of(x[e], token + e) >= lo)) add(run.step(m, x[e]), w[e]);
      });
    } else {
      const float x_lo = of_key((uint32_t)(lo >> kIndexBits)), x_hi = of_key((uint32_t)(hi >> kIndexBits));
      if (!tried) list();
      for_some(s, r, run.listed, [&](float x, int token) {
        // (an x_lo that is no number has all above it; -infinity is no token)
        if (!(x < x_lo) && x <= x_hi && x > -INFINITY) {
          const uint64_t o = order_of(x, token);
          if (o >= lo && o <= hi && (run.last < 0 || run.step(m, x) == run.last))
            add(kBins - 1 - (int)((o - lo) >> shift), masses ? weigh(x) : 0);
        }
      });
    }
    join_bins(s, r);
    // from the top bin (the first) on: where the target is reached
    const uint32_t n = s.all_cnt[b];
    const uint64_t w = s.all_mass[b];
    uint32_t n_upto = n, n_all;
    uint64_t w_upto = w, w_all;
    block_scan(n_upto, w_upto, s.warp32, s.warp64, n_all, w_all);
    n_upto += cnt_above;
    w_upto += mass_above;
    w_all += mass_above;
    if (target == 0) target = max(share_of(p, w_all, true), (uint64_t)1);
    const uint64_t own = by_mass ? w : n, upto = by_mass ? w_upto : n_upto;
    if (own && upto >= target && upto - own < target) {
      s.found = 1;
      s.bin = b;
      s.bin_cnt = n;
      s.cnt_before = n_upto - n;
      s.mass_before = w_upto - w;
      s.mass = w;
    }
    __syncthreads();
    if (!s.found) {
      mass = w_all;
      return kAll;
    }
    const int bin = s.bin;
    const uint32_t bin_cnt = s.bin_cnt;
    cnt_above = s.cnt_before;
    mass_above = s.mass_before;
    mass = mass_above + s.mass;
    if (linear) {
      // the step's order numbers, with room for the roundings of a logit's place
      run.last = bin;
      const float room = (fabsf(m) + (bin + 1) / run.scale) * 1e-6f;
      const float x_hi = fminf(m, m - bin / run.scale + room);
      const float x_lo = bin == kBins - 1 ? -FLT_MAX : m - (bin + 1) / run.scale - room;
      lo = max(lo, (uint64_t)key_of(x_lo) << kIndexBits);
      hi = (uint64_t)key_of(x_hi) << kIndexBits | kIndexMask;
    } else {
      lo += (uint64_t)(kBins - 1 - bin) << shift;
      hi = lo + ((1ull << shift) - 1);
    }
    run.floor = lo;
    if (cnt_above + bin_cnt <= kFew) return kSmall;
    if (bin_cnt <= kFew) {
      // the first CTA puts the bin's in order and says from which number on the run goes
      if (!tried) list();
      const int which = by_mass ? 1 : 0;  // (both searches of a row may come here)
      gather(s, r, which, run.listed, [&](float x, int token) {
        const uint64_t o = order_of(x, token);
        return o >= lo && o <= hi && (run.last < 0 || run.step(m, x) == run.last) && (!by_mass || weigh(x));
      });
      if (r.rank == 0) {
        uint64_t o, w = 0, all_w;
        uint32_t place;
        const bool in = in_order(s, which, o, place);
        if (in) w = weigh(of_key((uint32_t)(o >> kIndexBits)));
        if (b < kFew) s.weight[b] = 0;
        __syncthreads();
        if (in) s.weight[place] = w;
        __syncthreads();
        uint32_t one = 1, ones;
        uint64_t upto = b < kFew ? s.weight[b] : 0;
        block_scan(one, upto, s.warp32, s.warp64, ones, all_w);
        if (b < kFew) s.sums[b] = upto;
        __syncthreads();
        if (in) {
          const uint64_t with = by_mass ? mass_above + s.sums[place] : cnt_above + place + 1;
          if (with >= target && with - (by_mass ? w : 1) < target)
            for (uint32_t c = 0; c < r.C; ++c) {
              remote_st64(remote(&s.cut_floor, c), o);
              remote_st64(remote(&s.cut_mass, c), mass_above + s.sums[place]);
            }
        }
      }
      cluster_sync();
      run.floor = s.cut_floor;
      run.last = -1;
      mass = s.cut_mass;
      return kExact;
    }
    linear = false;
    __syncthreads();
  }
}

// The rest for a run of kFew tokens at most, in the cluster's first CTA, a thread for
// each: places in the order by counting, top-k (k tokens), top-p (target: mass that is
// held; 0: p times that of the k), min-p and the draw.
__device__ void finish(Shared& s, const Mass& weigh, float m, uint32_t k, float p, uint64_t target, uint64_t least_mass,
                       float u, float temperature, int32_t* token_out, float* logprob_out) {
  const uint32_t n = min(s.n_list[2], (uint32_t)kFew), i = threadIdx.x;
  uint64_t o;
  uint32_t place;
  const bool in = in_order(s, 2, o, place) && place < k;
  const float x = of_key((uint32_t)(o >> kIndexBits));
  const uint32_t token = kIndexMask - ((uint32_t)o & kIndexMask);
  const uint64_t w = in ? weigh(x) : 0;
  bool keep = in;
  if (i < kFew) s.weight[i] = 0;
  __syncthreads();
  if (p < 1.f) {
    if (in) s.weight[place] = w;
    __syncthreads();
    uint32_t one = 0, ones;
    uint64_t upto = i < kFew ? s.weight[i] : 0, all;
    block_scan(one, upto, s.warp32, s.warp64, ones, all);
    if (i < kFew) s.sums[i] = upto;
    __syncthreads();
    if (target == 0) target = max(share_of(p, all, true), (uint64_t)1);
    keep = in && s.sums[place] - w < target;
    if (i < kFew) s.weight[i] = 0;
    __syncthreads();
  }
  keep = in && (place == 0 || (keep && w >= least_mass));
  if (keep) s.weight[i] = w;
  __syncthreads();
  // the mass of all that are kept, and of those with a lower index
  uint64_t before = 0, total = 0;
  if (in)
    for (uint32_t j = 0; j < n; ++j) {
      const uint64_t v = s.weight[j];
      total += v;
      before += kIndexMask - ((uint32_t)s.list[j] & kIndexMask) < token ? v : 0;
    }
  const uint64_t want = min(share_of(u, total, false), total - 1);
  if (keep && want >= before && want - before < w) put(m, x, token, total, temperature, token_out, logprob_out);
}

// A warp's part of the floor of the first k (the floor: the least of all warps'): of its
// threads' largest, `top` the first of them, the j-th, where j in each of the `full` warps
// that are full of tokens are k or more; 0 where that is more than its threads, no limit
// for a warp that is not full.  (The k-th of all warps' lies higher, but to find it took
// as long as it saved.)
__device__ __noinline__ uint32_t warp_floor(uint32_t key, uint32_t top, int k, int full, int warp, int threads) {
  if (full == 0 || (k + full - 1) / full > threads) return 0;
  if (warp >= full) return ~0u;
  for (int j = (k + full - 1) / full; j > 1; --j) {
    if ((threadIdx.x & 31) == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) key = 0;
    top = __reduce_max_sync(0xffffffffu, key);
  }
  return top;
}

template <int DT>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if (DT == LILY_DTYPE_F32) return static_cast<const float*>(p)[i];
  return lo16_f32(static_cast<const uint16_t*>(p)[i], DT == LILY_DTYPE_F16);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2)
    decode_sample_kernel(const SampleArgs a, int C, int seg) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  float* v = reinterpret_cast<float*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / C;
  Row r;
  r.v = v;
  r.seg = seg;
  r.C = C;
  r.rank = cluster_rank();

  cluster_arrive();  // (before its first store into another CTA it waits until all run)
  pdl_wait();
  pdl_trigger();

  const float temperature = a.temperature[b];
  const int k = a.top_k ? a.top_k[b] : 0;
  const float p = a.top_p ? a.top_p[b] : 1.f, least_p = a.min_p ? a.min_p[b] : 0.f;
  const float given_u = a.u ? a.u[b] : 0.f;

  // ---- the row into shared memory, in whole 16-byte pieces from the one it begins in
  constexpr int kVec = DT == LILY_DTYPE_F32 ? 4 : 8, kBatch = 4;  // pieces on the way at once
  const int64_t first = (int64_t)b * a.stride;
  const int off = (int)(first % kVec);
  r.at0 = (int)r.rank * kWarps * seg - off;
  float most = -INFINITY, fewest = INFINITY;
  bool nan = false;
  auto held = [&](float x) {  // -0 is 0; a NaN is -infinity
    nan |= x != x;
    x = fmaxf(x + 0.f, -INFINITY);
    most = fmaxf(most, x);
    return x;
  };
  for (int i0 = lane * kVec; i0 < seg; i0 += kBatch * 32 * kVec) {
    uint4 p[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * 32 * kVec, t = r.at0 + warp * seg + i;  // the piece's first token
      if (i < seg && t >= 0 && t + kVec <= a.V)
        p[j] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.logits) + (first + t) * (16 / kVec));
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * 32 * kVec, t = r.at0 + warp * seg + i;
      if (i >= seg) break;
      const bool whole = t >= 0 && t + kVec <= a.V;
      const uint32_t w[4] = {p[j].x, p[j].y, p[j].z, p[j].w};
#pragma unroll
      for (int h = 0; h < kVec; h += 4) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (whole)
            x[e] = kVec == 4 ? __uint_as_float(w[e])
                   : e & 1   ? hi16_f32(w[(h + e) / 2], DT == LILY_DTYPE_F16)
                             : lo16_f32(w[(h + e) / 2], DT == LILY_DTYPE_F16);
          else
            x[e] = t + h + e >= 0 && t + h + e < a.V ? logit_at<DT>(a.logits, first + t + h + e) : -INFINITY;
          x[e] = held(x[e]);
        }
        // (a sample will do: it only sets the steps of a search)
        if (x[0] > -INFINITY) fewest = fminf(fewest, x[0]);
        *reinterpret_cast<float4*>(v + warp * seg + i + h) = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  if (nan) set_status(a.status, LILY_STATUS_NAN_LOGIT);

  // ---- the largest and the least logit, and the floor
  if (threadIdx.x < 3) s.n_list[threadIdx.x] = 0;
  {
    const uint32_t key = key_of(most);
    const uint32_t top = __reduce_max_sync(0xffffffffu, key), low = __reduce_min_sync(0xffffffffu, key_of(fewest));
    const uint32_t least = k > 0 ? warp_floor(key, top, k, (a.V + off) / seg, r.rank * kWarps + warp, min(32, seg / kVec)) : 0;
    if (lane == 0) s.warp_max[warp] = top, s.warp_least[warp] = least, s.warp_min[warp] = low;
    cluster_wait();
    __syncthreads();
    if (threadIdx.x < r.C) {
      uint32_t m = 0, ll = ~0u, ml = ~0u;
      for (int w = 0; w < kWarps; ++w) {
        m = max(m, s.warp_max[w]);
        ll = min(ll, s.warp_least[w]);
        ml = min(ml, s.warp_min[w]);
      }
      remote_st32(remote(&s.cta_max[r.rank], threadIdx.x), m);
      remote_st32(remote(&s.cta_least[r.rank], threadIdx.x), ll);
      remote_st32(remote(&s.cta_min[r.rank], threadIdx.x), ml);
    }
    cluster_sync();
  }
  uint32_t key_max = 0, key_floor = ~0u, key_min = ~0u;
  for (int c = 0; c < C; ++c) {
    key_max = max(key_max, s.cta_max[c]);
    key_floor = min(key_floor, s.cta_least[c]);
    key_min = min(key_min, s.cta_min[c]);
  }
  float m = of_key(key_max);
  if (m == INFINITY) {
    // infinities share all mass: logits of 0 among none
    for (int i = threadIdx.x; i < kWarps * seg; i += kThreads) v[i] = v[i] == INFINITY ? 0.f : -INFINITY;
    __syncthreads();
    m = 0.f;
    key_max = key_min = key_of(0.f);
    key_floor = 0;
  }
  const bool greedy = !(temperature > 0.f) || !a.u || k == 1 || p <= 0.f || least_p > 1.f;

  if (m == -INFINITY || greedy) {
    // the first token of the largest logit
    uint32_t at = ~0u;
    for_slots(r, [&](float x, int token) {
      if (x == m && m > -INFINITY) at = min(at, (uint32_t)token);
    });
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) s.warp_least[warp] = at;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 0; w < kWarps; ++w) at = min(at, s.warp_least[w]);
      remote_st32(remote(&s.cta64[r.rank], 0), at);
    }
    cluster_sync();
    if (r.rank == 0 && threadIdx.x == 0) {
      for (int c = 0; c < C; ++c) at = min(at, (uint32_t)s.cta64[c]);
      a.tokens[b] = (int32_t)at;  // (none: ~0 is -1)
      if (a.logprobs) a.logprobs[b] = at == ~0u ? -INFINITY : 0.f;
    }
    return;
  }

  Mass weigh;
  weigh.set(temperature, m);
  if (!(fabsf(weigh.k) <= 4096.f)) {
    // logits so large beside the temperature that those with a mass lie next to the
    // largest: their distances are exact, and take their place
    for (int i = threadIdx.x; i < kWarps * seg; i += kThreads) v[i] -= m;
    __syncthreads();
    auto shifted = [&](uint32_t key) { return key_of(of_key(key) - m + 0.f); };
    if (key_floor) key_floor = shifted(key_floor);
    key_min = shifted(key_min);
    m = 0.f;
    key_max = key_of(0.f);
    weigh.set(temperature, m);
  }
  const uint64_t top = (uint64_t)key_max << kIndexBits | kIndexMask;
  uint64_t least_mass = 1;
  if (least_p > 0.f) least_mass = max(share_of(least_p, kOne, true), (uint64_t)1);
  const float u = fminf(fmaxf(given_u, 0.f), 0.99999994f);
  Run run = {0, -1, 0.f, -1};
  uint64_t mass = 0, before, target = 0;
  uint32_t first_k = ~0u;
  bool small = false;
  if (k > 0 && k < a.V) {
    run.floor = (uint64_t)key_floor << kIndexBits;
    uint64_t number = k;
    const Found f = search(s, r, weigh, m, false, p < 1.f, false, p, top, number, run, mass);
    if (f == kAll) run.floor = 0;
    if (f == kSmall) {
      small = true;
      first_k = k;
    } else if (p < 1.f) {
      target = max(share_of(p, mass, true), (uint64_t)1);
    }
  }
  if (!small && p < 1.f) {
    // (no mass is further from the largest than 32 temperatures)
    const float range = fminf(32.f * temperature, m - of_key(key_min));
    const bool linear = range > 1e-30f && range < 1e30f;
    run.scale = linear ? kBins / range : 0.f;
    __syncthreads();  // (the search before is read)
    small = search(s, r, weigh, m, true, true, linear, p, top, target, run, mass) == kSmall;
  }
  if (small) {
    // (tokens without mass are not drawn, and were not counted by mass)
    // (by mass the list is that of the last steps alone)
    const int listed = run.last < 0 ? run.listed : -1;
    const float x_floor = of_key((uint32_t)(run.floor >> kIndexBits));
    gather(s, r, 2, listed, [&](float x, int token) {
      return !(x < x_floor) && order_of(x, token) >= run.floor && (run.last < 0 || run.step(m, x) <= run.last) && weigh(x);
    });
    if (r.rank == 0)
      finish(s, weigh, m, first_k, p, target, least_mass, u, temperature, a.tokens + b, a.logprobs ? a.logprobs + b : nullptr);
    return;
  }

  // ---- the draw
  // (floor 0: the logit is no number and the index the last, so that all are kept)
  const float x_floor = of_key((uint32_t)(run.floor >> kIndexBits));
  const int last_token = (int)(kIndexMask - ((uint32_t)run.floor & kIndexMask));
  auto in_run = [&](float x, int token) { return !(x <= x_floor) || (x == x_floor && token <= last_token); };
  auto kept = [&](float x, int token) -> uint64_t {
    const uint64_t w = weigh(x);
    return in_run(x, token) && w >= least_mass ? w : 0;
  };
  uint64_t mine = 0;
  {
    const bool any_mass = least_mass == 1;
    uint32_t high = 0, low = 0, n = 0;
    for_fours(r, [&](const float(&x)[4], int token) {
      const float most4 = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      if (!__any_sync(0xffffffffu, !(most4 < x_floor))) return;
      if (any_mass && run.floor == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, l;
          weigh.split(x[e], h, l);
          high += h;
          low += l;
        }
        n += 4;
      } else if (any_mass) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t h, l;
          weigh.split(x[e], h, l);
          const bool in = in_run(x[e], token + e);
          high += in ? h : Mass::kSplitBits;
          low += in ? l : Mass::kRoundBits;
        }
        n += 4;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) mine += kept(x[e], token + e);
      }
    });
    mine += Mass::joined(high, low, n);
  }
  const uint64_t all = cluster_sum(s, r, mine, before);
  uint64_t want = min(share_of(u, all, false), all - 1);
  // the CTA and the warp whose slots hold it (every warp of a CTA looks)
  uint64_t upto = lane < kWarps ? s.warp64[lane] : 0;
  const uint64_t own = upto;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  const uint32_t at = __ballot_sync(0xffffffffu, lane < kWarps && want >= before + upto - own && want < before + upto);
  if (at == 0) return;
  const int q = __ffs(at) - 1;
  want -= before + __shfl_sync(0xffffffffu, upto - own, q);
  // all warps look through its slots
  const int part = ((seg + kWarps - 1) / kWarps + 7) & ~7, i = warp * part + lane * 8;
  uint64_t w[8], sum = 0;
  const int token = r.at0 + q * seg + i;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = lane * 8 < part && i < seg ? v[q * seg + i + j] : -INFINITY;
    w[j] = kept(x, token + j);
    sum += w[j];
  }
  upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) s.weight[warp] = upto;
  __syncthreads();
  uint64_t pre = 0;
#pragma unroll
  for (int k2 = 0; k2 < kWarps; ++k2) pre += k2 < warp ? s.weight[k2] : 0;
  upto += pre;
  if (want >= upto || want < upto - sum) return;
  uint64_t run_up = upto - sum;
  int hit = -1;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    run_up += w[j];
    if (hit < 0 && want < run_up) hit = j;
  }
  put(m, v[q * seg + i + hit], token + hit, all, temperature, a.tokens + b, a.logprobs ? a.logprobs + b : nullptr);
}

}  // namespace

// CTAs of a row's cluster: enough that two CTAs fit on an SM (20480 logits each), and
// twice as many while every CTA then has an SM of its own, since two on one take turns, and
// 2048 logits or more.  By top-p, in a graph: 14 rows of 20000 logits 15.3 us by 8 CTAs, 15.4
// by 4; 18 rows 17.3, 15.5; 36 rows 27.2, 17.3, and 19.2 by 2; 40 rows 20.9 by 4, 19.2 by 2;
// 76 rows 19.7 by 2, 26.5 by 1; 80 rows 25.9, 26.5.  (1250 logits a CTA: 8 rows of 10000 12.4
// us by 8, 13.4 by 4; 18 rows 14.8, 13.6.)  16 only for a few rows, or where a row takes them,
// since few clusters of that size find room at once: 4 rows of 131072 22.5 us by 16, 27.5 by
// 8; 8 rows 30.2, 27.7.  (Six find room on the GPU that this was measured on, and other GPUs
// of its kind may place fewer.)
static int cluster_of(int B, int V, int sms) {
  int C = 1;
  while (C < kMaxCluster && V > C * 20480) C *= 2;
  const int most = B <= 4 ? kMaxCluster : kMaxCluster / 2;
  while (C < most && (int64_t)B * C * 2 <= sms && V >= C * 2 * 2048) C *= 2;
  return C;
}

cudaError_t launch_decode_sample(const SampleArgs& a, int sms, cudaStream_t s) {
  const int C = cluster_of(a.B, a.V, sms);
  const int kVec = 8;  // (a row may begin up to 7 elements into a 16-byte piece)
  const int64_t slots = (int64_t)a.V + kVec - 1;
  const int seg = (int)((slots + (int64_t)C * kWarps - 1) / ((int64_t)C * kWarps) + 7) & ~7;
  const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + (size_t)seg * kWarps * 4;
  auto launch = [&](auto kern) {
    const void* f = reinterpret_cast<const void*>(kern);
    cudaError_t e = ensure_smem_attr(f, smem);
    if (e == cudaSuccess && C > 8) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.B * C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, C, seg);
  };
  return a.dtype == LILY_DTYPE_F32   ? launch(decode_sample_kernel<LILY_DTYPE_F32>)
         : a.dtype == LILY_DTYPE_F16 ? launch(decode_sample_kernel<LILY_DTYPE_F16>)
                                     : launch(decode_sample_kernel<LILY_DTYPE_BF16>);
}

}  // namespace lily
