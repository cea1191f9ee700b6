// attn_rope.cu -- rotation of q and k by position and the append of k and v
// to a paged cache, in one launch (lily_attn_rope_append; into an 8-bit cache:
// lily_attn_rope_append8).
//
// The pair (a, b) number i of a head of token t becomes
//   (a cos - b sin, b cos + a sin),  angle = position[t] * inv_freq[i].
// At far positions an fp32 product loses the angle (position 10^6 leaves an
// error of 0.06 rad), and fp64 arithmetic is slow on this GPU.  So frequencies
// become 64-bit fractions of a turn; position times fraction is then one 64-bit
// integer multiply whose overflow is exactly the whole turns that do not matter;
// what the fraction was cut off by (below 2^-64) grows with the position to 2^-33 of
// a turn at most.
//
// HBM bounds it: q, k and v are read once, in 16-byte pieces, and written
// once.  A CTA takes whole tokens, so that a token's sines are computed once
// for all its heads (shared memory); a short row of lanes covers a head.  Measured:
// 8192 tokens of 16 + 2 + 2 heads of 256 dimensions 30.3 us, 168 MB, 5.5 TB/s; 5
// tokens 2.1 us in a graph.
//
// Into 8 bits (Q8) the lanes of a head find its largest size among them and each
// rounds what it holds, in fp32 since the load, once.  Heads of k and v are few beside
// q's and each costs some ten times the instructions, so all lanes share them out after
// q's, over the CTA's tokens (with q's in one loop, two warps of eight had them all and
// the code took 123 registers a thread: 47 us).  8192 tokens of 16 + 2 + 2 heads of 256
// dimensions 31.0 us, 160 MB, 5.2 TB/s; with 80 registers a thread, three CTAs an SM in
// place of four, 31.8.  One token 3.0 us in a graph.
#include <type_traits>

#include "attn.cuh"

namespace lily {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 8;      // tokens per CTA, at most
constexpr int kMaxPairs = 128;  // rotary_dim / 2, at most

// inv_freq as a 0.64 fixed-point fraction of a turn per position: its 53-bit
// integer mantissa times 2^66 / (2 pi), shifted by its exponent; whole turns
// fall off the top.  In integers, since fp64 instructions are slow enough here
// to show (they took a third of the kernel's time).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int be = (int)(bits >> 52) & 0x7FF;
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (be ? 1ull << 52 : 0ull);
  const int e = (be ? be : 1) - 1075;  // |f| = m 2^e
  const uint64_t c = 0xA2F9836E4E441529ull;  // 2^66 / (2 pi)
  const uint64_t hi = __umul64hi(m, c), lo = m * c;
  const int s = 2 - e;  // |f| / (2 pi) 2^64 = (hi:lo) >> s
  uint64_t t;
  if (s >= 128) t = 0;
  else if (s >= 64) t = s == 64 ? hi : hi >> (s - 64);
  else if (s > 0) t = hi << (64 - s) | lo >> s;
  else t = s > -64 ? lo << -s : 0;
  return (int64_t)bits < 0 ? 0 - t : t;
}

// What both kernels do first: the slots and the sines of the CTA's tokens.
struct alignas(16) Tables {
  float2 cs[kMaxTok][kMaxPairs];  // cos, sin
  int64_t slot[kMaxTok];          // -1: nothing to append
  int64_t cell[kMaxTok];          // its offset in the cache, head 0
};
// (two sines and cosines are read as one float4)
static_assert(alignof(Tables) % alignof(float4) == 0, "16-byte reads of Tables::cs");
__device__ __forceinline__ int64_t cell_of(const RopeArgs& a, int64_t slot) {
  return (slot >> a.page_shift) * a.c_page + (slot & ((1 << a.page_shift) - 1)) * a.c_tok;
}
__device__ __forceinline__ void fill_tables(Tables& tb, const RopeArgs& a, int t0, int nt) {
  for (int i = threadIdx.x; i < nt; i += kThreads) {
    int64_t slot = a.k ? a.slots[t0 + i] : -1;
    if (slot >= a.n_slots) {
      set_status(a.status, LILY_STATUS_BAD_SLOT);
      slot = -1;
    }
    tb.slot[i] = slot < 0 ? -1 : slot;
    tb.cell[i] = slot < 0 ? 0 : cell_of(a, slot);
  }
  // a thread keeps its frequency over the tokens (kThreads / 128 at a time)
  const int p = threadIdx.x % kMaxPairs;
  if (p < a.rot >> 1) {
    const uint64_t fr = turn_fraction(a.inv_freq[p]);
    for (int i = threadIdx.x / kMaxPairs; i < nt; i += kThreads / kMaxPairs) {
      const uint64_t turn = fr * (uint64_t)(int64_t)a.pos[t0 + i];
      float s, c;
      sincospif((float)(int64_t)turn * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
      tb.cs[i][p] = make_float2(c, s);
    }
  }
  __syncthreads();
}
// A head's scale in an 8-bit cache, size / 448, from the bits of its largest size
// (that of a NaN is above all others): 0 where that is no normal number, none where
// the size is no number; and its reciprocal, 0 for those.
__device__ __forceinline__ float scale8(uint32_t size_bits, float& inverse) {
  const float s = __uint_as_float(size_bits) / 448.f;
  inverse = size_bits < 0x7F800000u && s >= 1.17549435e-38f ? 1.f / s : 0.f;
  return size_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : inverse > 0.f ? s : 0.f;
}
__device__ __forceinline__ uint16_t pack8(float a, float b) {  // a in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// x / scale, 0 where `inverse` is that, whatever x.  A product with the reciprocal lies a
// bit beside some quotients, which then fall on the other side of a code's border; by the
// reciprocal rounded to nearest, one step with the product's residue gives the quotient
// itself (Markstein 1990).  Sixteen divisions took 1 us of a token's 3.4.
__device__ __forceinline__ float unit8(float x, float scale, float inverse) {
  const float q = x * inverse;
  return inverse > 0.f ? fmaf(fmaf(-q, scale, x), inverse, q) : 0.f;
}
// Heads of small numbers: the residue above would fall below fp32's least number (codes
// differ where the scale is below 2^-114), so they and their scale are taken 2^64 times as large.
__device__ __forceinline__ bool small8(float scale) { return scale < 0x1p-90f; }
template <int N>
__device__ __forceinline__ void lift8(float (&a)[N], float (&b)[N], float& scale, float& inverse) {
#pragma unroll
  for (int e = 0; e < N; ++e) a[e] *= 0x1p64f, b[e] *= 0x1p64f;
  scale *= 0x1p64f;
  inverse *= 0x1p-64f;
}
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ int64_t scale_cell(const RopeArgs& a, int64_t slot) {
  return (slot >> a.page_shift) * a.s_page + (slot & ((1 << a.page_shift) - 1)) * a.s_tok;
}

// Heads in runs of eight elements (rotary_dim a multiple of 16, or of 8 with
// adjacent pairs).  A lane has two runs of every head it visits, the same ones
// in all: of a turning head a pair that turns together (STYLE 0: u and u +
// rot/2), or two runs past rot or of adjacent pairs (STYLE 1); of V any two.
// A thread keeps the addresses of its NI heads over the CTA's tokens and takes
// 4 / NI tokens at a time, all their loads in flight before the first is used,
// and before the slots and sines are looked up.  (Addresses worked out anew for
// each 16 bytes bound the kernel by its instructions: 217 per 512 bytes, 56 us
// for 8192 tokens of 20 heads of 256.)
// (The 16-bit kernels name no least number of blocks on an SM: with one block the compiler
// took 108 to 145 registers in place of 64 to 104, and 8192 such tokens 39.5 us in place of 32.9.)
template <bool Q8, int STYLE, bool F16, int NI>
__global__ void __launch_bounds__(kThreads, Q8 ? NI == 4 ? 2 : 4 : 0)
    rope_append_runs_kernel(const RopeArgs a, int tok_per_cta, int lanes_log2) {
  constexpr int NB = 4 / NI;
  __shared__ Tables tb;
  const int t0 = blockIdx.x * tok_per_cta;
  const int nt = min(tok_per_cta, a.T - t0);
  const int u = threadIdx.x & ((1 << lanes_log2) - 1), first = threadIdx.x >> lanes_log2;
  const int step = kThreads >> lanes_log2;
  const int half = a.rot >> 1, runs = a.D >> 3;
  const int pairs = STYLE == 0 ? half >> 3 : 0;  // lanes with a pair of runs
  const bool turns = STYLE == 0 ? u < pairs : true;
  // offsets of the two runs in a turning head and in a head of V; -1: none
  const int w = u - pairs, rest = runs - 2 * pairs, rest2 = (rest + 1) >> 1;
  const int ra = u < pairs ? 8 * u : w < rest2 ? 2 * 8 * pairs + 8 * w : -1;
  const int rb = u < pairs ? half + 8 * u : ra >= 0 && w + rest2 < rest ? ra + 8 * rest2 : -1;
  const int v2 = (runs + 1) >> 1;
  const int va = u < v2 ? 8 * u : -1, vb = va >= 0 && u + v2 < runs ? 8 * (u + v2) : -1;
  const int hk = a.hq + a.hkv, H = Q8 ? a.hq : hk + a.hkv;

  pdl_wait();
  pdl_trigger();
  // Q8: the CTA's heads of k and v, all tokens', one at a time and the first one's
  // elements on their way from the start; from the last lanes on, which have no head of
  // q where there are few
  const int heads8 = Q8 && a.k ? 2 * a.hkv : 0;
  auto ahead = [&](int& i, int& h) {  // head h (V's from hkv on) of token i, h too large
    while (h >= heads8 && i < nt) h -= heads8, ++i;
  };
  auto load = [&](int i, int h, uint4& xa, uint4& xb) {
    const bool v = h >= a.hkv;
    const uint16_t* at = v ? static_cast<const uint16_t*>(a.v) + (int64_t)(t0 + i) * a.v_tok + (int64_t)(h - a.hkv) * a.v_head
                           : static_cast<const uint16_t*>(a.k) + (int64_t)(t0 + i) * a.k_tok + (int64_t)h * a.k_head;
    const int oa = v ? va : ra, ob = v ? vb : rb;
    xa = oa >= 0 ? *reinterpret_cast<const uint4*>(at + oa) : make_uint4(0, 0, 0, 0);
    xb = ob >= 0 ? *reinterpret_cast<const uint4*>(at + ob) : make_uint4(0, 0, 0, 0);
  };
  int i8 = heads8 ? 0 : nt, h8 = step - 1 - first;
  uint4 ya, yb;
  if (Q8) ahead(i8, h8);
  if (Q8 && i8 < nt) load(i8, h8, ya, yb);
  bool filled = false;
  for (int h0 = 0; h0 < H; h0 += NI * step) {
    const uint16_t* src[NI];
    uint16_t* dst[NI];
    int src_tok[NI], oa[NI], ob[NI];
    int kind[NI];  // 0: none, 1: q, 2: k, 3: v
#pragma unroll
    for (int n = 0; n < NI; ++n) {
      const int h = h0 + first + n * step;
      kind[n] = h < a.hq ? 1 : Q8 ? 0 : h < hk ? 2 : h < H ? 3 : 0;
      src[n] = nullptr;
      dst[n] = nullptr;
      src_tok[n] = 0;
      if (kind[n] == 1) {
        src[n] = static_cast<const uint16_t*>(a.q) + (int64_t)t0 * a.q_tok + (int64_t)h * a.q_head;
        dst[n] = static_cast<uint16_t*>(a.qo) + (int64_t)t0 * a.qo_tok + (int64_t)h * a.qo_head;
        src_tok[n] = a.q_tok;
      } else if (kind[n] == 2) {
        src[n] = static_cast<const uint16_t*>(a.k) + (int64_t)t0 * a.k_tok + (int64_t)(h - a.hq) * a.k_head;
        dst[n] = static_cast<uint16_t*>(a.kc) + (h - a.hq) * a.c_head;
        src_tok[n] = a.k_tok;
      } else if (kind[n] == 3) {
        src[n] = static_cast<const uint16_t*>(a.v) + (int64_t)t0 * a.v_tok + (int64_t)(h - hk) * a.v_head;
        dst[n] = static_cast<uint16_t*>(a.vc) + (h - hk) * a.c_head;
        src_tok[n] = a.v_tok;
      }
      oa[n] = kind[n] == 3 ? va : kind[n] ? ra : -1;
      ob[n] = kind[n] == 3 ? vb : kind[n] ? rb : -1;
    }
    for (int i0 = 0; i0 < nt; i0 += NB) {
      uint4 xa[NB][NI], xb[NB][NI];
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          const uint16_t* at = src[n] + (int64_t)(i0 + j) * src_tok[n];
          if (i0 + j < nt && oa[n] >= 0) xa[j][n] = *reinterpret_cast<const uint4*>(at + oa[n]);
          if (i0 + j < nt && ob[n] >= 0) xb[j][n] = *reinterpret_cast<const uint4*>(at + ob[n]);
        }
      if (!filled) fill_tables(tb, a, t0, nt);
      filled = true;
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const int i = i0 + j;
        if (i >= nt) break;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          uint16_t* to = dst[n] + (kind[n] == 1 ? (int64_t)i * a.qo_tok : tb.cell[i]);
          if (kind[n] > 1 && tb.slot[i] < 0) continue;
          if (turns && kind[n] != 3) {
            uint32_t wa[4] = {xa[j][n].x, xa[j][n].y, xa[j][n].z, xa[j][n].w};
            uint32_t wb[4] = {xb[j][n].x, xb[j][n].y, xb[j][n].z, xb[j][n].w};
            if (STYLE == 0) {
              const float2* tab = tb.cs[i] + 8 * u;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 c = *reinterpret_cast<const float4*>(tab + 2 * e);
                const float a0 = lo16_f32(wa[e], F16), a1 = hi16_f32(wa[e], F16);
                const float b0 = lo16_f32(wb[e], F16), b1 = hi16_f32(wb[e], F16);
                wa[e] = pack16(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w, F16);
                wb[e] = pack16(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w, F16);
              }
            } else {
              auto turn4 = [&](uint32_t(&x)[4], int at) {
                if (at < 0 || at >= a.rot) return;
                const float2* tab = tb.cs[i] + (at >> 1);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 c = tab[e];
                  const float p = lo16_f32(x[e], F16), r = hi16_f32(x[e], F16);
                  x[e] = pack16(p * c.x - r * c.y, r * c.x + p * c.y, F16);
                }
              };
              turn4(wa, oa[n]);
              turn4(wb, ob[n]);
            }
            xa[j][n] = make_uint4(wa[0], wa[1], wa[2], wa[3]);
            xb[j][n] = make_uint4(wb[0], wb[1], wb[2], wb[3]);
          }
          if (oa[n] >= 0) *reinterpret_cast<uint4*>(to + oa[n]) = xa[j][n];
          if (ob[n] >= 0) *reinterpret_cast<uint4*>(to + ob[n]) = xb[j][n];
        }
      }
    }
  }
  if (Q8) {
    if (!filled) fill_tables(tb, a, t0, nt);
#pragma unroll 1
    while (i8 < nt) {
      const int i = i8, h = h8;
      const bool v = h >= a.hkv;
      const uint32_t wa[4] = {ya.x, ya.y, ya.z, ya.w}, wb[4] = {yb.x, yb.y, yb.z, yb.w};
      h8 += step;
      ahead(i8, h8);
      if (i8 < nt) load(i8, h8, ya, yb);
      if (tb.slot[i] < 0) continue;  // (the lanes of a head together)
      const int oa = v ? va : ra, ob = v ? vb : rb;
      float fa[8], fb[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        fa[2 * e] = lo16_f32(wa[e], F16);
        fa[2 * e + 1] = hi16_f32(wa[e], F16);
        fb[2 * e] = lo16_f32(wb[e], F16);
        fb[2 * e + 1] = hi16_f32(wb[e], F16);
      }
      if (turns && !v) {
        if (STYLE == 0) {
          const float2* tab = tb.cs[i] + 8 * u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = tab[e];
            const float p = fa[e], r = fb[e];
            fa[e] = p * c.x - r * c.y;
            fb[e] = r * c.x + p * c.y;
          }
        } else {
          auto turn8 = [&](float(&x)[8], int at) {
            if (at < 0 || at >= a.rot) return;
            const float2* tab = tb.cs[i] + (at >> 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 c = tab[e];
              const float p = x[2 * e], r = x[2 * e + 1];
              x[2 * e] = p * c.x - r * c.y;
              x[2 * e + 1] = r * c.x + p * c.y;
            }
          };
          turn8(fa, oa);
          turn8(fb, ob);
        }
      }
      uint32_t size = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) size = max(size, max(size_bits(fa[e]), size_bits(fb[e])));
      const uint32_t lanes = 1u << lanes_log2;
      const uint32_t mask = (lanes == 32 ? ~0u : (1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
      for (uint32_t o = lanes >> 1; o > 0; o >>= 1) size = max(size, __shfl_xor_sync(mask, size, o));
      float inverse;
      float scale = scale8(size, inverse);
      if (u == 0) (v ? a.vs : a.ks)[scale_cell(a, tb.slot[i]) + (v ? h - a.hkv : h) * a.s_head] = scale;
      if (small8(scale)) lift8(fa, fb, scale, inverse);
      uint8_t* to = static_cast<uint8_t*>(v ? a.vc : a.kc) + (v ? h - a.hkv : h) * a.c_head + tb.cell[i];
      auto put = [&](const float(&x)[8], int at) {
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[e] = pack8(unit8(x[4 * e], scale, inverse), unit8(x[4 * e + 1], scale, inverse)) |
                 (uint32_t)pack8(unit8(x[4 * e + 2], scale, inverse), unit8(x[4 * e + 3], scale, inverse)) << 16;
        *reinterpret_cast<uint2*>(to + at) = make_uint2(w[0], w[1]);
      };
      if (oa >= 0) put(fa, oa);
      if (ob >= 0) put(fb, ob);
    }
  }
}

// Any even rotary_dim: a pair or an element at a time.
template <bool Q8>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeArgs a, int tok_per_cta,
                                                               int lanes_log2) {
  __shared__ Tables tb;
  const bool f16 = a.dtype == LILY_DTYPE_F16;
  const int t0 = blockIdx.x * tok_per_cta;
  const int nt = min(tok_per_cta, a.T - t0);
  pdl_wait();
  pdl_trigger();
  fill_tables(tb, a, t0, nt);

  const int half = a.rot >> 1;
  const int hk = a.hq + a.hkv, H = hk + a.hkv;
  const int lanes = 1 << lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), first = threadIdx.x >> lanes_log2;
  const int step = kThreads >> lanes_log2;
  for (int i = 0; i < nt; ++i) {
    const int64_t t = t0 + i, slot = tb.slot[i];
    const int64_t cell = tb.cell[i];
    for (int h = first; h < H; h += step) {
      const bool is_v = h >= hk;
      const uint16_t* src;
      uint16_t* dst;
      if (h < a.hq) {
        src = static_cast<const uint16_t*>(a.q) + t * a.q_tok + (int64_t)h * a.q_head;
        dst = static_cast<uint16_t*>(a.qo) + t * a.qo_tok + (int64_t)h * a.qo_head;
      } else {
        if (slot < 0) continue;
        const int64_t kv = h - (is_v ? hk : a.hq);  // (a head's offset may pass 31 bits)
        src = is_v ? static_cast<const uint16_t*>(a.v) + t * a.v_tok + kv * a.v_head
                   : static_cast<const uint16_t*>(a.k) + t * a.k_tok + kv * a.k_head;
        dst = Q8 ? nullptr : static_cast<uint16_t*>(is_v ? a.vc : a.kc) + cell + kv * a.c_head;
      }
      const int pairs = is_v ? 0 : half;
      const int units = pairs + (is_v ? a.D : a.D - a.rot);
      if (Q8 && h >= a.hq) {  // a whole warp per head (lanes = 32): eight units a lane at most
        float p[8], r[8];
        uint32_t size = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int u = lane + 32 * e;
          p[e] = r[e] = 0.f;
          if (u < pairs) {
            const int ia = a.style == 0 ? u : 2 * u, ib = a.style == 0 ? u + half : 2 * u + 1;
            const float2 c = tb.cs[i][u];
            const float x = lo16_f32(src[ia], f16), y = lo16_f32(src[ib], f16);
            p[e] = x * c.x - y * c.y;
            r[e] = y * c.x + x * c.y;
          } else if (u < units) {
            p[e] = lo16_f32(src[u - pairs + (is_v ? 0 : a.rot)], f16);
          }
          size = max(size, max(size_bits(p[e]), size_bits(r[e])));
        }
        size = __reduce_max_sync(0xffffffffu, size);
        float inverse;
        float scale = scale8(size, inverse);
        const int64_t kv = h - (is_v ? hk : a.hq);
        if (lane == 0) (is_v ? a.vs : a.ks)[scale_cell(a, slot) + kv * a.s_head] = scale;
        if (small8(scale)) lift8(p, r, scale, inverse);
        uint8_t* to = static_cast<uint8_t*>(is_v ? a.vc : a.kc) + cell + kv * a.c_head;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int u = lane + 32 * e;
          if (u >= units) break;
          const uint16_t both = pack8(unit8(p[e], scale, inverse), unit8(r[e], scale, inverse));
          if (u < pairs) {
            to[a.style == 0 ? u : 2 * u] = (uint8_t)both;
            to[a.style == 0 ? u + half : 2 * u + 1] = (uint8_t)(both >> 8);
          } else {
            to[u - pairs + (is_v ? 0 : a.rot)] = (uint8_t)both;
          }
        }
        continue;
      }
      for (int u = lane; u < units; u += lanes) {
        if (u < pairs) {
          const int ia = a.style == 0 ? u : 2 * u, ib = a.style == 0 ? u + half : 2 * u + 1;
          const float2 c = tb.cs[i][u];
          const float p = lo16_f32(src[ia], f16), r = lo16_f32(src[ib], f16);
          dst[ia] = pack1(p * c.x - r * c.y, f16);
          dst[ib] = pack1(r * c.x + p * c.y, f16);
        } else {
          const int c = u - pairs + (is_v ? 0 : a.rot);
          dst[c] = src[c];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  prof_begin(K_ATTN_APPEND, s);
  const bool vec = a.style == 0 ? a.rot % 16 == 0 : a.rot % 8 == 0;
  // a power of two of lanes that covers a head's units: two runs each (at most 16)
  const int runs = a.D / 8, pairs = a.style == 0 ? a.rot / 16 : 0;
  const int units = pairs + (runs - 2 * pairs + 1) / 2;
  int lg = vec ? 0 : 5;
  while (vec && lg < 5 && (1 << lg) < units) ++lg;
  // heads per thread; tokens per CTA: four loads of each thread in flight
  // together, twice, but no more than leave every SM four CTAs
  const int H = a.ks ? a.hq : a.hq + 2 * a.hkv, step = kThreads >> lg;
  const int ni = H <= step ? 1 : H <= 2 * step ? 2 : 4;
  int tok = 8 / ni;
  if (tok > a.T / (4 * 152)) tok = a.T / (4 * 152);
  tok = tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
  const dim3 grid((unsigned)(((int64_t)a.T + tok - 1) / tok));  // (T may be 2^31 - 1)
  auto launch = [&](auto kern) { return launch_pdl(kern, grid, dim3(kThreads), 0, s, a, tok, lg); };
  auto by_heads = [&](auto one, auto two, auto four) {
    return ni == 1 ? launch(one) : ni == 2 ? launch(two) : launch(four);
  };
  const bool f16 = a.dtype == LILY_DTYPE_F16;
  auto pick = [&](auto q8) {
    constexpr bool Q8 = decltype(q8)::value;
    return !vec ? launch(rope_append_kernel<Q8>)
           : a.style == 0
               ? f16 ? by_heads(rope_append_runs_kernel<Q8, 0, true, 1>, rope_append_runs_kernel<Q8, 0, true, 2>,
                                rope_append_runs_kernel<Q8, 0, true, 4>)
                     : by_heads(rope_append_runs_kernel<Q8, 0, false, 1>, rope_append_runs_kernel<Q8, 0, false, 2>,
                                rope_append_runs_kernel<Q8, 0, false, 4>)
               : f16 ? by_heads(rope_append_runs_kernel<Q8, 1, true, 1>, rope_append_runs_kernel<Q8, 1, true, 2>,
                                rope_append_runs_kernel<Q8, 1, true, 4>)
                     : by_heads(rope_append_runs_kernel<Q8, 1, false, 1>, rope_append_runs_kernel<Q8, 1, false, 2>,
                                rope_append_runs_kernel<Q8, 1, false, 4>);
  };
  const cudaError_t e = a.ks ? pick(std::true_type{}) : pick(std::false_type{});
  prof_end(K_ATTN_APPEND, s);
  return e;
}

}  // namespace lily
