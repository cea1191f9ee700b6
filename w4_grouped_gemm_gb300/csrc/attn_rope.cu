// attn_rope.cu -- rotation of q and k by position and the append of k and v
// to a paged cache, in one launch (lily_attn_rope_append).
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
// Heads in runs of eight elements (rotary_dim a multiple of 16, or of 8 with
// adjacent pairs).  A lane has two runs of every head it visits, the same ones
// in all: of a turning head a pair that turns together (STYLE 0: u and u +
// rot/2), or two runs past rot or of adjacent pairs (STYLE 1); of V any two.
// A thread keeps the addresses of its NI heads over the CTA's tokens and takes
// 4 / NI tokens at a time, all their loads in flight before the first is used,
// and before the slots and sines are looked up.  (Addresses worked out anew for
// each 16 bytes bound the kernel by its instructions: 217 per 512 bytes, 56 us
// for 8192 tokens of 20 heads of 256.)
template <int STYLE, bool F16, int NI>
__global__ void __launch_bounds__(kThreads)
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
  const int hk = a.hq + a.hkv, H = hk + a.hkv;

  pdl_wait();
  pdl_trigger();
  bool filled = false;
  for (int h0 = 0; h0 < H; h0 += NI * step) {
    const uint16_t* src[NI];
    uint16_t* dst[NI];
    int src_tok[NI], oa[NI], ob[NI];
    int kind[NI];  // 0: none, 1: q, 2: k, 3: v
#pragma unroll
    for (int n = 0; n < NI; ++n) {
      const int h = h0 + first + n * step;
      kind[n] = h < a.hq ? 1 : h < hk ? 2 : h < H ? 3 : 0;
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
}

// Any even rotary_dim: a pair or an element at a time.
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
        dst = static_cast<uint16_t*>(is_v ? a.vc : a.kc) + cell + kv * a.c_head;
      }
      const int pairs = is_v ? 0 : half;
      const int units = pairs + (is_v ? a.D : a.D - a.rot);
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
  const int H = a.hq + 2 * a.hkv, step = kThreads >> lg;
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
  const cudaError_t e =
      !vec ? launch(rope_append_kernel)
      : a.style == 0
          ? f16 ? by_heads(rope_append_runs_kernel<0, true, 1>, rope_append_runs_kernel<0, true, 2>,
                           rope_append_runs_kernel<0, true, 4>)
                : by_heads(rope_append_runs_kernel<0, false, 1>, rope_append_runs_kernel<0, false, 2>,
                           rope_append_runs_kernel<0, false, 4>)
          : f16 ? by_heads(rope_append_runs_kernel<1, true, 1>, rope_append_runs_kernel<1, true, 2>,
                           rope_append_runs_kernel<1, true, 4>)
                : by_heads(rope_append_runs_kernel<1, false, 1>, rope_append_runs_kernel<1, false, 2>,
                           rope_append_runs_kernel<1, false, 4>);
  prof_end(K_ATTN_APPEND, s);
  return e;
}

}  // namespace lily
