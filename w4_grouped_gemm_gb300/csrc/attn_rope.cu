// attn_rope.cu -- rotation of q and k by position and the append of k and v
// to a paged cache, in one launch (lily_attn_rope_append).
//
// The pair (a, b) number i of a head of token t becomes
//   (a cos - b sin, b cos + a sin),  angle = position[t] * inv_freq[i].
// At far positions an fp32 product loses the angle (position 10^6 leaves an
// error of 0.06 rad), and fp64 arithmetic per angle is slow on this GPU.  So
// each CTA turns its frequencies once into 64-bit fractions of a turn (two
// fp64 products); position times fraction is then one 64-bit integer multiply
// whose overflow is exactly the whole turns that do not matter.
//
// HBM bounds it: q, k and v are read once, in 16-byte pieces, and written
// once.  A CTA takes whole tokens, so that a token's sines are computed once
// for all its heads (shared memory); a short row of lanes covers a head.
#include "attn.cuh"

namespace lily {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 4;      // tokens per CTA, at most
constexpr int kMaxPairs = 128;  // rotary_dim / 2, at most

// inv_freq as a 0.64 fixed-point fraction of a turn per position.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const double hi = f * 0.15915494309189535;  // 1 / (2 pi), and the rest of it below
  const double lo = fma(f, 0.15915494309189535, -hi) + f * -9.839338337591243e-18;
  const double frac = hi - floor(hi);
  return (uint64_t)__double2ull_rz(frac * 18446744073709551616.0) +
         (uint64_t)__double2ll_rn(lo * 18446744073709551616.0);
}

struct Item {
  const uint16_t* src;
  uint16_t* dst;  // NULL: nothing to write
  bool rotate;
};

// VEC: every run of eight elements is whole (rotary_dim a multiple of 16, or
// of 8 with adjacent pairs).  Else pairs go one at a time.
template <bool VEC>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeArgs a, int tok_per_cta,
                                                               int lanes_log2) {
  __shared__ float2 cs[kMaxTok][kMaxPairs];  // cos, sin
  __shared__ int64_t slot_s[kMaxTok];
  const bool f16 = a.dtype == LILY_DTYPE_F16;
  const int t0 = blockIdx.x * tok_per_cta;
  const int nt = min(tok_per_cta, a.T - t0);
  const int half = a.rot >> 1;

  pdl_wait();
  pdl_trigger();

  for (int i = threadIdx.x; i < nt; i += kThreads) {
    int64_t slot = a.k ? a.slots[t0 + i] : -1;
    if (slot >= a.n_slots) {
      set_status(a.status, LILY_STATUS_BAD_SLOT);
      slot = -1;
    }
    slot_s[i] = slot;
  }
  // a thread keeps its frequency over the tokens (kThreads / 128 at a time)
  {
    const int p = threadIdx.x % kMaxPairs;
    if (p < half) {
      const uint64_t fr = turn_fraction(a.inv_freq[p]);
      for (int i = threadIdx.x / kMaxPairs; i < nt; i += kThreads / kMaxPairs) {
        const uint64_t turn = fr * (uint64_t)(int64_t)a.pos[t0 + i];
        float s, c;
        sincospif((float)(int64_t)turn * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
        cs[i][p] = make_float2(c, s);
      }
    }
  }
  __syncthreads();

  const int H = a.hq + 2 * a.hkv;
  auto item = [&](int it) {
    const int i = it / H, h = it - i * H;
    const int64_t t = t0 + i;
    Item m;
    if (h < a.hq) {
      m.src = static_cast<const uint16_t*>(a.q) + t * a.q_tok + h * a.q_head;
      m.dst = static_cast<uint16_t*>(a.qo) + t * a.qo_tok + h * a.qo_head;
      m.rotate = true;
      return m;
    }
    const bool is_k = h < a.hq + a.hkv;
    const int kv = h - a.hq - (is_k ? 0 : a.hkv);
    const int64_t slot = slot_s[i];
    const int64_t page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
    const int64_t off = page * a.c_page + kv * a.c_head + at * a.c_tok;
    m.src = is_k ? static_cast<const uint16_t*>(a.k) + t * a.k_tok + kv * a.k_head
                 : static_cast<const uint16_t*>(a.v) + t * a.v_tok + kv * a.v_head;
    m.dst = slot < 0 ? nullptr : static_cast<uint16_t*>(is_k ? a.kc : a.vc) + off;
    m.rotate = is_k;
    return m;
  };

  const int lanes = 1 << lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), first = threadIdx.x >> lanes_log2;
  const int step = kThreads >> lanes_log2;
  for (int it = first; it < nt * H; it += step) {
    const Item m = item(it);
    if (!m.dst) continue;
    const float2* tab = cs[it / H];
    if (VEC && a.style == 0) {
      // rot/16 pairs of runs (i, i + rot/2), then the runs past rot as they are
      const int pairs = m.rotate ? half >> 3 : 0;
      const int units = pairs + ((m.rotate ? a.D - a.rot : a.D) >> 3);
      for (int u = lane; u < units; u += lanes) {
        if (u < pairs) {
          const uint4 xa = *reinterpret_cast<const uint4*>(m.src + 8 * u);
          const uint4 xb = *reinterpret_cast<const uint4*>(m.src + half + 8 * u);
          const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
          uint32_t oa[4], ob[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 c = *reinterpret_cast<const float4*>(&tab[8 * u + 2 * j]);
            const float a0 = lo16_f32(wa[j], f16), a1 = hi16_f32(wa[j], f16);
            const float b0 = lo16_f32(wb[j], f16), b1 = hi16_f32(wb[j], f16);
            oa[j] = pack16(a0 * c.x - b0 * c.y, a1 * c.z - b1 * c.w, f16);
            ob[j] = pack16(b0 * c.x + a0 * c.y, b1 * c.z + a1 * c.w, f16);
          }
          *reinterpret_cast<uint4*>(m.dst + 8 * u) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
          *reinterpret_cast<uint4*>(m.dst + half + 8 * u) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
        } else {
          const int c = 8 * (u - pairs) + (m.rotate ? a.rot : 0);
          *reinterpret_cast<uint4*>(m.dst + c) = *reinterpret_cast<const uint4*>(m.src + c);
        }
      }
    } else if (VEC) {
      for (int u = lane; u < a.D >> 3; u += lanes) {
        uint4 x = *reinterpret_cast<const uint4*>(m.src + 8 * u);
        if (m.rotate && 8 * u < a.rot) {
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 c = tab[4 * u + j];
            const float p = lo16_f32(w[j], f16), q = hi16_f32(w[j], f16);
            w[j] = pack16(p * c.x - q * c.y, q * c.x + p * c.y, f16);
          }
          x = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4*>(m.dst + 8 * u) = x;
      }
    } else {
      const int pairs = m.rotate ? half : 0;
      const int units = pairs + (m.rotate ? a.D - a.rot : a.D);
      for (int u = lane; u < units; u += lanes) {
        if (u < pairs) {
          const int ia = a.style == 0 ? u : 2 * u, ib = a.style == 0 ? u + half : 2 * u + 1;
          const float2 c = tab[u];
          const float p = lo16_f32(m.src[ia], f16), q = lo16_f32(m.src[ib], f16);
          m.dst[ia] = pack1(p * c.x - q * c.y, f16);
          m.dst[ib] = pack1(q * c.x + p * c.y, f16);
        } else {
          const int c = u - pairs + (m.rotate ? a.rot : 0);
          m.dst[c] = m.src[c];
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  prof_begin(K_ATTN_APPEND, s);
  const bool vec = a.style == 0 ? a.rot % 16 == 0 : a.rot % 8 == 0;
  // units of a rotating head, and a power of two of lanes that covers them
  const int units = !vec ? a.D - a.rot / 2 : a.style == 0 ? (a.D - a.rot / 2) / 8 : a.D / 8;
  int lg = 2;
  while (lg < 5 && (1 << lg) < units) ++lg;
  const int tok = a.T >= 4096 ? 4 : a.T >= 1024 ? 2 : 1;
  const dim3 grid((unsigned)((a.T + tok - 1) / tok));
  const cudaError_t e = vec ? launch_pdl(rope_append_kernel<true>, grid, dim3(kThreads), 0, s, a, tok, lg)
                            : launch_pdl(rope_append_kernel<false>, grid, dim3(kThreads), 0, s, a, tok, lg);
  prof_end(K_ATTN_APPEND, s);
  return e;
}

}  // namespace lily
