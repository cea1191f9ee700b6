// attn_norm.cu -- residual addition and RMSNorm, with 16-bit rows or 8-bit
// rows and scales out (lily_attn_add_rmsnorm).
//
//   r = residual + x,  n_i = r_i / sqrt(mean(r^2) + eps) * w_i,
//   8 bits: s_g = max over group g of |n_i| / 448,  out_i = e4m3(n_i / s_g)
//
// One pass: a row stays in registers between its sum of squares, the maxima
// of its groups and its stores, so that x and the residual are read once and
// the outputs written once.  HBM bounds it from some hundred rows on, the
// latency of one load and two block reductions below.
#include <cuda_fp8.h>

#include "attn.cuh"

namespace lily {
namespace {

// Raw bits of eight consecutive elements: 16-bit types use a, fp32 a and b.
// Loading the bits first and converting later keeps a row's loads of both
// operands in flight together.
struct Raw8 {
  uint4 a, b;
};

__device__ __forceinline__ void load_raw8(Raw8& r, const void* p, int64_t i, int type) {
  if (type == LILY_DTYPE_F32) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    r.a = q[0];
    r.b = q[1];
  } else {
    r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
}

// (one branch per eight elements, not a choice per element)
__device__ __forceinline__ void unpack8(const Raw8& r, int type, float (&v)[8]) {
  if (type == LILY_DTYPE_F32) {
    v[0] = __uint_as_float(r.a.x); v[1] = __uint_as_float(r.a.y);
    v[2] = __uint_as_float(r.a.z); v[3] = __uint_as_float(r.a.w);
    v[4] = __uint_as_float(r.b.x); v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z); v[7] = __uint_as_float(r.b.w);
    return;
  }
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  if (type == LILY_DTYPE_F16) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = lo16_f32(w[j], true);
      v[2 * j + 1] = hi16_f32(w[j], true);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = lo16_f32(w[j], false);
      v[2 * j + 1] = hi16_f32(w[j], false);
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8], bool f16) {
  if (f16)
    return make_uint4(pack16(v[0], v[1], true), pack16(v[2], v[3], true), pack16(v[4], v[5], true),
                      pack16(v[6], v[7], true));
  return make_uint4(pack16(v[0], v[1], false), pack16(v[2], v[3], false),
                    pack16(v[4], v[5], false), pack16(v[6], v[7], false));
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int type) {
  if (type == LILY_DTYPE_F32) return static_cast<const float*>(p)[i];
  return lo16_f32(static_cast<const uint16_t*>(p)[i], type == LILY_DTYPE_F16);
}

__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Sum over the WPR warps of a row (tmp: one float per warp of the block).
// fmaxf drops a NaN, so NaN reaches the scales through the norm's factor
// instead (see below).
template <int WPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? fmaxf(v, u) : v + u;
  }
  if (WPR == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) tmp[warp] = v;
  __syncthreads();
  const int first = warp / WPR * WPR;
  v = tmp[first];
#pragma unroll
  for (int w = 1; w < WPR; ++w) v = MAX ? fmaxf(v, tmp[first + w]) : v + tmp[first + w];
  return v;
}

// A row on WPR warps, C chunks of eight elements per thread.  VEC: chunk c of
// thread t covers columns 8 (c*threads + t) .. +7; else its elements are the
// columns (8c + e)*threads + t, one at a time (any alignment).
// XT, RT, OT: element types known when compiling, -1: asked at run time (OT 0:
// one of the 16-bit types).  Asked at run time they cost half of the issue
// slots, which then bound the kernel (16384 rows of 4096 into 8 bits: 93 us).
template <int WPR, int C, bool VEC, int XT, int RT, int OT>
__global__ void __launch_bounds__(WPR * 32 > 256 ? WPR * 32 : 256)
    add_rmsnorm_kernel(const NormArgs a) {
  constexpr int kTPR = WPR * 32;
  constexpr int kThreads = kTPR > 256 ? kTPR : 256;
  constexpr int kRows = kThreads / kTPR;
  const int xt = XT >= 0 ? XT : a.xt, rt = RT >= 0 ? RT : a.rt;
  const bool bits8 = OT >= 0 ? OT == LILY_DTYPE_E4M3 : a.ot == LILY_DTYPE_E4M3;
  __shared__ float tmp[2][kThreads / 32];
  __shared__ uint32_t gmax[VEC ? 1 : kRows][VEC ? 1 : 256];  // element-wise groups: bits of the maxima

  const int t = threadIdx.x % kTPR;
  const int sub = threadIdx.x / kTPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + sub;
  const bool live = row < a.T;
  auto col = [&](int c, int e) { return VEC ? 8 * (c * kTPR + t) + e : (8 * c + e) * kTPR + t; };

  pdl_wait();
  pdl_trigger();

  float r[C][8];
  const int64_t xi = row * a.x_stride, ri = row * a.res_stride;
  if (VEC) {
    Raw8 rx[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (live && col(c, 0) < a.d) {
        load_raw8(rx[c], a.x, xi + col(c, 0), xt);
        if (a.res) load_raw8(rr[c], a.res, ri + col(c, 0), rt);
      }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (live && col(c, 0) < a.d) {
        unpack8(rx[c], xt, r[c]);
        if (a.res) {
          float v[8];
          unpack8(rr[c], rt, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[c][e] += v[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = 0.f;
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        r[c][e] = live && col(c, e) < a.d ? load1(a.x, xi + col(c, e), xt) : 0.f;
    if (a.res)
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (live && col(c, e) < a.d) r[c][e] += load1(a.res, ri + col(c, e), rt);
  }

  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(r[c][e], r[c][e], ss);
  ss = row_reduce<WPR, false>(ss, tmp[0]);
  const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);

  // the rounded residual leaves, and r becomes n
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (VEC) {
      if (!(live && col(c, 0) < a.d)) continue;
      if (a.res_out) {
        const int64_t o = row * a.res_out_stride + col(c, 0);
        if (rt == LILY_DTYPE_F32) {
          float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.res_out) + o);
          p[0] = make_float4(r[c][0], r[c][1], r[c][2], r[c][3]);
          p[1] = make_float4(r[c][4], r[c][5], r[c][6], r[c][7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.res_out) + o) =
              pack8(r[c], rt == LILY_DTYPE_F16);
        }
      }
      if (a.w) {
        float w[8];
        Raw8 rw;
        load_raw8(rw, a.w, col(c, 0), a.wt);
        unpack8(rw, a.wt, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] *= rstd * w[e];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] *= rstd;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!(live && col(c, e) < a.d)) continue;
        if (a.res_out) {
          const int64_t o = row * a.res_out_stride + col(c, e);
          if (rt == LILY_DTYPE_F32) static_cast<float*>(a.res_out)[o] = r[c][e];
          else static_cast<uint16_t*>(a.res_out)[o] = pack1(r[c][e], rt == LILY_DTYPE_F16);
        }
        r[c][e] *= a.w ? rstd * load1(a.w, col(c, e), a.wt) : rstd;
      }
    }
  }

  if (!bits8) {
    const bool h = a.ot == LILY_DTYPE_F16;
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (VEC) {
        if (live && col(c, 0) < a.d)
          *reinterpret_cast<uint4*>(out + col(c, 0)) = pack8(r[c], h);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (live && col(c, e) < a.d) out[col(c, e)] = pack1(r[c][e], h);
      }
    }
    return;
  }

  // E4M3.  max|n| of each group; the group's columns lie on 8 or 16
  // neighbouring lanes (VEC), or go through shared memory.  A NaN must reach
  // its group's scale: maxima are taken on the bits of |n|, where NaN is
  // above every number.
  const bool per_row = a.group == 0;
  const int n_groups = per_row ? 1 : a.d / a.group;
  uint32_t m[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    m[c] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[c] = max(m[c], __float_as_uint(r[c][e]) & 0x7FFFFFFFu);
  }
  if (per_row) {
#pragma unroll
    for (int c = 1; c < C; ++c) m[0] = max(m[0], m[c]);
    m[0] = __reduce_max_sync(0xffffffffu, m[0]);
    if (WPR > 1) {
      const int warp = threadIdx.x >> 5, first = warp / WPR * WPR;
      if ((threadIdx.x & 31) == 0) tmp[1][warp] = __uint_as_float(m[0]);
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WPR; ++w) m[0] = max(m[0], __float_as_uint(tmp[1][first + w]));
    }
#pragma unroll
    for (int c = 1; c < C; ++c) m[c] = m[0];
  } else if (VEC) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], 1));
      m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], 2));
      m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], 4));
      if (a.group == 128) m[c] = max(m[c], __shfl_xor_sync(0xffffffffu, m[c], 8));
    }
  } else {
    for (int g = threadIdx.x; g < kRows * 256; g += kThreads) (&gmax[0][0])[g] = 0;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (live && col(c, e) < a.d)
          atomicMax(&gmax[sub][col(c, e) / a.group], __float_as_uint(r[c][e]) & 0x7FFFFFFFu);
    __syncthreads();
  }
  if (!live) return;

  float* sc = a.scales + row * n_groups;
  uint8_t* out = static_cast<uint8_t*>(a.out) + row * a.out_stride;
  // n / s as n * (448 / max); where that would not be a normal number, divided
  // (the last bits of the quotient are lost in e4m3's rounding, and the largest
  // value still lands on 448)
  constexpr float kTiny = 1e-30f, kStep = 1.f / 448.f;
  if (per_row && t == 0) sc[0] = __uint_as_float(m[0]) * kStep;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (VEC) {
      if (col(c, 0) >= a.d) continue;
      const float top = __uint_as_float(m[c]), s = top * kStep;
      if (!per_row && (col(c, 0) & (a.group - 1)) == 0) sc[col(c, 0) / a.group] = s;
      if (s > 0.f && s < kTiny) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = r[c][e] / s;
      } else {
        const float inv = top == 0.f ? 0.f : __fdividef(448.f, top);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] *= inv;
      }
      uint2 o;
      o.x = e4m3x2(r[c][0], r[c][1]) | (uint32_t)e4m3x2(r[c][2], r[c][3]) << 16;
      o.y = e4m3x2(r[c][4], r[c][5]) | (uint32_t)e4m3x2(r[c][6], r[c][7]) << 16;
      *reinterpret_cast<uint2*>(out + col(c, 0)) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = col(c, e);
        if (i >= a.d) continue;
        const float s = __uint_as_float(per_row ? m[0] : gmax[sub][i / a.group]) * kStep;
        if (!per_row && i % a.group == 0) sc[i / a.group] = s;
        const float q = s == 0.f ? 0.f : r[c][e] / s;
        out[i] = (uint8_t)e4m3x2(q, 0.f);
      }
    }
  }
}

template <int WPR, int C, int XT, int RT, int OT>
cudaError_t launch_types(const NormArgs& a, bool vec, cudaStream_t s) {
  constexpr int kThreads = WPR * 32 > 256 ? WPR * 32 : 256;
  constexpr int kRows = kThreads / (WPR * 32);
  const unsigned grid = (unsigned)(((int64_t)a.T + kRows - 1) / kRows);
  if (XT < 0 && !vec)
    return launch_pdl(add_rmsnorm_kernel<WPR, C, false, -1, -1, -1>, dim3(grid), dim3(kThreads), 0, s, a);
  return launch_pdl(add_rmsnorm_kernel<WPR, C, true, XT, RT, OT>, dim3(grid), dim3(kThreads), 0, s, a);
}
// The types of one kind throughout, with an fp32 residual or without one, are
// compiled in; other mixtures, and rows of any alignment, ask at run time.
template <int WPR, int C>
cudaError_t launch_as(const NormArgs& a, bool vec, cudaStream_t s) {
  constexpr int B = LILY_DTYPE_BF16, H = LILY_DTYPE_F16, F = LILY_DTYPE_F32, Q = LILY_DTYPE_E4M3;
  const bool q = a.ot == Q;
  if (vec && (a.rt == F || a.rt == a.xt)) {
    if (a.xt == B && a.rt == B) return q ? launch_types<WPR, C, B, B, Q>(a, vec, s) : launch_types<WPR, C, B, B, 0>(a, vec, s);
    if (a.xt == B) return q ? launch_types<WPR, C, B, F, Q>(a, vec, s) : launch_types<WPR, C, B, F, 0>(a, vec, s);
    if (a.xt == H && a.rt == H) return q ? launch_types<WPR, C, H, H, Q>(a, vec, s) : launch_types<WPR, C, H, H, 0>(a, vec, s);
    if (a.xt == H) return q ? launch_types<WPR, C, H, F, Q>(a, vec, s) : launch_types<WPR, C, H, F, 0>(a, vec, s);
    return q ? launch_types<WPR, C, F, F, Q>(a, vec, s) : launch_types<WPR, C, F, F, 0>(a, vec, s);
  }
  return launch_types<WPR, C, -1, -1, -1>(a, vec, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, bool vec, cudaStream_t s) {
  prof_begin(K_ATTN_NORM, s);
  const int n8 = (a.d + 7) / 8;  // chunks of a row
  cudaError_t e;
  if (n8 <= 32) e = launch_as<1, 1>(a, vec, s);
  else if (n8 <= 128) e = launch_as<4, 1>(a, vec, s);
  else if (n8 <= 256) e = launch_as<8, 1>(a, vec, s);
  else if (n8 <= 512) e = launch_as<8, 2>(a, vec, s);
  else e = launch_as<16, 4>(a, vec, s);
  prof_end(K_ATTN_NORM, s);
  return e;
}

}  // namespace lily
