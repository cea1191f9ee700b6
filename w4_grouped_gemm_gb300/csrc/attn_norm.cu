// attn_norm.cu -- residual addition and RMSNorm, with 16-bit rows or 8-bit
// rows and scales out (lily_attn_add_rmsnorm).
//
//   r = residual + x,  n_i = r_i / sqrt(mean(r^2) + eps) * w_i,
//   8 bits: s_g = max over group g of |n_i| / 448,  out_i = e4m3(n_i / s_g)
//
// One pass: a row stays in registers between its sum of squares, the maxima
// of its groups and its stores, so that x and the residual are read once and
// the outputs written once.  HBM bounds it from some hundred rows on, the
// latency of one load and two block reductions below.  Measured: 8192 fp32 rows
// of 2048 into bf16 35.6 us, 235 MB, 6.6 TB/s (0.98 of a copy); 16384 bf16 rows
// of 4096 into 8 bits with a scale per 128 columns 77.6 us, 472 MB, 6.1 TB/s; one
// row of 2048 2.1 us in a graph.
#include <climits>
#include <cuda_fp8.h>
#include <type_traits>

#include "attn.cuh"

namespace lily {
namespace {

constexpr int kMaxWarps = 16;  // of a block

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

__device__ __forceinline__ void store1(void* p, int64_t i, float v, int type) {
  if (type == LILY_DTYPE_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = pack1(v, type == LILY_DTYPE_F16);
}

__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

// Sum over the warps of a row: WPR of them, or the whole block (0).  tmp: a
// float per warp of the block.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* tmp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (WPR == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) tmp[warp] = v;
  __syncthreads();
  if (WPR == 0) {
    const int lane = threadIdx.x & 31;
    v = lane < (int)blockDim.x >> 5 ? tmp[lane] : 0.f;
#pragma unroll
    for (int o = kMaxWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return __shfl_sync(0xffffffffu, v, 0);
  }
  const int first = warp / (WPR ? WPR : 1) * WPR;
  v = tmp[first];
#pragma unroll
  for (int w = 1; w < WPR; ++w) v += tmp[first + w];
  return v;
}

// r[e] *= f * w for the columns O before a boundary of eight: w[0..7] are the
// weights of the eight columns before it, w[8..15] those from it on.
template <int O>
__device__ __forceinline__ void scale8(float (&r)[8], const float (&w)[16], float f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] *= f * w[8 - O + e];
}

// How a row's elements lie on its threads, C chunks of eight per thread:
//   kWhole: chunk c of thread t covers columns 8 (c*threads + t) .. +7
//   kShift: the same, less the row's first element's distance from a boundary
//     of eight (rows of odd widths one behind the other: every operand of a
//     row has the same distance).  The first and last chunk's vectors reach
//     into the neighbouring rows, whose elements count as zeros and are not
//     written; only past the last row are they loaded one by one.  The
//     weights, which have no distance, come as two vectors and a uniform
//     choice of eight shifts.  (10394 fp32 rows of 4426 into 8 bits: 113 us;
//     element by element 293.)
//   kAny: columns (8c + e)*threads + t, one at a time
enum Lay { kAny, kWhole, kShift };

// A row on WPR warps, or on a block of as many warps as its chunks need (0).
// XT, RT, OT: element types known when compiling, -1: asked at run time (OT 0:
// one of the 16-bit types).  Asked at run time they cost half of the issue
// slots, which then bound the kernel (16384 rows of 4096 into 8 bits: 93 us).
template <int WPR, int C, Lay LAY, int XT, int RT, int OT>
__global__ void __launch_bounds__(WPR ? 256 : 32 * kMaxWarps)
    add_rmsnorm_kernel(const NormArgs a) {
  constexpr bool VEC = LAY != kAny;
  constexpr int kRows = WPR ? 8 / WPR : 1;  // rows of a block
  const int kThreads = WPR ? 256 : blockDim.x, kTPR = WPR ? WPR * 32 : blockDim.x;
  const int xt = XT >= 0 ? XT : a.xt, rt = RT >= 0 ? RT : a.rt;
  const bool bits8 = OT >= 0 ? OT == LILY_DTYPE_E4M3 : a.ot == LILY_DTYPE_E4M3;
  __shared__ float tmp[2][kMaxWarps];
  __shared__ uint32_t gmax[VEC ? 1 : kRows][VEC ? 1 : 256];  // element-wise groups: bits of the maxima

  const int t = threadIdx.x % kTPR;
  const int sub = threadIdx.x / kTPR;
  const int64_t row = (int64_t)blockIdx.x * kRows + sub;
  const bool live = row < a.T;
  const int shift = LAY == kShift ? (int)(row * a.x_stride & 7) : 0;
  auto col = [&](int c, int e) { return VEC ? 8 * (c * kTPR + t) + e - shift : (8 * c + e) * kTPR + t; };
  auto inside = [&](int c, int e) { return col(c, e) >= 0 && col(c, e) < a.d; };
  auto some = [&](int c) { return live && col(c, 0) < a.d && (LAY != kShift || col(c, 7) >= 0); };
  auto whole = [&](int c) { return LAY != kShift || (col(c, 0) >= 0 && col(c, 7) < a.d); };
  // columns from this row's first on that are there in every operand
  const int there = LAY == kShift ? (int)min((int64_t)(a.T - row) * a.d, (int64_t)INT_MAX) : 0;
  auto vectors = [&](int c) { return some(c) && (LAY != kShift || col(c, 7) < there); };

  pdl_wait();
  pdl_trigger();

  float r[C][8];
  const int64_t xi = row * a.x_stride, ri = row * a.res_stride;
  if (VEC) {
    Raw8 rx[C], rr[C];
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (vectors(c)) {
        load_raw8(rx[c], a.x, xi + col(c, 0), xt);
        if (a.res) load_raw8(rr[c], a.res, ri + col(c, 0), rt);
      }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (LAY == kShift && some(c) && !vectors(c)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          r[c][e] = inside(c, e) ? load1(a.x, xi + col(c, e), xt) +
                                       (a.res ? load1(a.res, ri + col(c, e), rt) : 0.f)
                                 : 0.f;
      } else if (some(c)) {
        unpack8(rx[c], xt, r[c]);
        if (a.res) {
          float v[8];
          unpack8(rr[c], rt, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) r[c][e] += v[e];
        }
        if (!whole(c)) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (!inside(c, e)) r[c][e] = 0.f;
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
  ss = row_sum<WPR>(ss, tmp[0]);
  const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);

  // the rounded residual leaves, and r becomes n
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (VEC) {
      if (!some(c)) continue;
      if (LAY == kShift && a.res_out && !whole(c)) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (inside(c, e)) store1(a.res_out, row * a.res_out_stride + col(c, e), r[c][e], rt);
      } else if (a.res_out) {
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
      if (a.w && LAY == kShift && shift) {
        float w[16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = col(c, 0) + shift - 8 + 8 * k;
          float v[8];
          if (at >= 0 && at + 8 <= a.d) {
            Raw8 raw;
            load_raw8(raw, a.w, at, a.wt);
            unpack8(raw, a.wt, v);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = at + e >= 0 && at + e < a.d ? load1(a.w, at + e, a.wt) : 0.f;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) w[8 * k + e] = v[e];
        }
        switch (shift) {
          case 1: scale8<1>(r[c], w, rstd); break;
          case 2: scale8<2>(r[c], w, rstd); break;
          case 3: scale8<3>(r[c], w, rstd); break;
          case 4: scale8<4>(r[c], w, rstd); break;
          case 5: scale8<5>(r[c], w, rstd); break;
          case 6: scale8<6>(r[c], w, rstd); break;
          default: scale8<7>(r[c], w, rstd);
        }
      } else if (a.w) {  // (in the first row of kShift the last chunk may be partial)
        float w[8];
        if (LAY == kShift && col(c, 7) >= a.d) {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = inside(c, e) ? load1(a.w, col(c, e), a.wt) : 0.f;
        } else {
          Raw8 rw;
          load_raw8(rw, a.w, col(c, 0), a.wt);
          unpack8(rw, a.wt, w);
        }
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
        if (a.res_out) store1(a.res_out, row * a.res_out_stride + col(c, e), r[c][e], rt);
        r[c][e] *= a.w ? rstd * load1(a.w, col(c, e), a.wt) : rstd;
      }
    }
  }

  if (!bits8) {
    const bool h = a.ot == LILY_DTYPE_F16;
    uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_stride;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (VEC && some(c) && whole(c)) {
        *reinterpret_cast<uint4*>(out + col(c, 0)) = pack8(r[c], h);
      } else if (!VEC || (LAY == kShift && some(c))) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (live && inside(c, e)) out[col(c, e)] = pack1(r[c][e], h);
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
    if (WPR != 1) {
      const int warp = threadIdx.x >> 5;
      const int lane = threadIdx.x & 31;
      if (lane == 0) tmp[1][warp] = __uint_as_float(m[0]);
      __syncthreads();
      if (WPR == 0) {
        m[0] = __reduce_max_sync(0xffffffffu, lane < (int)blockDim.x >> 5 ? __float_as_uint(tmp[1][lane]) : 0u);
      } else {
        const int first = warp / (WPR ? WPR : 1) * WPR;
#pragma unroll
        for (int w = 0; w < WPR; ++w) m[0] = max(m[0], __float_as_uint(tmp[1][first + w]));
      }
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
  // n / s as n * (448 / max), both rounded to 32 bits like s and the quotient;
  // where 448 / max would not be a normal number, divided.  A maximum so small
  // that s rounds to 0 gives 0, like one that is 0 (448 / max would be infinite
  // there, and 0 times it NaN).
  constexpr float kTiny = 1e-30f, kStep = 1.f / 448.f;
  if (per_row && t == 0) sc[0] = __uint_as_float(m[0]) * kStep;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (VEC) {
      if (!some(c)) continue;
      const float top = __uint_as_float(m[c]), s = top * kStep;
      if (!per_row && (col(c, 0) & (a.group - 1)) == 0) sc[col(c, 0) / a.group] = s;
      if (s > 0.f && s < kTiny) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] = r[c][e] / s;
      } else {
        const float inv = s == 0.f ? 0.f : 448.f / top;
#pragma unroll
        for (int e = 0; e < 8; ++e) r[c][e] *= inv;
      }
      uint2 o;
      o.x = e4m3x2(r[c][0], r[c][1]) | (uint32_t)e4m3x2(r[c][2], r[c][3]) << 16;
      o.y = e4m3x2(r[c][4], r[c][5]) | (uint32_t)e4m3x2(r[c][6], r[c][7]) << 16;
      if (whole(c)) {
        *reinterpret_cast<uint2*>(out + col(c, 0)) = o;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (inside(c, e)) out[col(c, e)] = (uint8_t)((e < 4 ? o.x : o.y) >> (8 * (e & 3)));
      }
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
cudaError_t launch_types(const NormArgs& a, Lay lay, int chunks, cudaStream_t s) {
  constexpr int kRows = WPR ? 8 / WPR : 1;
  const dim3 grid((unsigned)(((int64_t)a.T + kRows - 1) / kRows));
  const dim3 threads(WPR ? 256 : (chunks + 32 * C - 1) / (32 * C) * 32);
  if (XT < 0 && lay == kAny)
    return launch_pdl(add_rmsnorm_kernel<WPR, C, kAny, -1, -1, -1>, grid, threads, 0, s, a);
  if (WPR != 8 && lay == kShift)
    return launch_pdl(add_rmsnorm_kernel<WPR, C, WPR == 8 ? kWhole : kShift, XT, RT, OT>, grid, threads, 0, s, a);
  return launch_pdl(add_rmsnorm_kernel<WPR, C, kWhole, XT, RT, OT>, grid, threads, 0, s, a);
}
// The types of one kind throughout, with an fp32 residual or without one, are
// compiled in; other mixtures, and rows of any alignment, ask at run time.
template <int WPR, int C>
cudaError_t launch_as(const NormArgs& a, Lay lay, int n8, cudaStream_t s) {
  constexpr int B = LILY_DTYPE_BF16, H = LILY_DTYPE_F16, F = LILY_DTYPE_F32, Q = LILY_DTYPE_E4M3;
  constexpr bool kOnly8 = WPR == 8 && C == 4;  // (16-bit rows do not come here)
  auto types = [&](auto x, auto r) {
    constexpr int X = decltype(x)::value, R = decltype(r)::value;
    return a.ot == Q ? launch_types<WPR, C, X, R, Q>(a, lay, n8, s)
                     : launch_types<WPR, C, X, R, kOnly8 ? Q : 0>(a, lay, n8, s);
  };
  using Bf = std::integral_constant<int, B>;
  using Hf = std::integral_constant<int, H>;
  using Ff = std::integral_constant<int, F>;
  if (lay != kAny && (a.rt == F || a.rt == a.xt)) {
    if (a.xt == B) return a.rt == B ? types(Bf(), Bf()) : types(Bf(), Ff());
    if (a.xt == H) return a.rt == H ? types(Hf(), Hf()) : types(Hf(), Ff());
    return types(Ff(), Ff());
  }
  return launch_types<WPR, C, -1, -1, -1>(a, lay, n8, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s) {
  // What the rows' addresses allow (the bases lie on 16 bytes).
  int64_t all[4] = {a.x_stride, a.out_stride, a.res ? a.res_stride : a.x_stride,
                    a.res_out ? a.res_out_stride : a.x_stride};
  const int types[4] = {a.xt, a.ot, a.rt, a.rt};
  bool same = a.group == 0, whole = a.d % 8 == 0;
  for (int i = 0; i < 4; ++i) {
    if (a.T == 1) all[i] = 0;  // (no second row)
    whole = whole && all[i] % (types[i] == LILY_DTYPE_F32 ? 4 : 8) == 0;
    same = same && (all[i] - all[0]) % 8 == 0;
  }
  int n8 = (a.d + 7) / 8;  // chunks of a row
  Lay lay = kAny;
  if (whole) {
    lay = kWhole;
  } else if (same && (a.d + 14) / 8 <= 2048) {
    lay = kShift;
    n8 = (a.d + 14) / 8;
  }
  // Rows that fill 13/16 of eight warps with C chunks a thread take eight warps known
  // when compiling, others a block of as many as they need.  Measured, a block of
  // any size against eight warps, 2^26 bf16 elements into 8 bits with groups of 128,
  // us: widths 1536 107 / 106, 1664 121 / 104, 1792 114 / 97, 2048 108 / 91;
  // 2816 89 / 91, 3328 90 / 84, 4096 84 / 77; 6144 86 / 82, 7168 91 / 80, 8192 89 /
  // 76; less filled ones lose (1152 119 / 129, 2304 88 / 103, 4608 86 / 95).  Into 16
  // bits, which HBM bounds, both take the same (2048 80 / 78, 4096 78 / 78) but with
  // four chunks eight warps are slower (8192, fp32 residual 117 / 119).
  auto fills = [&](int C) { return lay == kWhole && n8 <= 256 * C && 16 * n8 >= 13 * 256 * C; };
  prof_begin(K_ATTN_NORM, s);
  cudaError_t e;
  if (n8 <= 32) e = launch_as<1, 1>(a, lay, n8, s);
  else if (n8 <= 128) e = launch_as<4, 1>(a, lay, n8, s);
  else if (fills(1)) e = launch_as<8, 1>(a, lay, n8, s);
  else if (fills(2)) e = launch_as<8, 2>(a, lay, n8, s);
  else if (fills(4) && a.ot == LILY_DTYPE_E4M3) e = launch_as<8, 4>(a, lay, n8, s);
  // (kShift holds the weights of a chunk twice: one chunk per thread where that does)
  else if (n8 <= (lay == kShift ? 512 : 256)) e = launch_as<0, 1>(a, lay, n8, s);
  else if (n8 <= 1024) e = launch_as<0, 2>(a, lay, n8, s);
  else e = launch_as<0, 4>(a, lay, n8, s);
  prof_end(K_ATTN_NORM, s);
  return e;
}

}  // namespace lily
