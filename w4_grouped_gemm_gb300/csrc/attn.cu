// attn.cu -- the merge of attention's partial outputs, and the launches of
// lily_attn_shared_prefix's kernels (attn_keys.cuh, attn_tc.cu).
#include <atomic>
#include <type_traits>

#include "attn.cuh"

namespace lily {
namespace {

// A query row (token, query head) per W warps, 8 / W rows per block (W 16 and
// 32: one row in a block of W warps): the
// partials of the prefix and of the sequence's own keys, weighted by 2^(lse -
// largest lse) and added up.  Warp p of a row takes partials p, p + W, ..: a lane
// finds the weight of one of them, then all lanes add up their outputs, up to
// four at a time, two where rows are many and partials few: what counts then is
// rows in flight (26000 rows of two partials in a call: 52.4 us with four blocks
// of 64 registers on an SM, 47.1 with five of 48, 49.6 with six that spill).  What bounds it is the chain of loads (where a row's own
// partials lie, its sequence, lse, output), so the prefix's lse are requested
// with the first.  rows_at may hold anything for rows without own keys: an entry
// counts where its sequence has the row's token and keys, for then this call
// has written it, and where it lies within the partials.
template <int W>
__global__ void __launch_bounds__(W > 8 ? 32 * W : 256, W > 8 ? 32 / W : W == 1 ? 5 : 4)
    attn_merge_kernel(const AttnArgs a, const MergeArgs m) {
  constexpr int kWarps = W > 8 ? W : 8, kRows = kWarps / W;  // of a block
  __shared__ __align__(16) float acc_s[W > 1 ? kWarps : 1][W > 1 ? 256 : 4];
  __shared__ float2 ms_s[kWarps];  // largest lse and sum of weights of a warp
  __shared__ float f_s[kWarps], inv_s[kRows];  // a warp's factor, a row's last one
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = warp % W;  // of the row's warps
  const int rows = a.T * a.hq;  // (at most 2^30: 65536 tokens of 16384 heads)
  const int row = blockIdx.x * kRows + warp / W;
  const bool live = row < rows;
  const int t = row / a.hq, hq = row - t * a.hq;
  // partials [p0, p0 + np) of the prefix at row pr
  int p0 = 0, np = 0, pr = 0;
  if (live && m.pre_tiles) {
    const int h = hq / a.G;
    const int r = t * a.G + hq - h * a.G;
    const int u = h * m.pre_blocks + r / m.pre_rows;
    const int c0 = u * m.pre_tiles / m.pre_share;
    p0 = u + c0;
    np = (((u + 1) * m.pre_tiles - 1) / m.pre_share - c0 + 1) * m.pre_streams;
    pr = r % m.pre_rows;
  }
  auto pre_row = [&](int i) {  // row of partial i of the prefix
    return m.pre_streams == 1
               ? (int64_t)(p0 + i) * m.pre_slot_rows + pr
               : (int64_t)(p0 + (i >> 1)) * m.pre_slot_rows + (i & 1) * 128 + pr;
  };
  pdl_wait();
  pdl_trigger();
  if (!m.own.rows_at && blockIdx.x == 0)  // (no own keys: no key kernel has looked at the sequences)
    for (int i = threadIdx.x; i < m.own.n_seqs; i += blockDim.x)
      if (seq_info(m.own, a.T, i).bad) set_status(a.status, LILY_STATUS_BAD_LEN);
  const int first = part + W * lane;
  const float pre0 = first < np ? m.pre_lse[pre_row(first)] : -INFINITY;
  // partials [w0, w0 + nw) of the sequence at row wrow
  int w0 = 0, nw = 0, wrow = 0;
  if (live && m.own.rows_at) {
    const int4 at = m.own.rows_at[row];
    if (at.w >= 0 && at.w < m.own.n_seqs) {
      const SeqInfo q = seq_info(m.own, a.T, at.w);
      // (a CTA that gave up may not have written it: it may be a former call's then)
      const bool inside = at.x >= 0 && at.z >= 0 && at.z <= m.own_slots &&
                          at.x <= m.own_slots - at.z && at.y >= 0 && at.y < m.own.rows;
      if (t >= q.q0 && t < q.q0 + q.qn && q.len > 0 && inside) {
        w0 = at.x;
        wrow = at.y;
        nw = at.z;
      }
    }
  }
  const int n = np + nw;
  auto own_row = [&](int i) { return (int64_t)(w0 + i - np) * m.own.rows + wrow; };

  float M = -INFINITY, sum = 0.f;
  float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = 0; part + W * k0 < n; k0 += 32) {
    const int i = part + W * (k0 + lane);
    float lse = k0 == 0 ? pre0 : i < np ? m.pre_lse[pre_row(i)] : -INFINITY;
    if (i >= np && i < n) lse = m.own.part_lse[own_row(i)];
    float x = lse;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    x = fmaxf(x, M);
    const float z = x == -INFINITY ? 0.f : x;
    const float wt = i < n ? exp2f(lse - z) : 0.f;
    const float f = M == -INFINITY ? 0.f : exp2f(M - z);
    M = x;
    sum = sum * f + warp_sum(wt);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      acc[k].x *= f;
      acc[k].y *= f;
      acc[k].z *= f;
      acc[k].w *= f;
    }
    const int cnt = min(32, (n - part - W * k0 + W - 1) / W);
    auto add = [&](auto wide) {
      constexpr int kWide = decltype(wide)::value;  // quads of columns per lane
      constexpr int kAt = (W == 1 ? 2 : 4) / kWide;
      for (int j0 = 0; j0 < cnt; j0 += kAt) {
        float4 v[kAt][kWide];
        float w[kAt];
#pragma unroll
        for (int j = 0; j < kAt; ++j) {
          w[j] = __shfl_sync(0xffffffffu, wt, min(j0 + j, 31));
          if (j0 + j >= cnt) w[j] = 0.f;  // (a partial of weight 0 may have no output)
          const int p = part + W * (k0 + j0 + j);
          const float* o = p < np ? m.pre_o + pre_row(p) * a.D : m.own.part_o + own_row(p) * a.D;
#pragma unroll
          for (int k = 0; k < kWide; ++k) {
            v[j][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (w[j] != 0.f && k * 128 + lane * 4 < a.D)
              v[j][k] = *reinterpret_cast<const float4*>(o + k * 128 + lane * 4);
          }
        }
#pragma unroll
        for (int j = 0; j < kAt; ++j)
#pragma unroll
          for (int k = 0; k < kWide; ++k) {
            acc[k].x = fmaf(w[j], v[j][k].x, acc[k].x);
            acc[k].y = fmaf(w[j], v[j][k].y, acc[k].y);
            acc[k].z = fmaf(w[j], v[j][k].z, acc[k].z);
            acc[k].w = fmaf(w[j], v[j][k].w, acc[k].w);
          }
      }
    };
    if (a.D <= 128) add(std::integral_constant<int, 1>());
    else add(std::integral_constant<int, 2>());
  }
  if (W > 1) {
    // the warps' sums through shared memory, added up by all threads
    if (lane == 0) ms_s[warp] = make_float2(M, sum);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      *reinterpret_cast<float4*>(&acc_s[W > 1 ? warp : 0][W > 1 ? k * 128 + lane * 4 : 0]) = acc[k];
    __syncthreads();
    if (threadIdx.x < kWarps) {
      const int r = threadIdx.x / W;
      float top = -INFINITY, total = 0.f;
      for (int w = 0; w < W; ++w) top = fmaxf(top, ms_s[r * W + w].x);
      const float z = top == -INFINITY ? 0.f : top;
      auto factor = [&](float2 o) {  // (NaN sums stay)
        return o.x == -INFINITY ? (o.y != o.y ? 1.f : 0.f) : exp2f(o.x - z);
      };
      f_s[threadIdx.x] = factor(ms_s[threadIdx.x]);
      if (threadIdx.x % W == 0) {
        for (int w = 0; w < W; ++w) total += ms_s[r * W + w].y * factor(ms_s[r * W + w]);
        inv_s[r] = total == 0.f ? 0.f : 1.f / total;
        const int64_t to = (int64_t)blockIdx.x * kRows + r;
        if (m.lse && to < rows)
          m.lse[to] = total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
      }
    }
    __syncthreads();
    const int quads = a.D >> 2;
    for (int i = threadIdx.x; i < kRows * quads; i += 32 * kWarps) {
      const int r = i / quads, c = 4 * (i - r * quads);
      const int to = blockIdx.x * kRows + r;
      if (to >= rows) break;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int w = 0; w < W; ++w) {
        const float f = f_s[r * W + w];
        const float4 x = *reinterpret_cast<const float4*>(&acc_s[W > 1 ? r * W + w : 0][W > 1 ? c : 0]);
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
      }
      const float inv = inv_s[r];
      const int tt = to / a.hq, hh = to - tt * a.hq;
      uint16_t* out = static_cast<uint16_t*>(m.out) + (int64_t)tt * m.out_tok + (int64_t)hh * m.out_head;
      *reinterpret_cast<uint2*>(out + c) = make_uint2(pack16(v.x * inv, v.y * inv, a.f16),
                                                      pack16(v.z * inv, v.w * inv, a.f16));
    }
    return;
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* out = static_cast<uint16_t*>(m.out) + (int64_t)t * m.out_tok + (int64_t)hq * m.out_head;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k * 128 + lane * 4 < a.D)
      *reinterpret_cast<uint2*>(out + k * 128 + lane * 4) =
          make_uint2(pack16(acc[k].x * inv, acc[k].y * inv, a.f16),
                     pack16(acc[k].z * inv, acc[k].w * inv, a.f16));
  if (m.lse && lane == 0) m.lse[row] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace

int attn_grid(int D) {
  static std::atomic<int> known[64];  // SMs of a device, once asked; 0: not yet
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64) sms = known[dev].load(std::memory_order_relaxed);
  if (sms == 0) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  }
  const int g = sms * (padded_dim(D) <= 128 ? 2 : 1);
  return g < kAttnMaxGrid ? g : kAttnMaxGrid;
}

cudaError_t launch_attn_keys(const AttnArgs& a, const AttnSet& pa, const AttnSet& pb,
                             const CUtensorMap& mk, const CUtensorMap& mv, bool first,
                             cudaStream_t s) {
  prof_begin(K_ATTN_KEYS, s);
  const cudaError_t e = a.f16 ? launch_attn_keys_f16(a, pa, pb, mk, mv, first, s)
                              : launch_attn_keys_bf16(a, pa, pb, mk, mv, first, s);
  prof_end(K_ATTN_KEYS, s);
  return e;
}

cudaError_t launch_attn_merge(const AttnArgs& a, const MergeArgs& m, cudaStream_t s) {
  prof_begin(K_ATTN_MERGE, s);
  // Warps for a row: one per two to four partials (the prefix's are known here;
  // a sequence's own, whose lengths only the device knows, are taken as if all
  // were the longest), as long as all rows' warps find a place on the GPU at
  // once: 1000 rows of 33 partials took 23.6 us of a call with 4 warps each,
  // 26.2 with 8 and 53.5 with 32; 256 rows of 67, 23.1 with 8, 21.8 with 16 and
  // 27.0 with 32; 16 rows of 17, 17.7 with 1, 12.1 with 8.
  int n = 0;
  if (m.pre_tiles) n += (m.pre_tiles / m.pre_share + 2) * m.pre_streams;
  if (m.own.rows_at) n += 1 + m.own_parts;
  const int64_t rows = (int64_t)a.T * a.hq;
  int w = 1;
  while (w < 32 && n > (rows * w < 8 * 152 ? 2 : 4) * w && rows * 2 * w <= 4096) w *= 2;
  const int per = w > 8 ? 1 : 8 / w;
  const dim3 grid((unsigned)((rows + per - 1) / per));
  auto launch = [&](auto kern) {
    return launch_pdl(kern, grid, dim3(w > 8 ? 32 * w : 256), 0, s, a, m);
  };
  const cudaError_t e = w == 1    ? launch(attn_merge_kernel<1>)
                        : w == 2  ? launch(attn_merge_kernel<2>)
                        : w == 4  ? launch(attn_merge_kernel<4>)
                        : w == 8  ? launch(attn_merge_kernel<8>)
                        : w == 16 ? launch(attn_merge_kernel<16>)
                                  : launch(attn_merge_kernel<32>);
  prof_end(K_ATTN_MERGE, s);
  return e;
}

}  // namespace lily
