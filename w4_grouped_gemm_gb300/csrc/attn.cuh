// attn.cuh -- launch arguments and device helpers of the attention-side
// kernels (include/lily_attn.h).
#pragma once
#include "../../include/lily_attn.h"
#include "common.cuh"

namespace lily {

// Kinds of the per-kernel event timing beside lily_internal.h's.
enum AttnKernelKind : int {
  K_ATTN_NORM = 8,
  K_ATTN_APPEND = 10,
  K_ATTN_KEYS = 11,
  K_ATTN_MERGE = 15,
};

// ---------------------------------------------------------------- norm
struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* res_out;
  void* out;
  float* scales;
  int64_t x_stride, res_stride, res_out_stride, out_stride;
  int T, d, xt, rt, wt, ot, group;
  float eps;
};
cudaError_t launch_add_rmsnorm(const NormArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- rope + append
struct RopeArgs {
  const void *q, *k, *v;
  void *qo, *kc, *vc;
  const int32_t* pos;
  const int64_t* slots;
  const double* inv_freq;
  int32_t q_tok, q_head, k_tok, k_head, v_tok, v_head, qo_tok, qo_head;
  int64_t c_page, c_head, c_tok, n_slots;
  int T, hq, hkv, D, rot, style, page_shift, dtype;
  uint32_t* status;
  // an 8-bit cache (kc and vc are e4m3 codes): its scales, else NULL
  float *ks, *vs;
  int64_t s_page, s_head, s_tok;
};
cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s);

// LILY_OK on the library's device (compute capability 10.3), else the error code (api.cu).
int device_rc();
// SMs of the current device, asked once for each; 0 on a CUDA error (attn.cu).
int device_sms();

// ---------------------------------------------------------------- attention
// One set of sequences: the batch's own pages, or the shared prefix as one
// sequence that every query token belongs to.  A unit is one sequence, one KV
// head and one block of `rows` query rows (row r of a sequence = token r / G,
// query head h*G + r % G); units are numbered ((seq * n_kv_heads + h) *
// row_blocks + block).  The units' tiles of 64 keys form one list that the
// CTAs share out in equal runs, so a unit may be cut anywhere; the part of
// unit u that CTA c computed is partial u + c of the set.
struct AttnSet {
  const int32_t* q_start;  // NULL: sequence s owns tokens s*max_q_len ...
  const int32_t* lens;     // NULL: every sequence has max_len keys
  const int32_t* table;
  int n_seqs, max_q_len, max_len, table_stride;
  int rows, row_blocks;    // 8, 16, 32 or 64; ceil(max_q_len * G / rows)
  int causal;              // query j of q sees keys 0 .. len - q + j
  int min_share;           // tiles a CTA takes, at least
  int grid;                // CTAs; at most one per tile
  float* part_o;           // [units + grid][rows][D] normalised partial outputs
  float* part_lse;         // [units + grid][rows] log2 of their softmax sums
  int4* rows_at;           // [T][hq] (own pages) where a row's partials lie: the first
                           // partial, the row in it, their number, the sequence
};

struct AttnArgs {
  const void* q;
  int64_t q_tok, q_head;
  int T, hq, hkv, G, D, page_shift, n_pages, f16;
  float scale_log2;  // softmax scale * log2(e)
  uint32_t* status;
  // tries of a wait before it gives up (attn_set_wait): of the warps that bring
  // keys or issue MMAs, and of those that compute
  uint32_t wait_feed, wait_use;
};

// The shared prefix on the tensor cores of a batch with more than 64 rows per
// KV head (attn_tc.cu): units of block_rows rows, numbered h * row_blocks +
// block, whose 128-key tiles the CTAs share out as above.
struct TcArgs {
  const int32_t* pages;
  int len, tiles, share, total;  // keys; tiles of a unit, of a CTA, of all units
  int row_blocks, block_rows;    // 256 rows (paired) or 128
  int paired;
  int grid;
  float* part_o;    // [units + grid][attn_tc_rows(D)][D]
  float* part_lse;  // [units + grid][attn_tc_rows(D)]
};
constexpr int kTcKeys = 128;     // keys of a tile
constexpr int kTcMaxGrid = 160;  // CTAs, at most
int attn_tc_v_keys(int D);
int attn_tc_rows(int D);
cudaError_t launch_attn_prefix_tc(const AttnArgs& a, const TcArgs& p, const CUtensorMap& mk,
                                  const CUtensorMap& mv, cudaStream_t s);

struct MergeArgs {
  AttnSet own;  // (rows_at NULL: no own keys, the sequences are only looked at)
  // the prefix's partials: key tiles of a unit and of a CTA (0: no prefix);
  // row blocks of a KV head and their rows; rows of a partial, and partials
  // of one row in it, 128 rows apart (two where streams took alternate tiles)
  int pre_tiles, pre_share, pre_blocks, pre_rows, pre_slot_rows, pre_streams;
  int own_slots;  // partials that the own set has room for
  int own_parts;  // partials of a sequence's own keys, if all sequences were the longest
  const float* pre_o;
  const float* pre_lse;
  void* out;
  float* lse;
  int64_t out_tok, out_head;
};

constexpr int kAttnTile = 64;      // keys of a tile
// Head dimension that the kernels are built for: D rounded up.
__host__ __device__ constexpr int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
constexpr int kAttnMaxGrid = 512;  // CTAs of a key kernel, at most (sizes the workspace)

// CTAs of the key kernel on the current device for a head of D elements.
int attn_grid(int D);
// The partials of the prefix (pa) and the own pages (pb; not fewer rows in pa),
// or of one set (pb.grid 0); first: the call's first launch (attn.cu).
cudaError_t launch_attn_keys(const AttnArgs& a, const AttnSet& pa, const AttnSet& pb,
                             const CUtensorMap& mk, const CUtensorMap& mv, bool first,
                             cudaStream_t s);
cudaError_t launch_attn_keys_bf16(const AttnArgs& a, const AttnSet& pa, const AttnSet& pb,
                                  const CUtensorMap& mk, const CUtensorMap& mv, bool first,
                                  cudaStream_t s);
cudaError_t launch_attn_keys_f16(const AttnArgs& a, const AttnSet& pa, const AttnSet& pb,
                                 const CUtensorMap& mk, const CUtensorMap& mv, bool first,
                                 cudaStream_t s);
// Their merge into out and lse.
cudaError_t launch_attn_merge(const AttnArgs& a, const MergeArgs& m, cudaStream_t s);

// ---------------------------------------------------------------- sequences
// A sequence's query tokens and own keys, held inside the call's bounds.
struct SeqInfo {
  int q0, qn, len;
  bool bad;
};
// r.q0, and q1, the token after its last, and r.len, as they were given.
__device__ __forceinline__ void hold_tokens(SeqInfo& r, const AttnSet& s, int T, int q1) {
  if (r.q0 < 0 || r.q0 > T || q1 < r.q0 || q1 > T || q1 - r.q0 > s.max_q_len) {
    r.bad = true;
    r.q0 = min(max(r.q0, 0), T);
    q1 = min(max(q1, r.q0), min(T, r.q0 + s.max_q_len));
  }
  r.qn = q1 - r.q0;
}
__device__ __forceinline__ void hold_len(SeqInfo& r, const AttnSet& s) {
  if (r.len < 0 || r.len > s.max_len) {
    r.bad = true;
    r.len = min(max(r.len, 0), s.max_len);
  }
}
__device__ __forceinline__ SeqInfo seq_info(const AttnSet& s, int T, int i) {
  SeqInfo r;
  r.bad = false;
  int q1;
  if (s.q_start) {
    r.q0 = s.q_start[i];
    q1 = s.q_start[i + 1];
  } else {
    r.q0 = i * s.max_q_len;
    q1 = r.q0 + s.max_q_len;
  }
  hold_tokens(r, s, T, q1);
  r.len = s.lens ? s.lens[i] : s.max_len;
  hold_len(r, s);
  return r;
}

// ---------------------------------------------------------------- copies, waits, 2^x
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(tm), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
// Bounded wait of a whole warp, each lane on its own barrier: `tries` of them,
// each of which suspends the thread until the phase is complete, for kTryNs at
// most (measured on this GPU: 3.95 to 4.05 us, whatever suspend-time hint a try is
// given).  On giving up it sets *abort and the TIMEOUT status; the CTA's other
// roles, which then wait in vain too, give up by themselves.  The loop is a handful
// of instructions on purpose: with a time limit in line (%globaltimer, a second
// vote) each wait cost some 250 cycles even where it passed at once, plain polling
// took issue slots from the warps that compute, and a look at *abort after a try
// that failed took 4 percent of the tensor-core prefix (142 -> 148 us for 256
// sequences behind 32768 keys).
constexpr uint64_t kTryNs = 4000;
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint32_t tries, uint32_t* status) {
  bool ok = false;
  for (uint32_t n = 0; n < tries && !ok; ++n) ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  *abort = 1;
  set_status(status, LILY_STATUS_TIMEOUT);
  return false;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The z of a softmax, 2^(c score - z), for a largest c score of zx.  fp16 loses
// bits below 2^-14 and all below 2^-25, so with an fp16 cache the probabilities are
// held `up` powers of two above those of a z of zx; the factor is in their sum too.
// (A row with one dominant key over 131072 others of weight 2^-26 lost their 0.2
// percent of the output.)  Where zx is so large that zx - up would be a coarse
// number, z is zx: a rounding of z must not take them past fp16's range.
constexpr float kFineZ = 1048576.f;
template <bool F16>
__device__ __forceinline__ float softmax_z(float zx, float up) {
  return F16 && fabsf(zx) < kFineZ ? zx - up : zx;
}

// ---------------------------------------------------------------- 16-bit elements
__device__ __forceinline__ float lo16_f32(uint32_t w, bool f16) {
  return f16 ? __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)))
             : __uint_as_float(w << 16);
}
__device__ __forceinline__ float hi16_f32(uint32_t w, bool f16) {
  return f16 ? __half2float(__ushort_as_half((unsigned short)(w >> 16)))
             : __uint_as_float(w & 0xFFFF0000u);
}
// Two floats rounded to a pair of 16-bit elements (a in the low half).
__device__ __forceinline__ uint32_t pack16(float a, float b, bool f16) {
  uint32_t r;
  if (f16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// One float rounded to a 16-bit element.
__device__ __forceinline__ uint16_t pack1(float a, bool f16) {
  return f16 ? __half_as_ushort(__float2half_rn(a)) : __bfloat16_as_ushort(__float2bfloat16_rn(a));
}

}  // namespace lily
