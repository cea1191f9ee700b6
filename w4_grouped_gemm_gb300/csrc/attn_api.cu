// attn_api.cu -- the C ABI of include/lily_attn.h: argument checks, workspace
// layout and the launches of each call.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "attn.cuh"
#include "attn_share.h"

namespace lily {
namespace {

bool aligned(const void* p, size_t to) { return (uintptr_t)p % to == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
int rc_of(cudaError_t e) { return e == cudaSuccess ? LILY_OK : LILY_ERR_CUDA; }

// Give-up limit of the attention kernels' waits.
std::atomic<uint64_t> g_wait_ns{2000000000ull};

constexpr int64_t kMaxStride = (int64_t)1 << 39;

// A stride in elements: at least `least`, below 2^39.
bool stride_ok(int64_t s, int64_t least) { return s >= least && s < kMaxStride; }
bool head_stride_ok(int64_t s) { return s >= 0 && s < kMaxStride && s % 8 == 0; }

int check_cache(const lily_attn_cache* c) {
  if (!c || !c->k || !c->v) return LILY_ERR_INVALID_ARG;
  if (c->dtype != LILY_DTYPE_BF16 && c->dtype != LILY_DTYPE_F16) return LILY_ERR_UNSUPPORTED_SHAPE;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->head_dim < 1) return LILY_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128 &&
      c->page_size != 256)
    return LILY_ERR_UNSUPPORTED_SHAPE;
  if (c->n_kv_heads > 256 || c->head_dim > 256 || c->head_dim % 8) return LILY_ERR_UNSUPPORTED_SHAPE;
  if (c->page_stride < 1 || c->token_stride < 1 || c->head_stride < 1) return LILY_ERR_INVALID_ARG;
  if (!head_stride_ok(c->page_stride) || !head_stride_ok(c->head_stride) ||
      !head_stride_ok(c->token_stride))
    return LILY_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v)) return LILY_ERR_MISALIGNED;
  return LILY_OK;
}

int page_shift(const lily_attn_cache& c) {
  int s = 4;
  while ((1 << s) < c.page_size) ++s;
  return s;
}

bool is16(int t) { return t == LILY_DTYPE_BF16 || t == LILY_DTYPE_F16; }
bool is_float(int t) { return is16(t) || t == LILY_DTYPE_F32; }
int bytes_of(int t) { return t == LILY_DTYPE_F32 ? 4 : t == LILY_DTYPE_E4M3 ? 1 : 2; }

// ---------------------------------------------------------------- attention
int check_attn_dims(const lily_attn_dims* d, const lily_attn_cache* c) {
  int rc;
  if (!d) return LILY_ERR_INVALID_ARG;
  if ((rc = check_cache(c))) return rc;
  if (d->n_tokens < 1 || d->n_q_heads < 1 || d->n_seqs < 1 || d->max_q_len < 1 ||
      d->prefix_len < 0 || d->max_seq_len < 0 || d->table_stride < 0)
    return LILY_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return LILY_ERR_INVALID_ARG;
  if (d->n_tokens > 65536 || d->n_seqs > 65536 || d->n_q_heads % c->n_kv_heads || d->n_q_heads / c->n_kv_heads > 64)
    return LILY_ERR_UNSUPPORTED_SHAPE;
  if (d->prefix_len > INT_MAX - 256 || d->max_seq_len > INT_MAX - 256 ||
      (int64_t)d->max_seq_len > (int64_t)d->table_stride * c->page_size)
    return LILY_ERR_UNSUPPORTED_SHAPE;
  if (!head_stride_ok(d->q_token_stride) || !head_stride_ok(d->q_head_stride) ||
      !head_stride_ok(d->out_token_stride) || !head_stride_ok(d->out_head_stride))
    return LILY_ERR_UNSUPPORTED_SHAPE;
  return LILY_OK;
}

// Rows per unit: 8, 16, 32 or 64, the least that holds `rows` (64 at most).
int unit_rows(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// The prefix goes to the tensor-core kernel (LILY_PREFIX_TENSOR) where it has more rows per KV head
// than one mma.sync row block (above, both read it once) and enough tiles of 64
// rows and keys for that kernel's launch, its load of Q and its larger partials
// to pay (128 sequences of 8 rows on one KV head, D = 128: 15.9 against 17.3 us
// at 256 tiles, 14.9 against 14.4 at 64; D = 256: 23.3 against 20.6 at 256, 24.8
// against 29.4 at 512; 4 heads of 250 rows, D = 128: 28.6 against 47.3 at 4096).
constexpr int kTcRows = 64;
constexpr int tc_tiles(int D) { return D <= 128 ? 256 : 512; }

// What a call launches, and its workspace: the status word, then the two sets'
// partials and the own set's runs.  Sized for the largest grid, so that it
// does not depend on the device.
struct Plan {
  bool tc;
  AttnSet pre, own;  // pre: not on the tensor-core kernel
  TcArgs ptc;
  int64_t pre_units, pre_total, own_most;  // units; tiles; tiles at most
  size_t pre_o, pre_lse, own_o, own_lse, rows_at, bytes;
};

void set_shape(AttnSet& s, int n_seqs, int max_q_len, int max_len, int G, int least_rows = 8) {
  s = AttnSet{};
  s.n_seqs = n_seqs;
  s.max_q_len = max_q_len;
  s.max_len = max_len;
  const int64_t rows = (int64_t)max_q_len * G;
  s.rows = unit_rows(rows);
  if (s.rows < least_rows) s.rows = least_rows;
  s.row_blocks = (int)((rows + s.rows - 1) / s.rows);
  s.min_share = 1;
}

// false where the units or tiles do not fit 31 bits.
bool make_plan(const lily_attn_dims& d, const lily_attn_cache& c, Plan& p) {
  const int G = d.n_q_heads / c.n_kv_heads;
  p = Plan{};
  size_t off = 256;
  auto partials = [&](int64_t units, int64_t tiles, int64_t max_grid, int rows, size_t& o,
                      size_t& lse) {
    const size_t n = (size_t)(units + (tiles < max_grid ? tiles : max_grid));
    o = off;
    off += up256(n * rows * c.head_dim * 4);
    lse = off;
    off += up256(n * rows * 4);
  };
  if (d.prefix_len) {
    const int64_t rows = (int64_t)d.n_tokens * G;
    p.tc = rows > kTcRows && c.n_kv_heads * ((rows + 63) / 64) * ((d.prefix_len + 63) / 64) >= tc_tiles(c.head_dim);
    if (p.tc) {
      TcArgs& t = p.ptc;
      t.paired = rows > 128 && c.head_dim <= 128;
      t.block_rows = t.paired ? 256 : 128;
      t.row_blocks = (int)((rows + t.block_rows - 1) / t.block_rows);
      t.len = d.prefix_len;
      t.tiles = (d.prefix_len + kTcKeys - 1) / kTcKeys;
      p.pre_units = (int64_t)c.n_kv_heads * t.row_blocks;
      p.pre_total = p.pre_units * t.tiles;
      partials(p.pre_units, p.pre_total, kTcMaxGrid, attn_tc_rows(c.head_dim), p.pre_o, p.pre_lse);
    } else {
      set_shape(p.pre, 1, d.n_tokens, d.prefix_len, G);
      p.pre_units = (int64_t)c.n_kv_heads * p.pre.row_blocks;
      p.pre_total = p.pre_units * ((d.prefix_len + kAttnTile - 1) / kAttnTile);
      partials(p.pre_units, p.pre_total, kAttnMaxGrid, p.pre.rows, p.pre_o, p.pre_lse);
    }
    if (p.pre_total > INT_MAX / 2) return false;
  }
  // (no sequence has more tokens than the call)
  const int max_q_len = d.max_q_len < d.n_tokens ? d.max_q_len : d.n_tokens;
  // (pairs of row counts that share a launch: the smaller is 8, or the larger, or
  // 16 beside 64)
  int least = 8;
  const int own_rows = unit_rows((int64_t)max_q_len * G);
  if (p.pre.rows == 32 && own_rows == 16) least = 32;
  if (p.pre.rows == 64 && own_rows == 32) least = 64;
  set_shape(p.own, d.n_seqs, max_q_len, d.max_seq_len, G, least);
  p.own.causal = max_q_len > 1;
  const int64_t units = (int64_t)d.n_seqs * c.n_kv_heads * p.own.row_blocks;
  if (units > INT_MAX / 2) return false;
  if (units * ((d.max_seq_len + kAttnTile - 1) / kAttnTile) > INT_MAX / 2) return false;
  p.own_most = units * ((d.max_seq_len + kAttnTile - 1) / kAttnTile);
  if (d.max_seq_len) {
    partials(units, p.own_most, kAttnMaxGrid, p.own.rows, p.own_o, p.own_lse);
    p.rows_at = off;
    off += up256((size_t)d.n_tokens * d.n_q_heads * 16);
  }
  p.bytes = off;
  return true;
}

// The cache as a 4-D tensor [page][head][token][D]; boxes of 64 dimensions
// (past D: zeros) by the tokens of a page, 64 at most.
bool cache_map(CUtensorMap* tm, void* base, const lily_attn_cache& c, uint32_t box_tokens) {
  const uint64_t dims[4] = {(uint64_t)c.head_dim, (uint64_t)c.page_size, (uint64_t)c.n_kv_heads,
                            (uint64_t)c.n_pages};
  const uint64_t strides[3] = {(uint64_t)c.token_stride * 2, (uint64_t)c.head_stride * 2,
                               (uint64_t)c.page_stride * 2};
  const uint32_t box[4] = {64, box_tokens, 1, 1};
  return encode_tiled(tm, c.dtype == LILY_DTYPE_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace lily

using namespace lily;

extern "C" {

int lily_attn_add_rmsnorm(const lily_attn_norm_dims* dims, const void* x, const void* residual,
                          const void* weight, void* residual_out, void* out, float* scales,
                          void* stream) {
  if (!dims || !x || !out) return LILY_ERR_INVALID_ARG;
  const lily_attn_norm_dims& d = *dims;
  if (d.T < 1 || d.d < 1) return LILY_ERR_INVALID_ARG;
  if (d.d > 16384 || !is_float(d.x_dtype) || !is_float(d.res_dtype) || !is_float(d.w_dtype) ||
      !(is16(d.out_dtype) || d.out_dtype == LILY_DTYPE_E4M3))
    return LILY_ERR_UNSUPPORTED_SHAPE;
  const bool e4m3 = d.out_dtype == LILY_DTYPE_E4M3;
  if (e4m3 != (scales != nullptr)) return LILY_ERR_INVALID_ARG;
  if (e4m3 ? (d.group != 0 && d.group != 64 && d.group != 128) || (d.group && d.d % d.group)
           : d.group != 0)
    return LILY_ERR_UNSUPPORTED_SHAPE;
  if (!(d.eps >= 0.f) || !std::isfinite(d.eps)) return LILY_ERR_INVALID_ARG;
  if (!stride_ok(d.x_stride, d.d) || !stride_ok(d.out_stride, d.d) ||
      (residual && !stride_ok(d.res_stride, d.d)) ||
      (residual_out && !stride_ok(d.res_out_stride, d.d)))
    return LILY_ERR_INVALID_ARG;
  const void* ptrs[] = {x, residual, weight, residual_out, out, scales};
  for (const void* p : ptrs)
    if (!aligned16(p)) return LILY_ERR_MISALIGNED;
  if (const int rc = device_rc()) return rc;

  NormArgs a = {};
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.res_out = residual_out;
  a.out = out;
  a.scales = scales;
  a.x_stride = d.x_stride;
  a.res_stride = d.res_stride;
  a.res_out_stride = d.res_out_stride;
  a.out_stride = d.out_stride;
  a.T = d.T;
  a.d = d.d;
  a.xt = d.x_dtype;
  a.rt = d.res_dtype;
  a.wt = d.w_dtype;
  a.ot = d.out_dtype;
  a.group = d.group;
  a.eps = d.eps;
  return rc_of(launch_add_rmsnorm(a, (cudaStream_t)stream));
}

int lily_attn_rope_append(const lily_attn_rope_dims* dims, const lily_attn_cache* cache,
                          const void* q, const void* k, const void* v, const int32_t* positions,
                          const int64_t* slots, const double* inv_freq, void* q_out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  if (!dims) return LILY_ERR_INVALID_ARG;
  if (const int rc = check_cache(cache)) return rc;
  const lily_attn_rope_dims& d = *dims;
  if (d.T < 1 || d.n_q_heads < 0 || d.rotary_dim < 0) return LILY_ERR_INVALID_ARG;
  if ((q != nullptr) != (d.n_q_heads > 0) || (q != nullptr) != (q_out != nullptr) ||
      (k != nullptr) != (v != nullptr) || (!q && !k) || (k && !slots) || !workspace ||
      (d.rotary_dim && (!positions || !inv_freq)))
    return LILY_ERR_INVALID_ARG;
  if (d.rotary_dim % 2 || d.rotary_dim > cache->head_dim || (d.style != 0 && d.style != 1) ||
      d.n_q_heads > 16384)
    return LILY_ERR_UNSUPPORTED_SHAPE;
  const int64_t strides[] = {d.q_token_stride, d.q_head_stride, d.k_token_stride, d.k_head_stride,
                             d.v_token_stride, d.v_head_stride, d.qo_token_stride, d.qo_head_stride};
  for (int i = 0; i < 8; ++i) {
    const bool used = i < 2 || i >= 6 ? q != nullptr : k != nullptr;
    if (used && (!head_stride_ok(strides[i]) || strides[i] > INT_MAX))
      return LILY_ERR_UNSUPPORTED_SHAPE;
  }
  const void* ptrs[] = {q, k, v, q_out, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return LILY_ERR_MISALIGNED;
  if (!aligned(positions, 4) || !aligned(slots, 8) || !aligned(inv_freq, 8))
    return LILY_ERR_MISALIGNED;
  if (workspace_bytes < 256) return LILY_ERR_WORKSPACE_TOO_SMALL;
  if (const int rc = device_rc()) return rc;

  RopeArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.kc = cache->k;
  a.vc = cache->v;
  a.pos = positions;
  a.slots = slots;
  a.inv_freq = inv_freq;
  a.q_tok = d.q_token_stride;
  a.q_head = d.q_head_stride;
  a.k_tok = (int32_t)d.k_token_stride;
  a.k_head = (int32_t)d.k_head_stride;
  a.v_tok = (int32_t)d.v_token_stride;
  a.v_head = (int32_t)d.v_head_stride;
  a.qo_tok = (int32_t)d.qo_token_stride;
  a.qo_head = (int32_t)d.qo_head_stride;
  a.c_page = cache->page_stride;
  a.c_head = cache->head_stride;
  a.c_tok = cache->token_stride;
  a.n_slots = (int64_t)cache->n_pages * cache->page_size;
  a.T = d.T;
  a.hq = d.n_q_heads;
  a.hkv = k ? cache->n_kv_heads : 0;
  a.D = cache->head_dim;
  a.rot = d.rotary_dim;
  a.style = d.style;
  a.page_shift = page_shift(*cache);
  a.dtype = cache->dtype;
  a.status = static_cast<uint32_t*>(workspace);
  return rc_of(launch_rope_append(a, (cudaStream_t)stream));
}

uint64_t lily_attn_set_wait_ns(uint64_t ns) { return g_wait_ns.exchange(ns); }

size_t lily_attn_workspace_bytes(const lily_attn_dims* dims, const lily_attn_cache* cache) {
  Plan p;
  if (check_attn_dims(dims, cache) || !make_plan(*dims, *cache, p)) return 0;
  return p.bytes;
}

int lily_attn_prefix_kernel(const lily_attn_dims* dims, const lily_attn_cache* cache) {
  Plan p;
  if (const int rc = check_attn_dims(dims, cache)) return rc;
  if (!make_plan(*dims, *cache, p)) return LILY_ERR_UNSUPPORTED_SHAPE;
  return !dims->prefix_len ? LILY_PREFIX_NONE : p.tc ? LILY_PREFIX_TENSOR : LILY_PREFIX_WARP;
}

int lily_attn_shared_prefix(const lily_attn_dims* dims, const lily_attn_cache* cache,
                            const void* q, const int32_t* prefix_pages, const int32_t* q_start,
                            const int32_t* seq_lens, const int32_t* block_table, void* out,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int rc = check_attn_dims(dims, cache)) return rc;
  const lily_attn_dims& d = *dims;
  if (!q || !out || !workspace || !seq_lens || (d.prefix_len && !prefix_pages) ||
      (d.max_seq_len && !block_table))
    return LILY_ERR_INVALID_ARG;
  if (!q_start && (int64_t)d.n_seqs * d.max_q_len != d.n_tokens) return LILY_ERR_INVALID_ARG;
  const void* ptrs[] = {q, out, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return LILY_ERR_MISALIGNED;
  const void* words[] = {prefix_pages, q_start, seq_lens, block_table, lse};
  for (const void* p : words)
    if (!aligned(p, 4)) return LILY_ERR_MISALIGNED;
  Plan p;
  if (!make_plan(d, *cache, p)) return LILY_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < p.bytes) return LILY_ERR_WORKSPACE_TOO_SMALL;
  if (const int rc = device_rc()) return rc;
  const int grid = attn_grid(cache->head_dim);
  if (grid < 1) return LILY_ERR_CUDA;

  uint8_t* base = static_cast<uint8_t*>(workspace);
  AttnArgs a = {};
  a.q = q;
  a.q_tok = d.q_token_stride;
  a.q_head = d.q_head_stride;
  a.T = d.n_tokens;
  a.hq = d.n_q_heads;
  a.hkv = cache->n_kv_heads;
  a.G = d.n_q_heads / cache->n_kv_heads;
  a.D = cache->head_dim;
  a.page_shift = page_shift(*cache);
  a.n_pages = cache->n_pages;
  a.f16 = cache->dtype == LILY_DTYPE_F16;
  a.scale_log2 = (float)((double)d.scale * 1.4426950408889634);
  a.status = static_cast<uint32_t*>(workspace);
  const uint64_t wait = g_wait_ns.load(std::memory_order_relaxed);
  a.wait_feed = (uint32_t)std::clamp<uint64_t>(wait / kTryNs, 1, UINT32_MAX);
  a.wait_use = wait ? a.wait_feed : 0;
  CUtensorMap mk, mv;
  const uint32_t page = (uint32_t)cache->page_size;
  auto maps = [&](uint32_t k_rows, uint32_t v_rows) {
    return cache_map(&mk, cache->k, *cache, page < k_rows ? page : k_rows) &&
           cache_map(&mv, cache->v, *cache, page < v_rows ? page : v_rows);
  };
  cudaStream_t s = (cudaStream_t)stream;
  MergeArgs m = {};
  m.out = out;
  m.lse = lse;
  m.out_tok = d.out_token_stride;
  m.out_head = d.out_head_stride;

  int pre_grid, own_grid;
  share_grid(grid, p.tc ? 0 : p.pre_total, p.own_most, p.pre.rows > p.own.rows, pre_grid, own_grid);
  bool first = true;
  if (d.prefix_len) {
    float* part_o = reinterpret_cast<float*>(base + p.pre_o);
    float* part_lse = reinterpret_cast<float*>(base + p.pre_lse);
    // one tensor-core CTA per SM
    const int64_t sms = grid / (cache->head_dim <= 128 ? 2 : 1);
    const int64_t most = !p.tc ? pre_grid : sms < kTcMaxGrid ? sms : kTcMaxGrid;
    const int used = (int)(p.pre_total < most ? p.pre_total : most);
    m.pre_share = (int)((p.pre_total + used - 1) / used);
    m.pre_o = part_o;
    m.pre_lse = part_lse;
    if (p.tc) {
      TcArgs& t = p.ptc;
      t.pages = prefix_pages;
      t.total = (int)p.pre_total;
      t.share = m.pre_share;
      t.grid = used;
      t.part_o = part_o;
      t.part_lse = part_lse;
      m.pre_tiles = t.tiles;
      m.pre_blocks = t.row_blocks;
      m.pre_rows = t.block_rows;
      m.pre_slot_rows = attn_tc_rows(a.D);
      m.pre_streams = !t.paired && a.D <= 128 ? 2 : 1;
      if (!maps(kTcKeys, attn_tc_v_keys(a.D))) return LILY_ERR_CUDA;
      if (launch_attn_prefix_tc(a, t, mk, mv, s) != cudaSuccess) return LILY_ERR_CUDA;
      first = false;
    } else {
      AttnSet& t = p.pre;
      t.table = prefix_pages;
      t.grid = used;
      t.part_o = part_o;
      t.part_lse = part_lse;
      m.pre_tiles = (d.prefix_len + kAttnTile - 1) / kAttnTile;
      m.pre_blocks = t.row_blocks;
      m.pre_rows = m.pre_slot_rows = t.rows;
      m.pre_streams = 1;
    }
  }
  p.own.q_start = q_start;
  p.own.lens = seq_lens;
  m.own = p.own;
  if (d.max_seq_len) {
    AttnSet& o = p.own;
    o.table = block_table;
    o.table_stride = d.table_stride;
    o.part_o = reinterpret_cast<float*>(base + p.own_o);
    o.part_lse = reinterpret_cast<float*>(base + p.own_lse);
    o.rows_at = reinterpret_cast<int4*>(base + p.rows_at);
    o.grid = own_grid;
    m.own = o;
    m.own_slots = (int)((int64_t)d.n_seqs * cache->n_kv_heads * o.row_blocks) + own_grid;
    m.own_parts = (int)((d.max_seq_len + kAttnTile - 1) / kAttnTile /
                        ((p.own_most + own_grid - 1) / own_grid));
  }
  // the sets that mma.sync takes, in one launch
  if (p.pre.grid + p.own.grid) {
    if (!maps(kAttnTile, kAttnTile)) return LILY_ERR_CUDA;
    const bool pre = p.pre.grid > 0;
    if (launch_attn_keys(a, pre ? p.pre : p.own, pre ? p.own : AttnSet{}, mk, mv, first, s) != cudaSuccess)
      return LILY_ERR_CUDA;
  }
  return rc_of(launch_attn_merge(a, m, s));
}

}  // extern "C"
