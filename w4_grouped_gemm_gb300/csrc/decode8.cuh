// decode8.cuh -- launch arguments of the attention over an 8-bit cache.
#pragma once
#include "attn.cuh"

namespace lily {

constexpr int kDecode8Rows = 8;    // query rows of a unit
constexpr int kDecode8Grid = 640;  // CTAs, at most (sizes the workspace)

struct Decode8Args {
  const void* q;
  const float *ks, *vs;
  void* out;
  float* lse;
  uint32_t* status;
  // partials: two for each CTA (of the unit that it goes on with, and of the one
  // that goes on in the next); outputs, divided by their sums, [part][D padded / 16][32 lanes],
  // references (of z) and sums
  float4* part_o;
  float2* part_ml;
  int4* split;  // two for each CTA: {CTAs of the unit that begins in it and goes on (0: none),
                // its first token, rows, row block}, {KV head}
  int64_t q_tok, q_head, out_tok, out_head, s_page, s_head, s_tok;
  int T, hq, hkv, G, D, page_shift, n_pages, f16;
  int side;            // KV heads that neighbouring CTAs take at the same time; divides hkv
  uint32_t G_inverse;  // 2^32 / G, rounded up (G above 1; rows of a sequence are below 2^22)
  float scale_log2;
  uint32_t wait_feed, wait_use;  // tries of a wait before it gives up: of the warp that brings tiles, and of the others
};
int decode8_side(int hkv);
int decode8_tile(int D);                 // keys of a tile
// units, tiles: those of the longest lengths, the most that the list can have
void decode8_box(int D, int page, uint32_t& bytes, uint32_t& tokens);
// mk, mv: the codes as [page][head][token][D] in boxes of decode8_box
cudaError_t launch_decode8(const Decode8Args& a, const AttnSet& s, const CUtensorMap& mk, const CUtensorMap& mv,
                           int64_t units, int64_t tiles, int sms, cudaStream_t st);

}  // namespace lily
