// attn_share.h -- how attention's two sets of tiles share the GPU's places (host
// arithmetic alone).
#pragma once
#include <cstdint>

namespace lily {

inline int64_t ceil_div(int64_t n, int64_t by) { return (n + by - 1) / by; }

// CTAs for the prefix's A tiles and the own pages' tiles, B at most, in one launch
// on a GPU that holds `cap`.  Either both sets take all it holds, one after the
// other, or they share it so that both take about as long; a prefix tile of more
// rows than an own one (wide) counts twice, and a CTA costs about three tiles
// besides its own.  (4 sequences of 257 own keys behind 131072, D = 256: 64.2 us one
// after the other, 58.1 with 5 CTAs beside the prefix's 147.)
//
// B comes from the caller's bound on the lengths, which in a captured graph is the
// room that sequences have and not what they use.  So a division is taken only
// where it is no slower than one after the other whether the own pages are empty
// (the prefix's CTAs may lose three tiles' time and a sixteenth of theirs) or as
// long as the bound (the own pages keep CTAs enough), and gains where they are half
// of it.  (16 sequences of up to 400 own keys behind 1003: 14.2 us with room for
// 400, 16.6 one after the other, as with room for 4096; a division by half of B
// alone took 18.6 there and 55 with room for 32768.  What that one gained with tight
// bounds and long own pages is lost: 96 sequences of up to 2500 behind 300, 102 ->
// 109 us, and 153 us with room for 8192.)
inline void share_grid(int cap, int64_t A, int64_t B, bool wide, int& ga, int& gb) {
  ga = (int)(A < cap ? A : cap);
  gb = (int)(B < cap ? B : cap);
  if (ga + gb <= cap || ga == 0 || gb == 0) return;
  const int64_t half = ceil_div(B, 2), w = wide ? 2 : 1, first = w * ceil_div(A, ga);
  const int64_t most = first + (first / 16 < 3 ? first / 16 : 3);
  for (int64_t both = first; both <= most; ++both) {  // the time that each set takes
    const int64_t a = ceil_div(A, both / w);  // the least that take as long
    if (a >= cap) continue;
    const int64_t b = B < cap - a ? B : cap - a;
    const int64_t mid = ceil_div(half, b) > both ? ceil_div(half, b) : both;
    if (mid + 3 <= first + ceil_div(half, gb) + 6 && ceil_div(B, b) + 3 <= first + ceil_div(B, gb) + 6) {
      ga = (int)a;
      gb = (int)b;
      return;
    }
  }
}

}  // namespace lily
