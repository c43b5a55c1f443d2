// Which tile of which sequence a block of attn_prompt takes.
#pragma once

#include "internal.h"

namespace oscar {

struct PromptItem {
  int b, tile;     // sequence (-1: none) and its tile
  int start, len;  // the sequence's first packed row and length
};

// A sequence of len tokens has ceil(len * num / den) tiles; most that n packed
// tokens of B sequences can give.
__host__ __device__ inline int64_t prompt_items(const PromptArgs& a, int num, int den) { return int64_t(a.n) * num / den + a.B; }

__device__ __forceinline__ int2 prompt_span(const PromptArgs& a, int b) {
  const int lo = min(max(a.cu[b], 0), a.n), hi = min(max(a.cu[b + 1], lo), a.n);
  return make_int2(lo, hi - lo);
}

// One warp.
__device__ __forceinline__ void prompt_check(const PromptArgs& a) { packed_check(a.cu, a.B, a.n, a.status); }

// Item i of the tiles of all sequences, later tiles first: with a causal mask a
// tile's work grows with its index, and blocks start in the order of i, so the
// longest run first and the short ones fill the end.  Called by a whole warp.
// Sequences with more than L tiles have one of index L: item i has the index L
// with C(L + 1) <= i < C(L), C(L) = sum over the sequences of max(0, tiles - L).
// `at`: the index of an earlier item of the caller's, whose items come in
// increasing order (-1: none); it is searched from there.
__device__ __forceinline__ PromptItem prompt_item(const PromptArgs& a, int i, int num, int den, int& at) {
  const int lane = threadIdx.x & 31;
  // 32 bits hold them: n * num < 2^31, and that many tiles and one more for each sequence
  auto tiles = [&](int b) { return int((uint32_t(prompt_span(a, b).y) * uint32_t(num) + uint32_t(den) - 1) / uint32_t(den)); };
  auto above = [&](int level) {
    uint32_t c = 0;
#pragma unroll 4
    for (int b = lane; b < a.B; b += 32) c += uint32_t(max(0, tiles(b) - level));
    return int64_t(__reduce_add_sync(0xffffffffu, c));
  };
  PromptItem it{-1, 0, 0, 0};
  // C(lo) > i >= C(hi)
  int hi = at < 0 ? int(int64_t(a.n) * num / den) + 1 : at + 1, lo = at < 0 ? 0 : at;
  for (int step = 1; above(lo) <= i; step *= 2) {
    if (lo == 0) return it;
    hi = lo;
    lo = max(0, lo - step);
  }
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (above(mid) > i) lo = mid;
    else hi = mid;
  }
  at = lo;
  int64_t rank = i - above(lo + 1);  // among the sequences with more than lo tiles
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const bool has = b0 + lane < a.B && tiles(b0 + lane) > lo;
    const unsigned mask = __ballot_sync(0xffffffffu, has);
    const int count = __popc(mask);
    if (rank < count) {
      it.b = b0 + __fns(mask, 0, int(rank) + 1);
      it.tile = lo;
      const int2 s = prompt_span(a, it.b);
      it.start = s.x, it.len = s.y;
      return it;
    }
    rank -= count;
  }
  return it;
}

}  // namespace oscar
