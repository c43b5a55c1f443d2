// Device code shared by attn_prompt's tensor-core kernels.
#pragma once

#include <cfloat>

#include "prompt_items.cuh"
#include "rows_tc.cuh"

namespace oscar {

__device__ __forceinline__ uint32_t bf162_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
constexpr float kTop = 8.f;     // log2 of the largest P
constexpr float kAbove = 12.f;  // a new reference lies this far above its row's maximum

// What a row's weights refer to: P = 2^(s scale - M) of a score s.  M's rounding is common to the row and does not count while P
// stays within float32's range: up to |M| = 2^30 it is 2^5 at most.  Beyond, scores that are not the maximum have no weight,
// since their neighbours in float32 are 2^6 apart; scale then is the power of two that makes M, the maximum times it,
// 2^31 .. 2^32 without a rounding, and other scores at least 2^7 less.  Before the first score above -inf every
// exponent is -inf.
struct Reference {
  float scale = 0x1p-8f, M = -FLT_MAX;
  __device__ __forceinline__ float follow(float top, float qscale) {  // to the maximum `top`: the factor for what the row has
    const float next = fmaf(top, qscale, kAbove), f = scale == qscale ? exp2f(M - next) : 0.f;
    scale = qscale, M = next;
    if (!(fabsf(next) <= 0x1p30f)) {
      scale = pow2i(max(-126, min(127, 31 + 127 - (__float_as_int(fabsf(top)) >> 23))));
      M = top * scale;
    }
    return f;
  }
  __device__ __forceinline__ float lse(float l, float qscale) const {
    return ((scale == qscale ? M : M * (qscale / scale)) + log2f(l)) * 0.6931471805599453f;
  }
};

// A row's P as the products see it: l, its sum, and r, the sum of the rounded values, which is what the output is divided by.
// A rounding that all of a row's weight has in common then leaves the output as it is: with l there, too, one dominant weight's
// own 2^-9 went straight into the row (activations with outliers: 2.08e-3 of the output's norm instead of 1.59e-3, of which its
// rounding to bf16 is 1.5e-3).  lse has l.  Cost: two adds per pair of weights, 1265 -> 1286 us for 16,384 tokens; with the
// values unpacked by logic instructions and added in pairs 1313.
struct RowSums {
  uint64_t l = 0, r = 0;
  __device__ __forceinline__ void scale(float f) { l = mul2(l, splat_x2(f)), r = mul2(r, splat_x2(f)); }
  __device__ __forceinline__ float2 total() const {
    float a, b, c, d;
    unpack2(l, a, b), unpack2(r, c, d);
    return make_float2(a + b, c + d);
  }
};
// What a tile adds to them, in two chains.
struct TileSums {
  uint64_t l[2] = {0, 0};
  float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f};
  __device__ __forceinline__ void add(int chain, float y, float z, uint32_t rounded) {
    l[chain] = add2(l[chain], pack2(y, z));
    asm("{\n .reg .b16 x, y;\n mov.b32 {x, y}, %2;\n add.rn.f32.bf16 %0, x, %0;\n add.rn.f32.bf16 %1, y, %1;\n}\n"
        : "+f"(lo[chain]), "+f"(hi[chain])
        : "r"(rounded));
  }
  __device__ __forceinline__ void into(RowSums& s) const {
    s.l = add2(s.l, add2(l[0], l[1]));
    s.r = add2(s.r, add2(pack2(lo[0], hi[0]), pack2(lo[1], hi[1])));
  }
};
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Sixteen bf16 values of a row, 32 bytes: one store where the address allows it.  The threads of a warp have rows of their own,
// so a store costs by the rows that it touches, not by its bytes.
__device__ __forceinline__ void store16(__nv_bfloat16* to, const float (&x)[16], bool aligned32) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = bf162_of(x[2 * i], x[2 * i + 1]);
  if (aligned32) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]),
                 "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(q[0], q[1], q[2], q[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(q[4], q[5], q[6], q[7]);
  }
}

// `rows` V rows of 128 channels (two blocks of 64, swizzled) that some query rows of the block do not see: zero for what is
// infinite or not a number.  odd [3][channels]: the first token of the sequence with a NaN, +inf, -inf in a channel.  By 64
// threads, x of them.
template <int rows, int channels>
__device__ __forceinline__ void check_values(uint8_t* tile, int* odd, int token0, int seen_by_all, int len, int x) {
  constexpr int kBlock = rows * 128;
#pragma unroll 1
  for (int r = x; r < rows; r += 64) {
    const int token = token0 + r;
    if (token <= seen_by_all) continue;
    uint32_t most = 0;
#pragma unroll
    for (int block = 0; block < 2; ++block)
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // the 16-byte pieces of a row in an order of its own: no bank twice
        const uint4 v = *reinterpret_cast<const uint4*>(tile + block * kBlock + r * 128 + ((i + r) & 7) * 16);
        most = absmax2(absmax2(absmax2(absmax2(most, v.x), v.y), v.z), v.w);
      }
    if ((most & 0xFFFFu) < 0x7F80u && (most >> 16) < 0x7F80u) continue;
#pragma unroll 1
    for (int c = 0; c < 128; ++c) {
      uint16_t* at = reinterpret_cast<uint16_t*>(tile + (c / 64) * kBlock + r * 128 + (((c & 63) / 8) ^ (r & 7)) * 16 + (c & 7) * 2);
      const uint32_t v = *at;
      if ((v & 0x7FFFu) < 0x7F80u) continue;
      *at = 0;
      if (token < len) atomicMin(odd + ((v & 0x7FFFu) > 0x7F80u ? 0 : v < 0x8000u ? 1 : 2) * channels + c, token);
    }
  }
}

}  // namespace oscar
