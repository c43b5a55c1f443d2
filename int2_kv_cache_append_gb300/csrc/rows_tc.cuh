// Device code shared by the tensor-core row attention kernels: tcgen05 and
// packed-arithmetic wrappers, and the warps that expand cached K and V rows into
// fp16 operands.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rows.cuh"

namespace oscar {

constexpr int kTok = 128;    // positions per tile
constexpr int kUnit = 16384; // bytes of a K unit (64 channels of 128 tokens) or V unit (64 tokens of 128 channels)

// Shared-memory descriptors: their low word is the address and the leading byte
// offset, the high word constant.  128-byte swizzle: K-major, 8-row groups 1024
// bytes apart (the leading offset is not used); MN-major: 64-element blocks
// `lead` bytes apart, groups of eight k 1024 bytes apart.
constexpr uint32_t kDescSwizzled = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_of(uint32_t saddr, uint32_t lead) { return ((saddr >> 4) & 0x3FFF) | ((lead >> 4) << 16); }
// kind::f16, fp16 operands, float32 accumulator, M = 128.
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) |
         (uint32_t(128 >> 4) << 24);
}
// Issued by the lane with `leader` set; the whole warp comes along, so that
// descriptors are computed in uniform registers (in one lane's branch every
// product costs an extra eight instructions, more than its own 64 cycles).
template <uint32_t hi = kDescSwizzled>
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 x, y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " mov.b64 x, {%1, %6};\n mov.b64 y, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(leader), "n"(hi)
      : "memory");
}
// A from TMEM (fp16 pairs along k in a lane's columns)
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b64 y;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n mov.b64 y, {%2, %6};\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(leader), "n"(kDescSwizzled)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar, uint32_t leader) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 consecutive columns of the thread's TMEM lane, and their store.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(a)
      : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// true in every thread of the named barrier's 256 (128) if it is in one of them
__device__ __forceinline__ bool any256(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 256, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(p))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool any128(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(p))
      : "memory");
  return r != 0;
}
// Bounded wait of a whole warp.  All lanes poll, four instructions a turn: the
// waiting warps share the issue slots with the ones that work.  The hardware
// suspends a turn for a microsecond at most, so `turns` of them take at most
// about as many microseconds.  (Reading the clock in this loop instead made the attentions 3 to 8 % slower.)
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity, uint32_t turns) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 n;\n mov.b32 n, 0;\n"
      "again_%=:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n @p bra done_%=;\n"
      " add.u32 n, n, 1;\n setp.lt.u32 q, n, %3;\n @q bra again_%=;\n"
      "done_%=:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(turns)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t turns) {
  return __all_sync(0xffffffffu, poll(bar, parity, turns));
}
// The waits of a warp that goes on after one that ran out: those behind it only look.
struct Waits {
  uint32_t turns;
  bool ok = true;
  __device__ __forceinline__ void on(uint32_t bar, uint32_t parity) {
    if (!poll(bar, parity, turns)) ok = false, turns = 0;
  }
};
// Position in a ring of n buffers: index and phase, advanced without division.
template <int n>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == n) at = 0, phase ^= 1;
  }
};
// Arrival of the threads with `p`, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool p) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar),
               "r"(uint32_t(p))
               : "memory");
}
// 2^x, results below the normal range are 0
__device__ __forceinline__ float ex2z(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// v[j] of lane l, summed over the lanes, for column j = l (n = 32) or l % 16 (n = 16).
template <int n>
__device__ __forceinline__ float sum_columns(float (&v)[n], int lane) {
#pragma unroll
  for (int m = n / 2; m; m >>= 1)
#pragma unroll
    for (int j = 0; j < m; ++j) {
      const bool up = (lane & m) != 0;
      const float give = up ? v[j] : v[j + m];
      v[j] = (up ? v[j + m] : v[j]) + __shfl_xor_sync(0xffffffffu, give, m);
    }
  if (n == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  return v[0];
}
__device__ __forceinline__ uint32_t absmax2(uint32_t m, uint32_t x) {
  // bf16 pairs: magnitudes compare as integers (a NaN is above infinity)
  return __vmaxu2(m, x & 0x7FFF7FFFu);
}
// smallest e in [-60, 126] with x < 2^e (x >= 0 finite; 126 is not enough for x >= 2^126, whose 2^-126 x < 4 still
// fits; below 2^-60 a row keeps an absolute precision of 2^-85)
__device__ __forceinline__ int exponent_above(float x) {
  return min(126, max(-60, (int(__float_as_uint(x)) >> 23) - 126));
}
// Codes of a word at bits 2 p and 16 + 2 p as fp16 pairs, two p per shift: for
// w = code_shift(word, q), p = 2 q + 1 lies at bits 8 and 24 (1 + c / 4) and
// p = 2 q at bits 6 and 22 (1 + c / 16).
__device__ __forceinline__ uint32_t code_shift(uint32_t word, int q) {
  const int sh = 6 - 4 * q;
  return sh >= 0 ? word << sh : word >> -sh;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t code_odd(uint32_t w) { return and_or(w, 0x03000300u, 0x3C003C00u); }
__device__ __forceinline__ uint32_t code_even(uint32_t w) { return and_or(w, 0x00C000C0u, 0x3C003C00u); }
// c - 1 of a code
__device__ __forceinline__ uint32_t less_one_odd(uint32_t w) { return hfma2(code_odd(w), 0x44004400u /* 4 */, 0xC500C500u /* -5 */); }
__device__ __forceinline__ uint32_t less_one_even(uint32_t w) { return hfma2(code_even(w), 0x4C004C00u /* 16 */, 0xCC40CC40u /* -17 */); }
// Lloyd-Max values: 150 times the level's distance from the middle (rho + 1/2 levels),
// from c - 1: with x = 2 c - 3 = 2 (c - 1) - 1, 150 (level - middle) = x (74 + x^2)
// (75 = 1 * 75, 249 = 3 * 83), every step exact in fp16.
__device__ __forceinline__ uint32_t lm_value(uint32_t c1) {
  const uint32_t x = hfma2(c1, 0x40004000u /* 2 */, 0xBC00BC00u /* -1 */);
  return hmul2(x, hfma2(x, x, 0x54A054A0u /* 74 */));
}
constexpr float kLmMiddle = kLmRho + 0.5f;
// c - [c > 1] - 1 = -1, 0, 0, 1 from c - 1 = -1, 0, 1, 2 = k: k - (k > 0), the step taken from k by clamping to [0, 1].
__device__ __forceinline__ uint32_t lm_extra(uint32_t c1) {
  uint32_t step;
  asm("max.f16x2 %0, %1, %2;" : "=r"(step) : "r"(c1), "r"(0u));
  asm("min.f16x2 %0, %0, %1;" : "+r"(step) : "r"(0x3C003C00u));
  return hfma2(step, 0xBC00BC00u, c1);
}
// t = -1, 0, 0, 1 times: a where t is -1, b where it is 1
__device__ __forceinline__ uint32_t by_sign(uint32_t t, uint32_t minus_a, uint32_t b) {
  uint32_t up, down;
  asm("max.f16x2 %0, %1, %2;" : "=r"(up) : "r"(t), "r"(0u));
  asm("min.f16x2 %0, %1, %2;" : "=r"(down) : "r"(t), "r"(0u));
  return hfma2(up, b, hmul2(down, minus_a));
}
// unit * value of an fp16 pair in float32: its fp16 rounding (part 0) or what that leaves (part 1)
__device__ __forceinline__ uint32_t lm_part(uint32_t value, float unit, int part) {
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&value));
  const float a = x.x * unit, b = x.y * unit;
  const uint32_t hi = half2_of(a, b);
  if (!part) return hi;
  const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return half2_of(a - h.x, b - h.y);
}
// a bf16 pair times `scale`, as fp16
__device__ __forceinline__ uint32_t scaled_half2(uint32_t x, float scale) {
  return half2_of(__uint_as_float(x << 16) * scale, __uint_as_float(x & 0xFFFF0000u) * scale);
}


__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// (x, y) as the sum of two fp16 pairs; returns the sum of what they stand for
__device__ __forceinline__ float split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = half2_of(x, y);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&hi));
  lo = half2_of(x - a.x, y - a.y);
  const float2 b = __half22float2(*reinterpret_cast<__half2*>(&lo));
  return (a.x + b.x) + (a.y + b.y);
}

// Scale of a query row: a power of two that brings its largest finite component
// just below 2^7 (sums of 128 of them stay in fp16).  Every row has its own, so
// that no row's bits depend on the others of its CTA.
__device__ __forceinline__ int query_exponent(uint32_t max_bits) { return max(-119, (int(max_bits) >> 23) - 126 - 7); }

// Byte offset of element (row, k) of an operand of 16 k without swizzle: core
// matrices of 8 rows x 16 bytes, the two of a row group 128 bytes apart.
__device__ __forceinline__ uint32_t rank_offset(int row, int k) {
  return uint32_t(row >> 3) * 256 + uint32_t(k >> 3) * 128 + uint32_t(row & 7) * 16 + uint32_t(k & 7) * 2;
}
constexpr uint32_t kDescRank = (256 >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t rank_desc(uint32_t saddr) { return desc_of(saddr, 128); }
// (hi, hi, lo, lo) of a row's sum and (hi, lo, hi, lo) of a key row's middle: their products' sum is sum * middle
__device__ __forceinline__ uint2 rank_query(float x) {
  const uint32_t h = half2_of(x, x);
  const float r = x - __half2float(__ushort_as_half(uint16_t(h & 0xFFFF)));
  return make_uint2(h, half2_of(r, r));
}
__device__ __forceinline__ uint2 rank_key(float x) {
  const float h = __half2float(__float2half_rn(x));
  const uint32_t hl = half2_of(h, x - h);
  return make_uint2(hl, hl);
}

// The CTA's query rows as fp16 operands in shared memory, by `warps` warps
// (named barrier 3), a row at a time each: scaled (query_exponent), split into two
// fp16 values whose sum has 22 bits, written K-major in blocks of 64 channels.
// rank: the rows' sums per group for the rank-one term.  factor: the powers of
// two that undo the scaling.
template <int DG, int N, int warps>
__device__ __forceinline__ void load_queries(const RowsArgs& a, uint8_t* sq, int part, const int* outr, uint8_t* rank,
                                             float* factor, int warp, int lane) {
  constexpr int D = DG * 128;
#pragma unroll 2
  for (int c = warp; c < N; c += warps) {
    const int r = outr[c];
    float4 v[DG];
    uint32_t mx = 0;
#pragma unroll
    for (int gr = 0; gr < DG; ++gr) {
      v[gr] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r >= 0) v[gr] = *reinterpret_cast<const float4*>(a.qrot + int64_t(r) * D + gr * 128 + 4 * lane);
    }
#pragma unroll
    for (int gr = 0; gr < DG; ++gr) {
      const float f[4] = {v[gr].x, v[gr].y, v[gr].z, v[gr].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (isfinite(f[e])) mx = max(mx, __float_as_uint(fabsf(f[e])));
    }
    const int fe = query_exponent(__reduce_max_sync(0xffffffffu, mx));
    const float inv = pow2i(-fe);
    uint2 sums[4] = {make_uint2(0, 0), make_uint2(0, 0), make_uint2(0, 0), make_uint2(0, 0)};
#pragma unroll
    for (int gr = 0; gr < DG; ++gr) {
      uint32_t hi[2], lo[2];
      float sum = split_pair(v[gr].x * inv, v[gr].y * inv, hi[0], lo[0]);
      sum += split_pair(v[gr].z * inv, v[gr].w * inv, hi[1], lo[1]);
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      sums[gr] = rank_query(sum);
      // channels 4 lane .. 4 lane + 3: block lane / 16, 16-byte chunk (lane / 2) % 8, half lane % 2
      const int off = (2 * gr + (lane >> 4)) * (N * 128) + c * 128 + ((((lane >> 1) & 7) ^ (c & 7)) << 4) + ((lane & 1) << 3);
      *reinterpret_cast<uint2*>(sq + off) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(sq + part + off) = make_uint2(lo[0], lo[1]);
    }
    if (lane == 0) {
      factor[c] = pow2i(fe);
      *reinterpret_cast<uint4*>(rank + rank_offset(c, 0)) = make_uint4(sums[0].x, sums[0].y, sums[1].x, sums[1].y);
      *reinterpret_cast<uint4*>(rank + rank_offset(c, 8)) = make_uint4(sums[2].x, sums[2].y, sums[3].x, sums[3].y);
    }
  }
  fence_async();
  asm volatile("bar.sync 3, %0;" ::"n"(warps * 32) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
template <int DG>
__device__ __forceinline__ void prefetch_row(const __nv_bfloat16* row) {
#pragma unroll
  for (int e = 0; e < 128 * DG; e += 64) prefetch_l2(row + e);
}
// bits of a BF16 row's largest |value|, kU 16-byte loads on their way at once
template <int DG, int kU>
__device__ __forceinline__ uint32_t row_max(const __nv_bfloat16* row) {
  uint32_t w = 0;
  const uint4* src = reinterpret_cast<const uint4*>(row);
#pragma unroll kU
  for (int j = 0; j < DG * 16; ++j) {
    const uint4 v = src[j];
    w = absmax2(absmax2(absmax2(absmax2(w, v.x), v.y), v.z), v.w);
  }
  return max(w & 0xFFFFu, w >> 16) << 16;
}
// 64 BF16 channels (zeros where src is null), scaled, into row r of a unit
template <int kU>
__device__ __forceinline__ void write_wide(const __nv_bfloat16* src, uint8_t* dst, int r, float scale) {
  static_assert(8 % kU == 0);
#pragma unroll 1
  for (int p0 = 0; p0 < 8; p0 += kU) {
    uint4 v[kU];
#pragma unroll
    for (int p = 0; p < kU; ++p) v[p] = src ? reinterpret_cast<const uint4*>(src)[p0 + p] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int p = 0; p < kU; ++p)
      *reinterpret_cast<uint4*>(dst + (((p0 + p) ^ (r & 7)) << 4)) =
          make_uint4(scaled_half2(v[p].x, scale), scaled_half2(v[p].y, scale), scaled_half2(v[p].z, scale), scaled_half2(v[p].w, scale));
  }
}

// Constants of a tile, one slot of the ring: e[128] (the value rows' exponents),
// k[128] (the factors that undo the keys' scaling), two words that are set when
// some e is not 0 and when some k is not kKeyEven, and, for rows in the TMEM lanes
// (RV), rv[128] (2^-e).
constexpr float kKeyEven = 2.0f;
template <bool RV>
struct TileConsts {
  static constexpr int kBytes = (RV ? 3 : 2) * kTok * 4 + 16;
  float* p;
  __device__ __forceinline__ TileConsts(uint8_t* ring, int slot) : p(reinterpret_cast<float*>(ring + slot * kBytes)) {}
  __device__ __forceinline__ float* e() const { return p; }
  __device__ __forceinline__ float* k() const { return p + kTok; }
  __device__ __forceinline__ uint32_t* uneven() const { return reinterpret_cast<uint32_t*>(p + 2 * kTok); }
  __device__ __forceinline__ uint32_t* k_uneven() const { return uneven() + 1; }
  __device__ __forceinline__ float* rv() const { return p + 2 * kTok + 4; }
};
// 2^-e of a value row's exponent, 1 for the rows that have none
__device__ __forceinline__ float rv_of(float e) { return isfinite(e) ? pow2i(-int(e)) : 1.f; }

template <bool b>
struct Flag {
  static constexpr bool value = b;
};

// What the expanding warps work on: positions [p0, p1) of unit u.
struct Share {
  const RowsArgs* a;
  int u, T, p0, p1, nt;
  uint8_t* sm;                    // shared memory and its address
  uint32_t base;
  uint32_t k_full, k_empty, v_full, v_empty, c_full, c_empty;  // first barrier of each kind
  int oK, oV, oRawK, oRawV, oConst, oRank;
};
constexpr int kRawStage = kTok * 36;  // staged codes (32 bytes) and scale / zero pairs of one (tile, group) and role
constexpr int kRank = kTok * 32;      // one tile's rank-one operand

// First tile of share s of ns.  Tiles with BF16 rows take about kWideCost times an INT2 tile's time, and the shares are of
// equal time: 32 tokens over 16,384 positions at D = 512 with windows of 512 + 2048 take 608 / 528 / 448 / 423 us with
// costs of 1 / 2 / 3 / 4, 5 drafted tokens at D = 128 191 / 157 / 154 / 146 us, a chunk of 2048 the same with all of them.
constexpr int kWideCost = 4;
__device__ __forceinline__ int share_start(const Geom& g, int T, int blocks, int s, int ns) {
  const int w = g.vb ? 1 : kWideCost;
  const int lo = min(blocks, (g.S + kTok - 1) / kTok), hi = min(blocks, max(lo, (T - g.W) / kTok));  // INT2 tiles: lo .. hi - 1
  int64_t x = (int64_t(lo + blocks - hi) * w + (hi - lo)) * s / ns;
  if (x < int64_t(lo) * w) return int(x) / w;
  x -= int64_t(lo) * w;
  return x < hi - lo ? lo + int(x) : hi + int(x - (hi - lo)) / w;
}

// The tiles from position p0 on that lie within [from, to).
struct Tiles {
  int first;
  uint32_t count;
  __device__ Tiles(int p0, int from, int to) {
    first = from > p0 ? (from - p0 - 1) / kTok + 1 : 0;
    count = uint32_t(max(0, (to - p0) / kTok - first));
  }
  __device__ bool has(int i) const { return uint32_t(i - first) < count; }
};

// K, four warps, a thread per token.  An INT2 key is z + s c = (z + s) + s (c - 1),
// and s (c - 1) is -s, 0, s or 2 s: exact in fp16.  The middles z + s enter as a
// rank-one term of 16 more k (rank_key), so the products' sums are the scores.
// Lloyd-Max levels are the uniform ones plus 0.16 (0, 1, 1, 2): z + rho s is the
// middle, and s (-rho, 0, 1, rho + 1) is rounded to fp16 with the residues in a
// second set of units, which only Q's high part meets (up to 2^-22 of a product is lost).
// BF16 keys are exact in fp16 within its range.  Every key row is scaled by a
// power of two of its own, one half (which keeps 2 s and z + s within fp16) where
// its largest value lies between 2^-2 and 2^14, else what brings that just below
// 2^13: what is cut off, 2^-25 of a scaled row, is then 2^-22 of the row's largest
// value at most.  The factor that undoes it meets the row's scores; one factor
// for a tile would let a key of a later position cost the earlier ones' bits.
//
// Steps k = (tile, group); codes are staged kStages - 1 steps ahead by cp.async,
// each thread its own row.  Returns false after a timeout.
template <int DG, int KU, int CB, int kStages, int kU, bool LM, bool RV>
__device__ __forceinline__ bool expand_k(const Share& x, int tok, int lane) {
  // the rank-one operand of tile i + 2 is written after unit 0 of that tile has found the unit KU before it empty, and
  // tile i's is used with the first unit of its last group
  static_assert(2 * (DG + 1) >= KU, "two rank-one operands");
  const Geom& g = x.a->g;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_warp(bar, parity, x.a->wait_turns); };
  const int steps = x.nt * DG, per = LM ? 4 : 2;  // units of a step
  const uint8_t* role = x.a->layer_base + g.sink_bytes + g.ring_bytes;
  const int64_t row0 = int64_t(x.u) * g.ncap + (x.p0 + tok - g.S);  // INT2 row of the first tile's token
  const uint8_t* codes = role + row0 * (32 * DG);
  const uint8_t* szs = role + g.codes_bytes + row0 * (4 * DG);
  const int ring0 = max(g.S, x.T - g.W);  // INT2: S <= position < ring0
  const uint32_t raw = x.base + x.oRawK + tok * 32, rsz = x.base + x.oRawK + kTok * 32 + tok * 4;
  auto stage = [&](int k) {
    const int i = k / DG, gr = k % DG, pos = x.p0 + i * kTok + tok, st = (k % kStages) * kRawStage;
    if (k < steps && pos >= g.S && pos < ring0 && pos < x.p1) {
      const uint8_t* c = codes + int64_t(i) * (kTok * 32 * DG) + gr * 32;
      cp_async16(raw + st, c);
      cp_async16(raw + st + 16, c + 16);
      cp_async4(rsz + st, szs + int64_t(i) * (kTok * 4 * DG) + gr * 4);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int k = 0; k < kStages - 1; ++k) stage(k);
  for (int j = 0; j < 4; ++j)  // columns beyond 4 DG stay zero
    *reinterpret_cast<uint4*>(x.sm + x.oRank + (j >> 1) * kRank + rank_offset(tok, 8 * (j & 1))) = make_uint4(0, 0, 0, 0);
  auto ahead = [&](int i) {  // a BF16 row of tile i on its way to the L2 cache
    const int pos = x.p0 + i * kTok + tok;
    if (pos < x.p1 && (pos < g.S || pos >= ring0)) prefetch_row<DG>(row_ref(g, x.a->layer_base, 0, x.u, x.T, pos).wide);
  };
  ahead(0);
  const Tiles packed_tiles(x.p0, g.S, ring0);
  uint32_t nsz[DG];  // the next tile's scale / zero pairs
  auto pairs = [&](int i) {
    const int pos = x.p0 + i * kTok + tok;
    const bool packed = pos >= g.S && pos < ring0 && pos < x.p1;
#pragma unroll
    for (int gr = 0; gr < DG; ++gr)
      nsz[gr] = packed ? __ldg(reinterpret_cast<const uint32_t*>(szs + int64_t(i) * (kTok * 4 * DG)) + gr) : 0u;
  };
  pairs(0);
  float down = 0.5f;  // the row's power of two
  int n = 0;          // units written
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    stage(k + kStages - 1);
    cp_async_wait<kStages - 1>();
    const int i = k / DG, gr = k % DG, slot = i % CB, pos = x.p0 + i * kTok + tok;
    const bool valid = pos < x.p1, packed = valid && pos >= g.S && pos < ring0;
    const __nv_bfloat16* wide = valid && !packed ? row_ref(g, x.a->layer_base, 0, x.u, x.T, pos).wide : nullptr;
    if (gr == 0) {
      if (!packed_tiles.has(i + 1)) ahead(i + 1);
      float m = 0.f;
      if (packed) {
#pragma unroll
        for (int j = 0; j < DG; ++j) {
          const float2 sz = __half22float2(*reinterpret_cast<const __half2*>(&nsz[j]));
          m = fmaxf(m, fmaxf(fabsf(sz.y), fabsf(fmaf(sz.x, LM ? kLmSpan : 3.0f, sz.y))));
        }
      } else if (wide) {
        m = __uint_as_float(row_max<DG, 2 * kU>(wide));
      }
      pairs(i + 1);
      int e = 1;
      if (m > 0.f && !(m >= 0x1p-2f && m < 0x1p14f) && isfinite(m))
        e = max(-104, min(127, (int(__float_as_uint(m)) >> 23) - 126)) - 13;  // 2^-e m is just below 2^13
      down = pow2i(-e);
      if (i >= CB && !wait(x.c_empty + 8 * slot, ((i / CB) & 1) ^ 1)) return false;
      const TileConsts<RV> tc(x.sm + x.oConst, slot);
      tc.k()[tok] = pow2i(e);
      const bool uneven = __any_sync(0xffffffffu, e != 1);
      if (lane == 0) reinterpret_cast<volatile uint8_t*>(tc.k_uneven())[tok >> 5] = uneven;  // one byte per warp
      __syncwarp();
      mbar_arrive_if(x.c_full + 8 * slot, lane == 0);
    }
    const uint8_t* st = x.sm + x.oRawK + (k % kStages) * kRawStage;
    const uint4 c0 = *reinterpret_cast<const uint4*>(st + tok * 32), c1 = *reinterpret_cast<const uint4*>(st + tok * 32 + 16);
    float2 sz = make_float2(0.f, 0.f);
    if (packed) sz = __half22float2(*reinterpret_cast<const __half2*>(st + kTok * 32 + tok * 4));
    const uint32_t s1 = half2_of(sz.x * down, sz.x * down);
    // Lloyd-Max: -rho s, 0, s, (1 + rho) s as the uniform part plus d1 (-1, 0, 0, 1), rounded, and what that leaves
    uint32_t d1 = 0, left0 = 0, left3 = 0;
    if (LM) {
      const float x1 = sz.x * down;
      const __half d = __float2half_rn((kLmRho - 1.0f) * x1), h = __float2half_rn(x1);
      const float l0 = -kLmRho * x1 + __half2float(__hfma(d, __float2half_rn(1.0f), h));
      const float l3 = (kLmRho + 1.0f) * x1 - __half2float(__hfma(h, __float2half_rn(2.0f), d));
      d1 = half2_of(__half2float(d), __half2float(d));
      left0 = half2_of(-l0, -l0);
      left3 = half2_of(l3, l3);
    }
    const float middle = fmaf(LM ? kLmRho : 1.0f, sz.x, sz.y) * down;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      // word 2 c + half: pair c of every 16-byte chunk
      const uint32_t w[4] = {half ? c0.y : c0.x, half ? c0.w : c0.z, half ? c1.y : c1.x, half ? c1.w : c1.z};
#pragma unroll 1
      for (int set = 0; set < per; set += 2, ++n) {
        const int u = n % KU;
        if (n >= KU && !wait(x.k_empty + 8 * u, ((n / KU) & 1) ^ 1)) return false;
        if (half == 0 && set == 0)
          *reinterpret_cast<uint2*>(x.sm + x.oRank + (i & 1) * kRank + rank_offset(tok, 4 * gr)) = rank_key(middle);
        uint8_t* row = x.sm + x.oK + u * kUnit + tok * 128;
        if (packed && set == 0) {
          auto write = [&](auto lm) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[4], o[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t y = code_shift(w[c], q);
                if constexpr (decltype(lm)::value) {
                  v[c] = less_one_even(y);
                  o[c] = less_one_odd(y);
                  v[c] = hfma2(lm_extra(v[c]), d1, hmul2(v[c], s1));
                  o[c] = hfma2(lm_extra(o[c]), d1, hmul2(o[c], s1));
                } else {
                  v[c] = hmul2(less_one_even(y), s1);
                  o[c] = hmul2(less_one_odd(y), s1);
                }
              }
              *reinterpret_cast<uint4*>(row + (((2 * q) ^ (tok & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(row + (((2 * q + 1) ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          };
          write(Flag<LM>());
        } else if (packed) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t v[4], o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t y = code_shift(w[c], q);
              v[c] = by_sign(lm_extra(less_one_even(y)), left0, left3);
              o[c] = by_sign(lm_extra(less_one_odd(y)), left0, left3);
            }
            *reinterpret_cast<uint4*>(row + (((2 * q) ^ (tok & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(row + (((2 * q + 1) ^ (tok & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
          write_wide<kU>(wide && set == 0 ? wide + gr * 128 + half * 64 : nullptr, row, tok, down);
        }
        fence_async();
        __syncwarp();
        mbar_arrive_if(x.k_full + 8 * u, lane == 0);
      }
    }
  }
  return true;
}

// V, four warps.  Warp w holds tokens 64 h + 16 w .. + 15 of both unit halves h;
// lanes 16 c + j write the 64-channel block c of token 16 w + j.  For the
// exponents and the scale / zero pairs, fetched two tiles ahead, lane 16 h + j
// stands for the token of half h.  The exponents of a tile are published before
// the previous tile's units, which wait for products, are written.
template <int DG, int VU, int CB, int kStages, int kU, bool LM, bool RV>
__device__ __forceinline__ bool expand_v(const Share& x, int warp4, int lane) {
  const Geom& g = x.a->g;
  auto wait = [&](uint32_t bar, uint32_t parity) { return wait_warp(bar, parity, x.a->wait_turns); };
  const int steps = x.nt * DG, cb = lane >> 4, sub = 16 * warp4 + (lane & 15);
  const uint8_t* role = x.a->layer_base + g.role_bytes + g.sink_bytes + g.ring_bytes;
  const int64_t row0 = int64_t(x.u) * g.ncap + (x.p0 + sub - g.S);
  const uint8_t* codes = role + row0 * (32 * DG) + 16 * cb;
  const __half2* szs = reinterpret_cast<const __half2*>(role + g.codes_bytes) + (row0 + 64 * cb) * DG;
  const int pk0 = g.vb ? 0x7fffffff : g.S, pk1 = min(x.p1, max(g.S, x.T - g.W));  // INT2: pk0 <= position < pk1
  const uint32_t raw = x.base + x.oRawV + sub * 32 + 16 * cb;
  auto stage = [&](int k) {
    const int i = k / DG, pos = x.p0 + i * kTok + sub, st = (k % kStages) * kRawStage;
    const uint8_t* c = codes + int64_t(i) * (kTok * 32 * DG) + (k % DG) * 32;
    if (k < steps && pos >= pk0 && pos < pk1) cp_async16(raw + st, c);
    if (k < steps && pos + 64 >= pk0 && pos + 64 < pk1) cp_async16(raw + st + 64 * 32, c + 64 * 32 * DG);
    cp_async_commit();
  };
  const int mine = 64 * cb + sub;  // the lane's token for exponents
  const Tiles packed_tiles(x.p0, pk0, pk1);
  uint32_t sz[DG], nsz[DG], fsz[DG];  // this tile's pairs, the next one's and those on their way
  auto pairs = [&](int i, uint32_t (&d)[DG]) {
    const int pos = x.p0 + i * kTok + mine;
    const bool packed = pos >= pk0 && pos < pk1;
#pragma unroll
    for (int gr = 0; gr < DG; ++gr)
      d[gr] = packed ? __ldg(reinterpret_cast<const uint32_t*>(szs + int64_t(i) * (kTok * DG) + gr)) : 0u;
  };
  float e = 0.f, ne = 0.f;
  auto publish = [&](int i, const uint32_t (&pr)[DG]) {  // tile i's exponents
    const int pos = x.p0 + i * kTok + mine, slot = i % CB;
    float m = 0.f;
    if (pos >= pk0 && pos < pk1) {
#pragma unroll
      for (int j = 0; j < DG; ++j) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&pr[j]));
        m = fmax_nan(m, fmax_nan(fabsf(v.y), fabsf(fmaf(v.x, LM ? kLmSpan : 3.0f, v.y))));
      }
    } else if (pos < x.p1) {
      m = __uint_as_float(row_max<DG, 2 * kU>(row_ref(g, x.a->layer_base, 1, x.u, x.T, pos).wide));
    }
    // rows of ordinary size keep exponent 0
    ne = pos >= x.p1 ? -INFINITY
         : !isfinite(m) ? NAN
         : m >= 0x1p-8f && m < 0x1p12f ? 0.f : float(exponent_above(m));
    if (i >= CB && !wait(x.c_empty + 8 * slot, ((i / CB) & 1) ^ 1)) return false;
    const TileConsts<RV> tc(x.sm + x.oConst, slot);
    tc.e()[mine] = ne;
    if (RV) tc.rv()[mine] = rv_of(ne);
    const bool uneven = __any_sync(0xffffffffu, ne != 0.f);
    if (lane == 0) reinterpret_cast<volatile uint8_t*>(tc.uneven())[warp4] = uneven;  // one byte per warp
    __syncwarp();
    mbar_arrive_if(x.c_full + 8 * slot, lane == 0);
    return true;
  };
  auto ahead = [&](int i) {  // a BF16 row of tile i on its way to the L2 cache
    const int pos = x.p0 + i * kTok + mine;
    if (pos < x.p1 && (pos < pk0 || pos >= pk1)) prefetch_row<DG>(row_ref(g, x.a->layer_base, 1, x.u, x.T, pos).wide);
  };
  ahead(0);
  ahead(1);
  pairs(0, nsz);
  pairs(1, fsz);
#pragma unroll 1
  for (int k = 0; k < kStages - 1; ++k) stage(k);
  if (!publish(0, nsz)) return false;
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    stage(k + kStages - 1);
    const int i = k / DG, gr = k % DG;
    if (gr == 0) {
      e = ne;
#pragma unroll
      for (int j = 0; j < DG; ++j) sz[j] = nsz[j], nsz[j] = fsz[j];
      pairs(i + 2, fsz);
      if (!packed_tiles.has(i + 2)) ahead(i + 2);
      if (i + 1 < x.nt && !publish(i + 1, nsz)) return false;
    }
    cp_async_wait<kStages - 1>();
    __syncwarp();  // the other lane's half of the row has landed, too
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const int n = 2 * k + half, u = n % VU;
      const int pos = x.p0 + i * kTok + 64 * half + sub, from = 16 * half + (lane & 15);
      const float eh = __shfl_sync(0xffffffffu, e, from);
      uint32_t pair = 0;
#pragma unroll
      for (int j = 0; j < DG; ++j)
        if (j == gr) pair = __shfl_sync(0xffffffffu, sz[j], from);
      const uint8_t* st = x.sm + x.oRawV + (k % kStages) * kRawStage + (64 * half + sub) * 32;
      const uint4 c0 = *reinterpret_cast<const uint4*>(st), c1 = *reinterpret_cast<const uint4*>(st + 16);
      if (n >= VU && !wait(x.v_empty + 8 * u, ((n / VU) & 1) ^ 1)) return false;
      uint8_t* row = x.sm + x.oV + u * kUnit + cb * (kUnit / 2) + sub * 128;
      const bool fine = isfinite(eh);
      const float scale = fine ? pow2i(-int(eh)) : 0.f;
      if (fine && pos >= pk0 && pos < pk1) {
        const uint32_t sel = cb ? 0x7632u : 0x5410u;
        const uint32_t w[4] = {prmt(c0.x, c0.y, sel), prmt(c0.z, c0.w, sel), prmt(c1.x, c1.y, sel), prmt(c1.z, c1.w, sel)};
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&pair));
        // Uniform: c / 4 or c / 16 from 1 + that, exactly; then one rounding of s c + z.  Lloyd-Max: one of the unit, one
        // of the middle and one of the sum.
        uint32_t s_odd, s_even, z2;
        if (LM) {
          s_odd = s_even = half2_of(v.x * scale * (1.0f / 150.0f), v.x * scale * (1.0f / 150.0f));
          const float mid = fmaf(v.x, kLmMiddle, v.y) * scale;
          z2 = half2_of(mid, mid);
        } else {
          s_odd = half2_of(v.x * scale * 4.0f, v.x * scale * 4.0f);
          s_even = half2_of(v.x * scale * 16.0f, v.x * scale * 16.0f);
          z2 = half2_of(v.y * scale, v.y * scale);
        }
        auto write = [&](auto lm) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t a[4], o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t y = code_shift(w[c], q);
              if constexpr (decltype(lm)::value) {
                a[c] = hfma2(lm_value(less_one_even(y)), s_even, z2);
                o[c] = hfma2(lm_value(less_one_odd(y)), s_odd, z2);
              } else {
                a[c] = hfma2(hadd2(code_even(y), 0xBC00BC00u), s_even, z2);
                o[c] = hfma2(hadd2(code_odd(y), 0xBC00BC00u), s_odd, z2);
              }
            }
            *reinterpret_cast<uint4*>(row + (((2 * q) ^ (sub & 7)) << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
            *reinterpret_cast<uint4*>(row + (((2 * q + 1) ^ (sub & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        };
        write(Flag<LM>());
      } else {
        write_wide<kU>(fine && pos < x.p1 ? row_ref(g, x.a->layer_base, 1, x.u, x.T, pos).wide + gr * 128 + cb * 64 : nullptr, row, sub,
                       scale);
      }
      fence_async();
      __syncwarp();
      mbar_arrive_if(x.v_full + 8 * u, lane == 0);
    }
    __syncwarp();  // the stage has been read by both lanes before it is written again
  }
  return true;
}

}  // namespace oscar
