// Attention of blocks of query rows over one cache on the 5th-generation tensor
// cores: the kernel behind attn_extend and attn_decode_prefix when the output
// is bf16.
//
// One CTA holds N rotated query rows of one (sequence, KV head) and walks its
// share of the positions 128 at a time.  Both products are transposed, tokens
// (then channels) in the 128 TMEM lanes and query rows in the columns, so the
// cost of everything but the dequantisation follows the number of query rows:
//
//   S^T [128 tokens x N] = K [128 x 128] Q^T      per group of 128 channels
//   O^T [128 channels x N] += V^T [128 x 128 tokens] P^T
//
// and a token's scale, zero and exponents are one thread's scalars.
//
//   * Scores.  INT2 keys enter as the fp16 values y = 1 + code / 4 (Lloyd-Max:
//     150 times the level's distance from the middle, +-75 or +-249), which are
//     exact; the row's scale and zero are applied to the sum:
//       score = ks * sum_d q_d y_d + kz * sum_d q_d,
//     ks = 4 s, kz = z - 4 s.  BF16 keys are scaled by a power of two per row
//     and group (ks = 2^e, kz = 0), exact as well.  q, scaled by a power of two per CTA, is
//     the sum of two fp16 values, so scores have float32 accuracy.
//   * Probabilities carry the value row's exponent: with v_t = 2^(e_t) w_t, |w| < 1,
//     u = score + e_t, P = 2^(u - M) in fp16 and l += 2^(-e_t) 2^(u - M) in float32.
//     Value rows w in fp16 and P round with 2^-12 each, far below the bf16
//     output's 2^-9; without the exponent BF16 rows could leave fp16's range.
//   * The running reference M of a row need not be its maximum: P may reach
//     2^15.  A tile is computed with the M at hand; only when some t = u - M
//     exceeds 15 (the first tile, and rarely later) its columns get M = max - 6,
//     O^T and l are rescaled and P is computed again.  One barrier with an OR
//     per tile decides; no reduction over tokens is made otherwise.
//   * A value row that is not finite enters as zero with exponent NaN: rows that
//     see the token become NaN, rows that do not keep their values.
//
// Warps: two groups of four for the softmax (each all 128 tokens, N / 2
// columns), four that expand K, four that expand V, one thread that issues the
// MMAs.  K and V live in shared memory as units of 16 KB (64 channels of 128
// tokens; 64 tokens of 128 channels), the layout of both operands' 128-byte
// swizzle.
//
// Every wait is bounded; on a timeout the kernel flags OSCAR_DEV_TIMEOUT, waits
// (bounded) for its own MMAs and frees TMEM.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kTok = 128;              // positions per tile
constexpr int kUnit = 16384;           // bytes of a K or V unit
constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4 + 4 + 1) * 32;
constexpr float kNone = -1e30f;        // M before the first tile
constexpr float kTop = 15.f;           // largest t = u - M that P holds
constexpr float kRoom = 6.f;           // a new M lies this far below the maximum
constexpr int kConsts = 3;             // tiles whose token constants are kept

// Shared memory and TMEM of one instantiation.
template <int DG, int N>
struct Plan {
  static constexpr bool kBig = DG == 4 && N == 64;
  static constexpr int KU = kBig ? 2 : 4;                    // K units
  static constexpr int VU = kBig ? 2 : 3;                    // V units
  static constexpr int SB = kBig ? 1 : 2;                    // score buffers
  static constexpr int PB = (kBig || N == 128) ? 1 : 2;      // P buffers
  static constexpr int kQ = N * 256 * DG;                    // one of Q's two parts
  static constexpr int kP = (N > 64 ? 2 : 1) * kTok * 128;   // one P buffer
  static constexpr int oQ = 0;
  static constexpr int oP = oQ + 2 * kQ;
  static constexpr int oK = oP + PB * kP;
  static constexpr int oV = oK + KU * kUnit;
  static constexpr int oConst = oV + VU * kUnit;             // kConsts x (DG x 128 float2, 128 float)
  static constexpr int kConst = DG * kTok * 8 + kTok * 4;
  static constexpr int oRow = oConst + kConsts * kConst;     // per column: -M, limit, output row, factor, DG sums; scratch
  static constexpr int kRow = N * 4 * (4 + DG) + 8 * N / 2 * 4;
  static constexpr int oBar = oRow + kRow;
  static constexpr int kBars = 2 * KU + 2 * VU + 2 * SB + 2 * PB + 2 * kConsts + 2;
  static constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;  // + alignment slack
  static constexpr int cS = 0;                                // TMEM columns of the scores
  static constexpr int cO = SB * DG * N;                      // and of O^T
  static_assert(cO + DG * N <= 512, "TMEM");
  static_assert(kBytes <= 232448, "shared memory");
};

// Shared-memory descriptors, 128-byte swizzle.  K-major: 8-row groups 1024 bytes
// apart.  MN-major: 64-element blocks `lead` bytes apart, groups of eight k
// 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t saddr, uint32_t lead) {
  return uint64_t((saddr >> 4) & 0x3FFF) | (uint64_t(lead >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// kind::f16, fp16 operands, float32 accumulator, M = 128; bits 15 / 16: A / B MN-major.
template <int N>
__device__ __forceinline__ constexpr uint32_t idesc_of(bool mn_major) {
  return (1u << 4) | (mn_major ? 3u << 15 : 0u) | (uint32_t(N >> 3) << 17) | (uint32_t(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// true in every thread of the named barrier's 128 if it is in one of them
__device__ __forceinline__ bool any128(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n barrier.cta.red.or.pred q, %1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(id), "r"(uint32_t(p))
      : "memory");
  return r != 0;
}
// Bounded wait of a whole warp, given up at once when the CTA is aborting.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, int lane, const volatile uint32_t* abort_flag) {
  int ok = 1;
  if (lane == 0) ok = *abort_flag == 0 && mbar_wait(bar, parity);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
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
// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }
// smallest e in [-60, 126] with x < 2^e (x >= 0 finite; 126 is not enough for x >= 2^126, whose 2^-126 x < 4 still
// fits; below 2^-60 a row keeps an absolute precision of 2^-85)
__device__ __forceinline__ int exponent_above(float x) {
  return min(126, max(-60, (int(__float_as_uint(x)) >> 23) - 126));
}
// the two codes of a word at bits 2 p and 16 + 2 p, moved to bits 8 and 24
__device__ __forceinline__ uint32_t codes_at8(uint32_t w, int p) {
  const int sh = 8 - 2 * p;
  return (sh >= 0 ? w << sh : w >> -sh) & 0x03000300u;
}
// Lloyd-Max: 150 times the level's distance from the middle (rho + 1/2 levels),
// for codes at bits 8 and 24: with x = 2 c - 3, 150 (level - middle) = x (74 + x^2)
// (75 = 1 * 75, 249 = 3 * 83), every step exact in fp16.
__device__ __forceinline__ uint32_t lm_value(uint32_t c8) {
  const uint32_t x = hfma2(c8 | 0x3C003C00u, 0x48004800u /* 8 */, 0xC980C980u /* -11 */);
  return hmul2(x, hfma2(x, x, 0x54A054A0u /* 74 */));
}
constexpr float kLmMiddle = kLmRho + 0.5f;
// a bf16 pair times `scale`, as fp16
__device__ __forceinline__ uint32_t scaled_half2(uint32_t x, float scale) {
  return half2_of(__uint_as_float(x << 16) * scale, __uint_as_float(x & 0xFFFF0000u) * scale);
}

template <int DG, int N>
__global__ void __launch_bounds__(kThreads, 1) attn_rows_tc_kernel(const RowsArgs a) {
  using L = Plan<DG, N>;
  constexpr int D = DG * 128, C = N / 2;  // columns of a softmax group
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const Geom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // item: split s of row tile rt (last tiles first: with a causal mask they are the longest) of unit u
  const int units = g.B * g.Hkv, rows = a.n * g.G, tiles = (rows + N - 1) / N;
  const int s = int(blockIdx.x % unsigned(a.ns));
  const int it = int(blockIdx.x / unsigned(a.ns));
  const int u = it % units, rt = tiles - 1 - it / units;
  const int b = u / g.Hkv, h = u % g.Hkv;
  const int T = row_seq_len(a, b, threadIdx.x == 0 && rt == 0);
  const int ql = row_q_len(a, b);
  const int t_first = rt * N / g.G;
  if (t_first >= ql) return;  // only padding
  const int t_last = min((rt * N + N - 1) / g.G, ql - 1);
  const int vis = max(0, a.causal ? min(T, T - ql + t_last + 1) : T);
  const int see_all = a.causal ? T - ql + t_first : T - 1;  // every row sees the positions up to this one
  const int blocks = (vis + kTok - 1) / kTok;
  const int p0 = int(int64_t(blocks) * s / a.ns) * kTok;
  const int p1 = min(vis, int(int64_t(blocks) * (s + 1) / a.ns) * kTok);
  const int nt = (p1 - p0 + kTok - 1) / kTok;

  auto kconst = [&](int cb) { return reinterpret_cast<float2*>(sm + L::oConst + cb * L::kConst); };  // (ks, kz)
  auto econst = [&](int cb) { return reinterpret_cast<float*>(sm + L::oConst + cb * L::kConst + DG * kTok * 8); };
  float* negM = reinterpret_cast<float*>(sm + L::oRow);
  int* limit = reinterpret_cast<int*>(negM + N);   // last position that the row sees
  int* outr = limit + N;                            // its index among all query rows, -1 = none
  float* factor = reinterpret_cast<float*>(outr + N);
  float* qsum = factor + N;                         // [DG][N]
  float* part = qsum + DG * N;                      // [8 warps][C]
  const uint32_t bar = base + L::oBar;
  auto k_full = [&](int i) { return bar + 8u * i; };
  auto k_empty = [&](int i) { return bar + 8u * (L::KU + i); };
  auto v_full = [&](int i) { return bar + 8u * (2 * L::KU + i); };
  auto v_empty = [&](int i) { return bar + 8u * (2 * L::KU + L::VU + i); };
  constexpr int b1 = 2 * L::KU + 2 * L::VU;
  auto s_full = [&](int i) { return bar + 8u * (b1 + i); };
  auto s_empty = [&](int i) { return bar + 8u * (b1 + L::SB + i); };
  auto p_full = [&](int i) { return bar + 8u * (b1 + 2 * L::SB + i); };
  auto p_empty = [&](int i) { return bar + 8u * (b1 + 2 * L::SB + L::PB + i); };
  constexpr int b2 = b1 + 2 * L::SB + 2 * L::PB;
  auto c_full = [&](int i) { return bar + 8u * (b2 + i); };
  auto c_empty = [&](int i) { return bar + 8u * (b2 + kConsts + i); };
  const uint32_t q_full = bar + 8u * (b2 + 2 * kConsts), drained = q_full + 8;
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + L::oBar + L::kBars * 8);
  uint32_t* tmem_slot = words;
  volatile uint32_t* abort_flag = words + 1;
  uint32_t* qmax = words + 2;

  for (int c = threadIdx.x; c < N; c += kThreads) {
    const int row = rt * N + c, t = row / g.G;
    const bool live = row < rows && t < ql;
    outr[c] = live ? (b * a.n + t) * g.Hq + h * g.G + row % g.G : -1;
    limit[c] = live ? (a.causal ? T - ql + t : T - 1) : -1;
    negM[c] = -kNone;
    if (nt <= 0 && live) *reinterpret_cast<float2*>(a.ml + (int64_t(outr[c]) * a.ns + s) * 2) = make_float2(kNone, 0.f);
  }
  if (nt <= 0) return;  // nothing visible in this share
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::KU; ++i) mbar_init(k_full(i), 4), mbar_init(k_empty(i), 1);
    for (int i = 0; i < L::VU; ++i) mbar_init(v_full(i), 4), mbar_init(v_empty(i), 1);
    for (int i = 0; i < L::SB; ++i) mbar_init(s_full(i), 1), mbar_init(s_empty(i), kSoftWarps);
    for (int i = 0; i < L::PB; ++i) mbar_init(p_full(i), kSoftWarps), mbar_init(p_empty(i), 1);
    for (int i = 0; i < kConsts; ++i) mbar_init(c_full(i), 8), mbar_init(c_empty(i), kSoftWarps);
    mbar_init(q_full, kSoftWarps);
    mbar_init(drained, 1);
    mbar_fence_init();
    words[1] = 0;
    words[2] = 0;
  }
  if (warp == kSoftWarps + 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() {
    *abort_flag = 1;
    status_or(a.status, OSCAR_DEV_TIMEOUT);
  };
  auto wait = [&](uint32_t br, uint32_t parity) { return wait_warp(br, parity, lane, abort_flag); };

  if (warp < kSoftWarps) {
    // ------------------------------- softmax ---------------------------------
    const int grp = warp >> 2, c0 = grp * C;                // this group's columns
    const int tok = threadIdx.x & 127;                      // and this thread's token (TMEM lane)
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16; // the warp's TMEM lanes
    const int id = 1 + grp;                                 // named barrier of the group
    // Q: scaled by a power of two so that the largest component of the CTA's rows is just below 2^14, split into two
    // fp16 values (22 bits below that), written K-major; a warp takes one (row, group) at a time.
    {
      uint32_t mx = 0;
      for (int i = warp; i < N * DG; i += kSoftWarps) {
        const int r = outr[i / DG];
        if (r < 0) continue;
        const float4 v = *reinterpret_cast<const float4*>(a.qrot + int64_t(r) * D + (i % DG) * 128 + 4 * lane);
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (isfinite(f[e])) mx = max(mx, __float_as_uint(fabsf(f[e])));
      }
      mx = __reduce_max_sync(0xffffffffu, mx);
      if (lane == 0) atomicMax(qmax, mx);
    }
    asm volatile("bar.sync 3, 256;" ::: "memory");
    const int fe = max(-100, min(100, (int(*qmax) >> 23) - 126 - 14));  // q = 2^fe q^
    const float F = pow2i(fe), invF = pow2i(-fe);
    for (int i = warp; i < N * DG; i += kSoftWarps) {
      const int c = i / DG, gr = i % DG, r = outr[c];
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (r >= 0) {
        const float4 v = *reinterpret_cast<const float4*>(a.qrot + int64_t(r) * D + gr * 128 + 4 * lane);
        f[0] = v.x * invF, f[1] = v.y * invF, f[2] = v.z * invF, f[3] = v.w * invF;
      }
      uint32_t hi[2], lo[2];
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        hi[e] = half2_of(f[2 * e], f[2 * e + 1]);
        const float2 x = __half22float2(*reinterpret_cast<__half2*>(&hi[e]));
        lo[e] = half2_of(f[2 * e] - x.x, f[2 * e + 1] - x.y);
        const float2 y = __half22float2(*reinterpret_cast<__half2*>(&lo[e]));
        sum += (x.x + y.x) + (x.y + y.y);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      // channels 4 lane .. 4 lane + 3: block lane / 16, 16-byte chunk (lane / 2) % 8, half lane % 2
      const int off = (2 * gr + (lane >> 4)) * (N * 128) + c * 128 + ((((lane >> 1) & 7) ^ (c & 7)) << 4) + ((lane & 1) << 3);
      *reinterpret_cast<uint2*>(sm + L::oQ + off) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(sm + L::oQ + L::kQ + off) = make_uint2(lo[0], lo[1]);
      if (lane == 0) qsum[gr * N + c] = sum;
    }
    fence_async();
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (lane == 0) mbar_arrive(q_full);

    uint64_t l2[C / 2];  // this token's part of l, two columns at a time
#pragma unroll
    for (int i = 0; i < C / 2; ++i) l2[i] = 0;
    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      const int sb = i % L::SB, pb = i % L::PB, cb = i % kConsts;
      const int pos = p0 + i * kTok + tok;
      ok = ok && wait(c_full(cb), (i / kConsts) & 1);
      ok = ok && wait(s_full(sb), (i / L::SB) & 1);
      if (i >= L::PB) ok = ok && wait(p_empty(pb), ((i / L::PB) & 1) ^ 1);
      fence_after();
      uint64_t ks[DG], kz[DG];
#pragma unroll
      for (int gr = 0; gr < DG; ++gr) {
        const float2 k = kconst(cb)[gr * kTok + tok];
        ks[gr] = splat_x2(k.x * F);
        kz[gr] = splat_x2(k.y * F);
      }
      const float e = econst(cb)[tok];
      const uint64_t e2 = splat_x2(e), rv2 = splat_x2(isfinite(e) ? pow2i(-int(e)) : 1.f);
      const bool masked = p0 + i * kTok + kTok - 1 > see_all;  // some row does not see some position of the tile
      uint8_t* P = sm + L::oP + pb * L::kP + tok * 128;
      const uint32_t S = tmem + lanes + L::cS + sb * DG * N;
      // t = u - M (or u) of columns c .. c + 15
      auto scores = [&](int c, float (&t)[16], bool less_m) {
        uint64_t x[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          if (less_m) {
            const ulonglong2 m = *reinterpret_cast<const ulonglong2*>(negM + c + 2 * j);
            x[j] = add2(e2, m.x);
            x[j + 1] = add2(e2, m.y);
          } else {
            x[j] = x[j + 1] = e2;
          }
        }
        constexpr int GS = DG > 1 ? 2 : 1;  // groups in flight
#pragma unroll
        for (int g0 = 0; g0 < DG; g0 += GS) {
          uint32_t r[GS][16];
#pragma unroll
          for (int gr = 0; gr < GS; ++gr) tmem_ld16(S + (g0 + gr) * N + c, r[gr]);
#pragma unroll
          for (int gr = 0; gr < GS; ++gr)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qsum + (g0 + gr) * N + c + 2 * j);
              x[j] = fma2(q.x, kz[g0 + gr], x[j]);
              x[j + 1] = fma2(q.y, kz[g0 + gr], x[j + 1]);
            }
#pragma unroll
          for (int gr = 0; gr < GS; ++gr) tmem_wait16(r[gr]);
#pragma unroll
          for (int gr = 0; gr < GS; ++gr)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = fma2(pack2(__uint_as_float(r[gr][2 * j]), __uint_as_float(r[gr][2 * j + 1])), ks[g0 + gr], x[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) unpack2(x[j], t[2 * j], t[2 * j + 1]);
        if (masked) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (pos > limit[c + j]) t[j] = -INFINITY;
        }
      };
      auto store = [&](int c, const float (&p)[16]) {
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          const int cc = c + j;
          *reinterpret_cast<uint4*>(P + (cc >> 6) * (kTok * 128) + ((((cc >> 3) & 7) ^ (tok & 7)) << 4)) =
              make_uint4(half2_of(p[j], p[j + 1]), half2_of(p[j + 2], p[j + 3]), half2_of(p[j + 4], p[j + 5]),
                         half2_of(p[j + 6], p[j + 7]));
        }
      };
      // the first tile has no M yet and goes straight to the search for one
      float top = INFINITY;
      if (i > 0) {
        top = -INFINITY;
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          float t[16];
          scores(c0 + c, t, true);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            top = max3(top, t[j], t[j + 1]);
            t[j] = ex2(t[j]);
            t[j + 1] = ex2(t[j + 1]);
            l2[(c + j) / 2] = fma2(pack2(t[j], t[j + 1]), rv2, l2[(c + j) / 2]);
          }
          store(c0 + c, t);
        }
      }
      if (any128(id, !ok || top > kTop)) {
        if (any128(id, !ok)) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        // Some column left the range of P: the largest u of every column of the tile, and a new M where needed.
#pragma unroll 1
        for (int c = 0; c < C; c += 16) {
          float t[16];
          scores(c0 + c, t, false);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int x = __float_as_int(t[j] == t[j] ? t[j] : -INFINITY);
            const int key = __reduce_max_sync(0xffffffffu, x ^ ((x >> 31) & 0x7fffffff));
            if (lane == 0) part[warp * C + c + j] = __int_as_float(key ^ ((key >> 31) & 0x7fffffff));
          }
        }
        asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
        if (tok < C) {
          const float* w = part + grp * 4 * C + tok;
          const float mx = fmaxf(fmaxf(w[0], w[C]), fmaxf(w[2 * C], w[3 * C]));
          const float M = -negM[c0 + tok];
          float f = 1.f;
          if (mx - M > kTop) {
            f = exp2f(M - (mx - kRoom));
            negM[c0 + tok] = kRoom - mx;
          }
          factor[c0 + tok] = f;
        }
        // O^T must not be in use while it is rescaled: the previous tile's product is complete
        if (i > 0) ok = wait(p_empty((i - 1) % L::PB), ((i - 1) / L::PB) & 1);
        if (any128(id, !ok)) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        fence_after();
        if (i > 0) {
#pragma unroll 1
          for (int gr = 0; gr < DG; ++gr)
#pragma unroll 1
            for (int c = 0; c < C; c += 16) {
              uint32_t r[16];
              const uint32_t at = tmem + lanes + L::cO + gr * N + c0 + c;
              tmem_ld16(at, r);
              tmem_wait16(r);
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * factor[c0 + c + j]);
              tmem_st16(at, r);
            }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        // l already holds this tile at the old M, which is right unless a step of 2^100 or more made it infinite; what
        // this token had before is then below the resolution of its new term (by 2^44 more than the value rows'
        // magnitudes differ)
#pragma unroll
        for (int c = 0; c < C; c += 16) {
          float t[16];
          scores(c0 + c, t, true);
#pragma unroll
          for (int j = 0; j < 16; ++j) t[j] = ex2(t[j]);
          float rv, unused;
          unpack2(rv2, rv, unused);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float x, y;
            unpack2(l2[(c + j) / 2], x, y);
            const float fx = factor[c0 + c + j], fy = factor[c0 + c + j + 1];
            x = i == 0 || x == INFINITY ? t[j] * rv : x * fx;
            y = i == 0 || y == INFINITY ? t[j + 1] * rv : y * fy;
            l2[(c + j) / 2] = pack2(x, y);
          }
          store(c0 + c, t);
        }
      }
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(s_empty(sb));
        mbar_arrive(p_full(pb));
        mbar_arrive(c_empty(cb));
      }
    }
    // sums over the tokens, then O^T
    if (ok) ok = wait(p_empty((nt - 1) % L::PB), ((nt - 1) / L::PB) & 1);
    if (!any128(id, !ok)) {
      fence_after();
      if constexpr (C >= 32) {
#pragma unroll
        for (int c = 0; c < C; c += 32) {
          float v[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) unpack2(l2[c / 2 + j], v[2 * j], v[2 * j + 1]);
          part[warp * C + c + lane] = sum_columns(v, lane);
        }
      } else {
        float v[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) unpack2(l2[j], v[2 * j], v[2 * j + 1]);
        part[warp * C + (lane & 15)] = sum_columns(v, lane);
      }
      asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
      if (tok < C && outr[c0 + tok] >= 0) {
        const float* w = part + grp * 4 * C + tok;
        *reinterpret_cast<float2*>(a.ml + (int64_t(outr[c0 + tok]) * a.ns + s) * 2) =
            make_float2(-negM[c0 + tok], (w[0] + w[C]) + (w[2 * C] + w[3 * C]));
      }
#pragma unroll 1
      for (int gr = 0; gr < DG; ++gr)
#pragma unroll 1
        for (int c = 0; c < C; c += 16) {
          uint32_t r[16];
          tmem_ld16(tmem + lanes + L::cO + gr * N + c0 + c, r);
          tmem_wait16(r);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int row = outr[c0 + c + j];
            if (row >= 0) a.acc[(int64_t(row) * a.ns + s) * D + gr * 128 + 32 * (warp & 3) + lane] = __uint_as_float(r[j]);
          }
        }
    } else if (lane == 0) {
      fail();
    }
  } else if (warp < kSoftWarps + 4) {
    // ------------------------- K: codes to operands ---------------------------
    const int tok = threadIdx.x - kSoftWarps * 32;
    struct Raw {
      RowRef ref;
      uint4 c0, c1;
      __half2 sz;
    };
    auto load = [&](int k, Raw& x) {  // (tile k / DG, group k % DG)
      const int pos = p0 + k / DG * kTok + tok;
      x.ref = RowRef{nullptr, nullptr, nullptr};
      if (k >= nt * DG || pos >= p1) return;
      x.ref = row_ref(g, a.layer_base, 0, u, T, pos);
      if (x.ref.codes) {
        const uint4* c = reinterpret_cast<const uint4*>(x.ref.codes + 8 * (k % DG));
        x.c0 = __ldg(c);
        x.c1 = __ldg(c + 1);
        x.sz = __ldg(x.ref.sz + k % DG);
      }
    };
    auto emit = [&](int k, const Raw& x) {
      const int i = k / DG, gr = k % DG, cb = i % kConsts;
      if (gr == 0 && i >= kConsts && !wait(c_empty(cb), ((i / kConsts) & 1) ^ 1)) return false;
      float scale = 0.f;
      float2 kk = make_float2(0.f, 0.f);
      if (x.ref.wide) {
        uint32_t m = 0;
        const uint4* src = reinterpret_cast<const uint4*>(x.ref.wide + gr * 128);
#pragma unroll 4
        for (int j = 0; j < 16; ++j) {
          const uint4 v = src[j];
          m = absmax2(absmax2(absmax2(absmax2(m, v.x), v.y), v.z), v.w);
        }
        m = max(m & 0xFFFFu, m >> 16);
        const int e = max(-104, int(m >> 7) - 126) - 15;  // 2^-e times the row's largest value is just below 2^15
        scale = pow2i(-e);
        kk.x = pow2i(e);
      } else if (x.ref.codes) {
        const float2 sz = __half22float2(x.sz);
        if (g.lm) kk = make_float2(sz.x * (1.0f / 150.0f), fmaf(sz.x, kLmMiddle, sz.y));
        else kk = make_float2(4.0f * sz.x, fmaf(-4.0f, sz.x, sz.y));
      }
      kconst(cb)[gr * kTok + tok] = kk;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = 2 * k + half, st = n % L::KU;
        if (n >= L::KU && !wait(k_empty(st), ((n / L::KU) & 1) ^ 1)) return false;
        uint8_t* row = sm + L::oK + st * kUnit + tok * 128;
        if (x.ref.codes) {
          // word 2 c + half: pair c of every 16-byte chunk
          const uint32_t w[4] = {half ? x.c0.y : x.c0.x, half ? x.c0.w : x.c0.z, half ? x.c1.y : x.c1.x, half ? x.c1.w : x.c1.z};
          if (g.lm) {
#pragma unroll
            for (int p = 0; p < 8; ++p)
              *reinterpret_cast<uint4*>(row + ((p ^ (tok & 7)) << 4)) =
                  make_uint4(lm_value(codes_at8(w[0], p)), lm_value(codes_at8(w[1], p)), lm_value(codes_at8(w[2], p)),
                             lm_value(codes_at8(w[3], p)));
          } else {
#pragma unroll
            for (int p = 0; p < 8; ++p)
              *reinterpret_cast<uint4*>(row + ((p ^ (tok & 7)) << 4)) =
                  make_uint4(codes_at8(w[0], p) | 0x3C003C00u, codes_at8(w[1], p) | 0x3C003C00u,
                             codes_at8(w[2], p) | 0x3C003C00u, codes_at8(w[3], p) | 0x3C003C00u);
          }
        } else {
#pragma unroll 2
          for (int p = 0; p < 8; ++p) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (x.ref.wide) v = reinterpret_cast<const uint4*>(x.ref.wide + gr * 128 + half * 64)[p];
            *reinterpret_cast<uint4*>(row + ((p ^ (tok & 7)) << 4)) =
                make_uint4(scaled_half2(v.x, scale), scaled_half2(v.y, scale), scaled_half2(v.z, scale), scaled_half2(v.w, scale));
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full(st));
      }
      if (gr == DG - 1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(c_full(cb));
      }
      return true;
    };
    Raw x, y;
    load(0, x);
    load(1, y);
    bool ok = true;
    for (int k = 0; ok && k < nt * DG; k += 2) {
      ok = emit(k, x);
      load(k + 2, x);
      if (ok && k + 1 < nt * DG) ok = emit(k + 1, y);
      load(k + 3, y);
    }
    if (!ok && lane == 0) fail();
  } else if (warp < kSoftWarps + 8) {
    // ------------------------- V: codes to operands ---------------------------
    const int tid = threadIdx.x - (kSoftWarps + 4) * 32;
    const int cb = lane >> 4;                                // 64-channel block
    const int sub = 16 * (warp & 3) + (lane & 15);           // token within a unit
    struct Raw {
      RowRef ref;
      uint4 c0, c1;
      __half2 sz;
    };
    auto load = [&](int k, Raw& x) {  // unit k: tile k / (2 DG), group (k / 2) % DG, token half k % 2
      const int pos = p0 + k / (2 * DG) * kTok + 64 * (k & 1) + sub, gr = (k >> 1) % DG;
      x.ref = RowRef{nullptr, nullptr, nullptr};
      if (k >= 2 * nt * DG || pos >= p1) return;
      x.ref = row_ref(g, a.layer_base, 1, u, T, pos);
      if (x.ref.codes) {
        const uint4* c = reinterpret_cast<const uint4*>(x.ref.codes + 8 * gr);
        x.c0 = __ldg(c);
        x.c1 = __ldg(c + 1);
        x.sz = __ldg(x.ref.sz + gr);
      }
    };
    bool ok = true;  // a warp that gave up still comes to the group's next barrier
    // the exponents of a tile's 128 tokens, one per thread
    auto exponents = [&](int i) {
      const int buf = i % kConsts, pos = p0 + i * kTok + tid;
      if (i >= kConsts) ok = ok && wait(c_empty(buf), ((i / kConsts) & 1) ^ 1);
      float e = -INFINITY;
      if (pos < p1) {
        const RowRef r = row_ref(g, a.layer_base, 1, u, T, pos);
        float m = 0.f;
        if (r.codes) {
          for (int gr = 0; gr < DG; ++gr) {
            const float2 sz = __half22float2(__ldg(r.sz + gr));
            m = fmax_nan(m, fmax_nan(fabsf(sz.y), fabsf(fmaf(sz.x, g.lm ? kLmSpan : 3.0f, sz.y))));
          }
        } else {
          uint32_t w = 0;
          const uint4* src = reinterpret_cast<const uint4*>(r.wide);
#pragma unroll 4
          for (int j = 0; j < D / 8; ++j) {
            const uint4 v = src[j];
            w = absmax2(absmax2(absmax2(absmax2(w, v.x), v.y), v.z), v.w);
          }
          m = __uint_as_float(max(w & 0xFFFFu, w >> 16) << 16);
        }
        e = isfinite(m) ? float(exponent_above(m)) : NAN;
      }
      econst(buf)[tid] = e;
      __syncwarp();
      if (lane == 0) mbar_arrive(c_full(buf));
      return !any128(4, !ok);  // the group's exponents are written
    };
    auto emit = [&](int k, const Raw& x) {
      if (k % (2 * DG) == 0 && !exponents(k / (2 * DG))) return false;
      const int st = k % L::VU, gr = (k >> 1) % DG;
      const float e = econst(k / (2 * DG) % kConsts)[64 * (k & 1) + sub];
      if (k >= L::VU) ok = ok && wait(v_empty(st), ((k / L::VU) & 1) ^ 1);
      if (!ok) return true;
      uint8_t* row = sm + L::oV + st * kUnit + cb * (kUnit / 2) + sub * 128;
      const float scale = isfinite(e) ? pow2i(-int(e)) : 0.f;
      if (x.ref.codes && isfinite(e)) {
        const uint32_t sel = cb ? 0x7632u : 0x5410u;
        const uint32_t w[4] = {prmt(x.c0.x, x.c0.y, sel), prmt(x.c0.z, x.c0.w, sel), prmt(x.c1.x, x.c1.y, sel),
                               prmt(x.c1.z, x.c1.w, sel)};
        const float2 sz = __half22float2(x.sz);
        if (g.lm) {
          const uint32_t s2 = half2_of(sz.x * scale * (1.0f / 150.0f), sz.x * scale * (1.0f / 150.0f));
          const float mid = fmaf(sz.x, kLmMiddle, sz.y) * scale;
          const uint32_t z2 = half2_of(mid, mid);
#pragma unroll
          for (int p = 0; p < 8; ++p)
            *reinterpret_cast<uint4*>(row + ((p ^ (sub & 7)) << 4)) =
                make_uint4(hfma2(lm_value(codes_at8(w[0], p)), s2, z2), hfma2(lm_value(codes_at8(w[1], p)), s2, z2),
                           hfma2(lm_value(codes_at8(w[2], p)), s2, z2), hfma2(lm_value(codes_at8(w[3], p)), s2, z2));
        } else {
          // a code at bits 8 and 9 of a half is 2^-16 times the code (a subnormal, multiplied exactly)
          const uint32_t s2 = half2_of(sz.x * scale * 65536.0f, sz.x * scale * 65536.0f);
          const uint32_t z2 = half2_of(sz.y * scale, sz.y * scale);
#pragma unroll
          for (int p = 0; p < 8; ++p)
            *reinterpret_cast<uint4*>(row + ((p ^ (sub & 7)) << 4)) =
                make_uint4(hfma2(codes_at8(w[0], p), s2, z2), hfma2(codes_at8(w[1], p), s2, z2),
                           hfma2(codes_at8(w[2], p), s2, z2), hfma2(codes_at8(w[3], p), s2, z2));
        }
      } else {
        const uint4* src = x.ref.wide && isfinite(e) ? reinterpret_cast<const uint4*>(x.ref.wide + gr * 128 + cb * 64) : nullptr;
#pragma unroll 2
        for (int p = 0; p < 8; ++p) {
          const uint4 v = src ? src[p] : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(row + ((p ^ (sub & 7)) << 4)) =
              make_uint4(scaled_half2(v.x, scale), scaled_half2(v.y, scale), scaled_half2(v.z, scale), scaled_half2(v.w, scale));
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_full(st));
      return true;
    };
    Raw x, y;
    load(0, x);
    load(1, y);
    for (int k = 0; k < 2 * nt * DG; k += 2) {
      if (!emit(k, x)) break;  // the whole group leaves
      load(k + 2, x);
      emit(k + 1, y);  // an odd unit starts no tile
      load(k + 3, y);
    }
    if (!ok && lane == 0) fail();
  } else if (lane == 0) {
    // ------------------------------ MMA issuer --------------------------------
    constexpr uint32_t id_qk = idesc_of<N>(false), id_pv = idesc_of<N>(true);
    const uint32_t sQ = base + L::oQ, sK = base + L::oK, sV = base + L::oV, sP = base + L::oP;
    auto wait1 = [&](uint32_t br, uint32_t parity) { return *abort_flag == 0 && mbar_wait(br, parity); };
    auto product_qk = [&](int i) {
      const int sb = i % L::SB;
      if (i >= L::SB && !wait1(s_empty(sb), ((i / L::SB) & 1) ^ 1)) return false;
      for (int kb = 0; kb < 2 * DG; ++kb) {
        const int n = i * 2 * DG + kb, st = n % L::KU;
        if (!wait1(k_full(st), (n / L::KU) & 1)) return false;
        fence_after();
        const uint32_t d = tmem + L::cS + (sb * DG + (kb >> 1)) * N;
#pragma unroll
        for (int part = 0; part < 2; ++part)  // Q's high, then its low part
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ss(d, desc_of(sK + st * kUnit + 32 * k, 16), desc_of(sQ + part * L::kQ + kb * (N * 128) + 32 * k, 16),
                       id_qk, (kb & 1) | part | k);
        mma_commit(k_empty(st));
      }
      mma_commit(s_full(sb));
      return true;
    };
    auto product_pv = [&](int i) {
      const int pb = i % L::PB;
      if (!wait1(p_full(pb), (i / L::PB) & 1)) return false;
      for (int k = 0; k < 2 * DG; ++k) {  // group k / 2, token half k % 2
        const int n = i * 2 * DG + k, st = n % L::VU;
        if (!wait1(v_full(st), (n / L::VU) & 1)) return false;
        fence_after();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16_ss(tmem + L::cO + (k >> 1) * N, desc_of(sV + st * kUnit + 2048 * j, kUnit / 2),
                     desc_of(sP + pb * L::kP + (k & 1) * 8192 + 2048 * j, kTok * 128), id_pv, i | (k & 1) | j);
        mma_commit(v_empty(st));
      }
      mma_commit(p_empty(pb));
      return true;
    };
    bool ok = wait1(q_full, 0);
    if (ok) {
      fence_after();
      ok = product_qk(0);
    }
    for (int i = 0; ok && i < nt; ++i) {
      if (i + 1 < nt) ok = product_qk(i + 1);
      if (ok) ok = product_pv(i);
    }
    if (!ok) fail();
    mma_commit(drained);  // every product issued is complete before TMEM is freed
    mbar_wait(drained, 0);
  }
  fence_before();
  __syncthreads();
  if (warp == kSoftWarps + 8) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int DG, int N>
int launch(const RowsArgs& a, cudaStream_t stream) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_rows_tc_kernel<DG, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Plan<DG, N>::kBytes) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int64_t tiles = (int64_t(a.n) * a.g.G + N - 1) / N;
  const int64_t items = tiles * a.g.B * a.g.Hkv * a.ns;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_rows_tc_kernel<DG, N><<<unsigned(items), kThreads, Plan<DG, N>::kBytes, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

// Query rows per CTA: the smallest tile that holds a unit's rows, at most what TMEM and shared memory hold.
int tile_rows(int D, int64_t rows) {
  if (rows <= 32) return 32;
  return rows <= 64 || D > 128 ? 64 : 128;
}

}  // namespace

int rows_splits_tc(const Geom& g, int64_t rows, int seq_len_hint) {
  const int N = tile_rows(g.D, rows);
  const int64_t items = (rows + N - 1) / N * g.B * g.Hkv;
  const int64_t blocks = (int64_t(seq_len_hint) + kTok - 1) / kTok;
  // time of ns splits: waves of CTAs on 152 SMs, each its tiles and a fixed part worth `fixed` tiles
  const double fixed = 6.0;
  int best = 1;
  double least = 1e300;
  for (int ns = 1; ns <= OSCAR_KV_MAX_SPLITS && ns <= blocks; ++ns) {
    const double waves = double((items * ns + 151) / 152);
    const double t = waves * (fixed + double((blocks + ns - 1) / ns));
    if (t < least * 0.98) least = t, best = ns;
  }
  return best;
}

int launch_attn_rows_tc(const RowsArgs& a, cudaStream_t stream) {
  const int N = tile_rows(a.g.D, int64_t(a.n) * a.g.G);
  if (a.g.D == 128) return N == 32 ? launch<1, 32>(a, stream) : N == 64 ? launch<1, 64>(a, stream) : launch<1, 128>(a, stream);
  if (a.g.D == 256) return N == 32 ? launch<2, 32>(a, stream) : launch<2, 64>(a, stream);
  return N == 32 ? launch<4, 32>(a, stream) : launch<4, 64>(a, stream);
}

}  // namespace oscar
