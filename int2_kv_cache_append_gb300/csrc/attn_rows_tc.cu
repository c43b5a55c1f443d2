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
//   * Scores.  INT2 keys enter the product exactly, as s (c - 1) with the middles
//     z + s as a rank-one term, BF16 keys exactly (expand_k in rows_tc.cuh); q,
//     scaled by a power of two per row, is the sum of two fp16 values.  So the
//     products' sums are scores of float32 accuracy.
//   * Probabilities carry the value row's exponent: with v_t = 2^(e_t) w_t, |w| < 1,
//     u = score + e_t, P = 2^(u - M) in fp16 and l += 2^(-e_t) 2^(u - M) in float32.
//     Value rows w in fp16 and P round with 2^-11 each, far below the bf16
//     output's 2^-8; without the exponent BF16 rows could leave fp16's range.
//   * The running reference M of a row need not be its maximum: P may reach
//     2^15.  A tile is computed with the M at hand; only when some t = u - M
//     exceeds 15 (the first tile, and rarely later) its columns get the maximum
//     less 8 as M, O^T and l are rescaled and P is computed again.  Below 2^-14 P
//     is off by up to 2^-25, so with the maximum at 2^8 or above a weight is off
//     by 2^-33 of the largest; with M at the maximum every weight below 2^-25 of
//     it would be lost, 2^-8 of the sum beside 131,072 of them.  One barrier with an
//     OR per tile decides; no reduction over tokens is made otherwise.
//   * A value row that is not finite enters as zero with exponent NaN: rows that
//     see the token become NaN, rows that do not keep their values.
//
// Warps: two groups of four for the softmax (each all 128 tokens, N / 2
// columns), four that expand K, four that expand V, one thread that issues the
// MMAs.  K and V live in shared memory as units of 16 KB (64 channels of 128
// tokens; 64 tokens of 128 channels), the layout of both operands' 128-byte
// swizzle.
//
// What bounds it: the expansion, 16-bit arithmetic on every code and its stores
// to shared memory, by the eight expanding warps; per tile of 128 positions and
// group about 4200 cycles with INT2 rows and three times that where the rows are
// BF16 (their loads' latency).  16,384 positions, 8 KV heads, 8 sequences x 5
// tokens at D = 128: 106 us with INT2 rows only, 346 us with BF16 rows only; 4 x
// 32 tokens at D = 512, INT2 rows only: 284 us.
// Twice the expanding warps (which halves the registers) were slower, as were
// rolled loops and reading BF16 rows by whole warps, line by line.
//
// Every wait is bounded; on a timeout the kernel flags OSCAR_DEV_TIMEOUT, waits
// (bounded) for its own MMAs and frees TMEM.
#include <algorithm>

#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4 + 4 + 1) * 32;
constexpr float kNone = -1e30f;        // M before the first tile
constexpr float kTop = 15.f;           // largest t = u - M that P holds (fp16 below 2^16)
constexpr float kBelow = 8.f;          // a new M lies this far below its tile's maximum

// Shared memory and TMEM of one instantiation.
template <int DG, int N>
struct Plan {
  static constexpr bool kBig = DG == 4 && N == 64;
  static constexpr bool kFull = DG * N >= 128;               // Q leaves room for fewer buffers
  static constexpr int KU = kBig ? 2 : kFull ? 3 : 4;        // K units
  static constexpr int VU = kBig ? 1 : 3;                    // V units
  static constexpr int SB = 2;                               // score buffers
  static constexpr int PB = kFull ? 1 : 2;                   // P buffers
  static constexpr int CB = 3;                               // tiles whose constants are kept
  static constexpr int kStages = kBig ? 2 : DG * N == 32 ? 5 : 3;  // (tile, group) steps whose codes are staged, plus one
  static constexpr int kQ = N * 256 * DG;                    // one of Q's two parts
  static constexpr int kP = kTok * 128;                      // one P buffer
  static constexpr int oQ = 0;
  static constexpr int oP = oQ + 2 * kQ;
  static constexpr int oK = oP + PB * kP;
  static constexpr int oV = oK + KU * kUnit;
  static constexpr int oRawK = oV + VU * kUnit;
  static constexpr int oRawV = oRawK + kStages * kRawStage;
  static constexpr int oRank = oRawV + kStages * kRawStage;  // the keys' two and the queries' rank-one operands
  static constexpr int oConst = oRank + 2 * kRank + N * 32;
  static constexpr int oRow = oConst + CB * TileConsts<false>::kBytes;  // per column: -M, limit, output row, factor, query scale; sums
  static constexpr int kRow = N * 5 * 4 + 8 * N / 2 * 4;
  static constexpr int oBar = oRow + kRow;
  static constexpr int kBars = 2 * KU + 2 * VU + 2 * SB + 2 * PB + 2 * CB + 2;
  static constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;  // + alignment slack
  // The tensor cores cut each of their sums' additions off (towards zero).  At D = 512 a score would be 65 additions and
  // 1e-6 too small, so at D = 256 and 512 two accumulators share them.
  static constexpr int kParts = DG > 1 ? 2 : 1;
  static constexpr int cS = 0;                                // TMEM columns of the scores
  static constexpr int cO = SB * kParts * N;                  // and of O^T
  static_assert(cO + DG * N <= 512, "TMEM");
  static_assert(kBytes <= 232448, "shared memory");
};

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
  if (t_first >= ql) {  // only padding
    rows_wait(a);
    return;
  }
  const int t_last = min((rt * N + N - 1) / g.G, ql - 1);
  const int vis = max(0, a.causal ? min(T, T - ql + t_last + 1) : T);
  const int see_all = a.causal ? T - ql + t_first : T - 1;  // every row sees the positions up to this one
  const int blocks = (vis + kTok - 1) / kTok;
  const int p0 = share_start(g, T, blocks, s, a.ns) * kTok;
  const int p1 = min(vis, share_start(g, T, blocks, s + 1, a.ns) * kTok);
  const int nt = (p1 - p0 + kTok - 1) / kTok;

  float* negM = reinterpret_cast<float*>(sm + L::oRow);
  int* limit = reinterpret_cast<int*>(negM + N);   // last position that the row sees
  int* outr = limit + N;                            // its index among all query rows, -1 = none
  float* factor = reinterpret_cast<float*>(outr + N);
  float* qscale = factor + N;                       // power of two that undoes the row's scaling
  float* part = qscale + N;                         // [8 warps][C]
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
  auto c_empty = [&](int i) { return bar + 8u * (b2 + L::CB + i); };
  const uint32_t q_full = bar + 8u * (b2 + 2 * L::CB), drained = q_full + 8;
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + L::oBar + L::kBars * 8);
  uint32_t* tmem_slot = words;

  for (int c = threadIdx.x; c < N; c += kThreads) {
    const int row = rt * N + c, t = row / g.G;
    const bool live = row < rows && t < ql;
    outr[c] = live ? (b * a.n + t) * g.Hq + h * g.G + row % g.G : -1;
    limit[c] = live ? (a.causal ? T - ql + t : T - 1) : -1;
    negM[c] = -kNone;
    if (nt <= 0 && live) *reinterpret_cast<float2*>(a.ml + (int64_t(outr[c]) * a.ns + s) * 2) = make_float2(kNone, 0.f);
  }
  if (nt <= 0) {  // nothing visible in this share
    rows_wait(a);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::KU; ++i) mbar_init(k_full(i), 4), mbar_init(k_empty(i), 1);
    for (int i = 0; i < L::VU; ++i) mbar_init(v_full(i), 4), mbar_init(v_empty(i), 1);
    for (int i = 0; i < L::SB; ++i) mbar_init(s_full(i), 1 + (i == 0 && a.wait_poison > 0)), mbar_init(s_empty(i), kSoftWarps);
    for (int i = 0; i < L::PB; ++i) mbar_init(p_full(i), kSoftWarps), mbar_init(p_empty(i), 1);
    for (int i = 0; i < L::CB; ++i) mbar_init(c_full(i), 8), mbar_init(c_empty(i), kSoftWarps);
    mbar_init(q_full, kSoftWarps);
    mbar_init(drained, 1);
    mbar_fence_init();
    if (a.beside && !ready_wait(a.ready, a.wait_turns * 1000ull)) status_or(a.status, OSCAR_DEV_TIMEOUT);  // the queries
  }
  if (warp == kSoftWarps + 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (!a.beside) rows_wait(a);  // the queries
  if (a.early) pdl_trigger();
  auto fail = [&]() {
    status_or(a.status, OSCAR_DEV_TIMEOUT);
  };
  auto wait = [&](uint32_t br, uint32_t parity) { return wait_warp(br, parity, a.wait_turns); };

  if (warp < kSoftWarps) {
    // ------------------------------- softmax ---------------------------------
    const int grp = warp >> 2, c0 = grp * C;                // this group's columns
    const int tok = threadIdx.x & 127;                      // and this thread's token (TMEM lane)
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16; // the warp's TMEM lanes
    const int id = 1 + grp;                                 // named barrier of the group
    load_queries<DG, N, kSoftWarps>(a, sm + L::oQ, L::kQ, outr, sm + L::oRank + 2 * kRank, qscale, warp, lane);
    mbar_arrive_if(q_full, lane == 0);

    uint64_t l2[C / 2];  // this token's part of l, two columns at a time
#pragma unroll
    for (int i = 0; i < C / 2; ++i) l2[i] = 0;
    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      const int sb = i % L::SB, pb = i % L::PB, cb = i % L::CB;
      const int pos = p0 + i * kTok + tok;
      ok = ok && wait(c_full(cb), (i / L::CB) & 1);
      ok = ok && wait(s_full(sb), (i / L::SB) & 1);
      if (i >= L::PB) ok = ok && wait(p_empty(pb), ((i / L::PB) & 1) ^ 1);
      fence_after();
      const TileConsts<false> tc(sm + L::oConst, cb);
      const uint64_t phi2 = splat_x2(tc.k()[tok]);
      const uint64_t e2 = splat_x2(tc.e()[tok]), rv2 = splat_x2(rv_of(tc.e()[tok]));
      const bool masked = p0 + i * kTok + kTok - 1 > see_all;  // some row does not see some position of the tile
      uint8_t* P = sm + L::oP + pb * L::kP + tok * 128;
      const uint32_t S = tmem + lanes + L::cS + sb * (L::kParts * N);
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
        uint32_t r[16];
        tmem_ld16(S + c, r);
        tmem_wait16(r);
        if (L::kParts == 2) {
          uint32_t r2[16];
          tmem_ld16(S + N + c, r2);
          tmem_wait16(r2);
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(r2[j]));
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(qscale + c + 2 * j);
          x[j] = fma2(pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), mul2(phi2, f.x), x[j]);
          x[j + 1] = fma2(pack2(__uint_as_float(r[2 * j + 2]), __uint_as_float(r[2 * j + 3])), mul2(phi2, f.y), x[j + 1]);
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
            t[j] = ex2z(t[j]);
            t[j + 1] = ex2z(t[j + 1]);
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
            f = exp2f(M - (mx - kBelow));
            negM[c0 + tok] = kBelow - mx;
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
          for (int j = 0; j < 16; ++j) t[j] = ex2z(t[j]);
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
      mbar_arrive_if(s_empty(sb), lane == 0);
      mbar_arrive_if(p_full(pb), lane == 0);
      mbar_arrive_if(c_empty(cb), lane == 0);
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
  } else if (warp < kSoftWarps + 8) {
    Share x{&a, u, T, p0, p1, nt, sm, base, k_full(0), k_empty(0), v_full(0), v_empty(0),
            c_full(0), c_empty(0), L::oK, L::oV, L::oRawK, L::oRawV, L::oConst, L::oRank};
    const int tok = threadIdx.x - kSoftWarps * 32;
    const bool ok = warp < kSoftWarps + 4 ? (g.lm ? expand_k<DG, L::KU, L::CB, L::kStages, 8, true, false>(x, tok, lane) : expand_k<DG, L::KU, L::CB, L::kStages, 8, false, false>(x, tok, lane))
                                          : (g.lm ? expand_v<DG, L::VU, L::CB, L::kStages, 8, true, false>(x, warp & 3, lane) : expand_v<DG, L::VU, L::CB, L::kStages, 8, false, false>(x, warp & 3, lane));
    cp_async_wait<0>();  // also where a wait ran out
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------ MMA issuer --------------------------------
    // One warp issues every product; its instructions, not the tensor cores, would be the kernel's bound if it computed
    // buffer indices and looked at the outcome of every wait.
    const uint32_t leader = elect_one();
    constexpr uint32_t id_qk = idesc_of(N, false, false), id_pv = idesc_of(N, true, true);
    const uint32_t dQ = desc_of(base + L::oQ, 16), dK = desc_of(base + L::oK, 16), dV = desc_of(base + L::oV, kUnit / 2),
                   dP = desc_of(base + L::oP, kTok * 128), dRank = rank_desc(base + L::oRank);
    Waits waits{a.wait_turns};
    Ring<L::KU> kr;
    Ring<L::VU> vr;
    Ring<L::SB> sr;
    Ring<L::PB> pr;
    uint32_t odd = 0;  // the tile's rank-one operand
    auto product_qk = [&](bool reuse) {
      if (reuse) waits.on(s_empty(sr.at), sr.phase ^ 1);
      const uint32_t d = L::cS + sr.at * (L::kParts * N);
#pragma unroll 1
      for (int kb = 0; kb < 2 * DG; ++kb) {
        waits.on(k_full(kr.at), kr.phase);
        fence_after();
        const uint32_t k = dK + kr.at * (kUnit >> 4), q = dQ + kb * (N * 128 >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // Q's high, then its low part; descriptors count 16 bytes
          // two accumulators: the high parts of the first half of the channels in one, of the rest in the other
          const uint32_t at = L::kParts == 2 && (j < 4) == (kb >= DG) ? d + N : d;
          mma_f16_ss(at, k + 2 * (j & 3), q + (j >> 2) * (L::kQ >> 4) + 2 * (j & 3), id_qk,
                     (L::kParts == 2 ? j & 3 : j) ? 1 : kb, leader);
        }
        if (kb == 2 * DG - 2)  // the middles of all groups are there
          mma_f16_ss<kDescRank>(d, dRank + odd * (kRank >> 4), dRank + (2 * kRank >> 4), id_qk, 1, leader);
        mma_commit(k_empty(kr.at), leader);
        kr.next();
        if (g.lm) {
          waits.on(k_full(kr.at), kr.phase);
          fence_after();
          const uint32_t x = dK + kr.at * (kUnit >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_f16_ss(L::kParts == 2 && kb < DG ? d + N : d, x + 2 * j, q + 2 * j, id_qk, 1, leader);
          mma_commit(k_empty(kr.at), leader);
          kr.next();
        }
      }
      mma_commit(s_full(sr.at), leader);
      sr.next();
      odd ^= 1;
    };
    auto product_pv = [&](uint32_t acc) {
      waits.on(p_full(pr.at), pr.phase);
      const uint32_t p = dP + pr.at * (L::kP >> 4);
#pragma unroll 1
      for (int k = 0; k < 2 * DG; ++k) {  // group k / 2, token half k % 2
        waits.on(v_full(vr.at), vr.phase);
        fence_after();
        const uint32_t v = dV + vr.at * (kUnit >> 4), half = k & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16_ss(L::cO + (k >> 1) * N, v + 128 * j, p + half * 512 + 128 * j, id_pv, j ? 1 : acc | half, leader);
        mma_commit(v_empty(vr.at), leader);
        vr.next();
      }
      mma_commit(p_empty(pr.at), leader);
      pr.next();
    };
    waits.on(q_full, 0);
    waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
    fence_after();
    if (__all_sync(0xffffffffu, waits.ok)) product_qk(false);
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      if (!__all_sync(0xffffffffu, waits.ok)) break;
      if (i + 1 < nt) product_qk(i + 1 >= L::SB);
      product_pv(i > 0);
    }
    const bool ok = __all_sync(0xffffffffu, waits.ok);
    if (!ok && lane == 0) fail();
    mma_commit(drained, leader);  // every product issued is complete before TMEM is freed
    mbar_wait(drained, 0);
    __syncwarp();
  }
  if (a.beside) pdl_wait();
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
  return row_launch(true, attn_rows_tc_kernel<DG, N>, dim3(unsigned(items)), kThreads, Plan<DG, N>::kBytes, stream, a);
}

// Query rows per CTA: the least of 32, 64 (D > 128) or 128 that holds a unit's rows, because a CTA with more columns costs
// little more and the keys are expanded once.  D = 128 with more than 32 rows goes to the row-lane kernel; us a call here
// with 64 rows a CTA and there: 8 sequences x 9 / 12 / 16 tokens x 4 heads a KV head (36 / 48 / 64 rows) over 4096 positions
// 71 / 83 / 87 and 61 / 69 / 75, 512 rows on one prefix of 131,072 positions 808 and 450.  32 rows: 62 here, 69 with 64.
int tile_rows(int D, int64_t rows) {
  if (rows <= 32) return 32;
  return D > 128 ? 64 : 128;
}

}  // namespace

int rows_splits_tc(const Geom& g, int64_t rows, int seq_len_hint) {
  const int N = tile_rows(g.D, rows);
  const int64_t items = (rows + N - 1) / N * g.B * g.Hkv;
  const int64_t blocks = (int64_t(seq_len_hint) + kTok - 1) / kTok;
  // Time of ns splits: waves of CTAs on 152 SMs (written in, because the workspace query gives the same answer without a
  // device and results do not depend on the one that runs them), each its tiles and a fixed part worth `fixed` tiles (queries, set-up, the
  // first tile's latency, the merge).  With 3 in place of 6, 64 sequences on one prefix took 512 us, with 6 or 10 490 us;
  // the other sizes measured did not change.
  const double fixed = 6.0;
  auto time = [&](int ns) {
    return double((items * ns + 151) / 152) * (fixed + double((blocks + ns - 1) / ns));
  };
  const int most = int(std::max<int64_t>(1, std::min<int64_t>(OSCAR_KV_MAX_SPLITS, blocks)));
  int best = 1;
  for (int ns = 2; ns <= most; ++ns)
    if (time(ns) < time(best) * 0.98) best = ns;
  // Sequences of a batch differ in length, and shorter shares even that out: the most of them that cost at most a tenth
  // more on equal lengths.  5 tokens for each of 8 sequences of up to 16,384: 2 / 4 / 7 / 9 / 14 shares 176 / 159 / 150 /
  // 149 / 166 us.
  if (g.B > 1) {
    const double limit = time(best) * 1.1;
    for (int ns = best + 1; ns <= most; ++ns)
      if (time(ns) <= limit) best = ns;
  }
  return best;
}

int launch_attn_rows_tc(const RowsArgs& a, cudaStream_t stream) {
  const int N = tile_rows(a.g.D, int64_t(a.n) * a.g.G);
  if (N == 128) return launch_attn_rows_lanes(a, stream);
  if (a.g.D == 128) return launch<1, 32>(a, stream);
  if (a.g.D == 256) return N == 32 ? launch<2, 32>(a, stream) : launch<2, 64>(a, stream);
  return N == 32 ? launch<4, 32>(a, stream) : launch<4, 64>(a, stream);
}

}  // namespace oscar
