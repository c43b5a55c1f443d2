// attn_mass: the attention weight that every cached position receives.
//
//   mass_out[p] = mass_in[p] + sum over query rows r that see p of exp(scale q_r . k_p - lse_r)
//
// for each (sequence, KV head), over the K role of the cache alone.  In the
// rotated basis and log2 units an INT2 key gives
//   s = scale_p (q' . c_p) + zero_p sum(q')   per group of 128 channels.
//
// A decode step's rows are few, and the bytes of K bound it (36 per position at
// head_dim 128, and 8 of the masses); so keys go from global memory to registers
// to mma.sync m16n8k16, positions on M, and nothing but the sum over rows is
// written.  A warp takes 32 positions at a time, with the next ones' loads in
// flight: a lane's two code words of a row are exactly its A fragments of the
// group (the header's K layout), unpacked by a shift and an AND each into fp16
// subnormals, code * 2^-16, at the top of the mantissa, where the products lose
// nothing (common.cuh).  The columns are four query rows' high and low fp16 parts,
// 22 bits in all, scaled by a power of two per row; a lane then has its row's
// whole score in two accumulators, and the rows' sum is two shuffles.
// BF16 rows take the same path with three bf16 parts; a lane's 16-byte pieces
// of a row are its fragments, channels in an order of their own.
//
// Blocks of query rows (up to 16) follow each other over a block's positions, the
// masses of which stay in shared memory.
#include <algorithm>

#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kBatch = 32;          // positions of a warp's turn
constexpr int kMostChunk = 4096;    // positions of a block

// The codes at bits 2 p and 16 + 2 p of a word as fp16 values code * 2^-16.
template <uint32_t mask>
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&r)[8]) {
#pragma unroll
  for (int p = 0; p < 8; ++p) r[p] = (p < 4 ? w << (8 - 2 * p) : w >> (2 * p - 8)) & mask;
}

template <int D, int NB>
struct Mass {
  static constexpr int Dg = D / kGroup, KS = D / 16, R = 4 * NB;  // groups, k steps, rows of a block
  static constexpr int o16 = 0;                       // fp16 fragments [NB][KS][32] x 8 bytes
  static constexpr int oBf = o16 + NB * KS * 32 * 8;  // bf16 fragments [NB][2][KS][32] x 8 bytes
  static constexpr int oSum = oBf + 2 * NB * KS * 32 * 8;  // [R][Dg] sums of the row
  static constexpr int oRow = oSum + R * Dg * 4;      // [R] factor, reference (high, low), last position
  static constexpr int oMass = oRow + R * 16;
  static constexpr int kBytes = oMass + kMostChunk * 4;
};

// Blocks on an SM at least, for the registers.
template <int D, int NB>
constexpr int resident() { return NB == 4 || D == 512 ? 2 : D == 256 ? 3 : NB == 1 ? 5 : 4; }

template <int D, int NB, bool LM>
__global__ void __launch_bounds__(kThreads, (resident<D, NB>())) attn_mass_kernel(const MassArgs a) {
  using C = Mass<D, NB>;
  constexpr int Dg = C::Dg, KS = C::KS, R = C::R;
  extern __shared__ __align__(16) uint8_t sm[];
  uint2* f16 = reinterpret_cast<uint2*>(sm + C::o16);
  uint2* fbf = reinterpret_cast<uint2*>(sm + C::oBf);
  float* qsum = reinterpret_cast<float*>(sm + C::oSum);
  float4* rowc = reinterpret_cast<float4*>(sm + C::oRow);
  float* mass = reinterpret_cast<float*>(sm + C::oMass);
  const Geom& g = a.g;
  const int unit = blockIdx.y, b = unit / g.Hkv, h = unit % g.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row8 = lane >> 2, col = lane & 3;
  const int given = a.seq_lens[b], T = max(0, min(given, g.cap));
  if (given > g.cap && blockIdx.x == 0 && threadIdx.x == 0) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
  const int ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n), rows = ql * g.G;
  const int window = max(g.S, T - g.W);  // the ring's first position
  const uint8_t* base = a.layer_base;
  const uint8_t* codes = base + g.sink_bytes + g.ring_bytes + int64_t(unit) * g.ncap * (D / 4);
  const uint8_t* sz = base + g.sink_bytes + g.ring_bytes + g.codes_bytes + int64_t(unit) * g.ncap * (Dg * 4);
  const uint8_t* sink = base + int64_t(unit) * g.S * (2 * D);
  const uint8_t* ring = base + g.sink_bytes + int64_t(unit) * g.W * (2 * D);
  pdl_wait();  // the rotated queries

  for (int64_t c0 = int64_t(blockIdx.x) * a.chunk; c0 < T; c0 += int64_t(gridDim.x) * a.chunk) {
    const int p0 = int(c0), p1 = min(T, p0 + a.chunk);
    const int i0 = max(p0, g.S), i1 = min(p1, window);        // INT2 positions
    const bool wide = p0 < min(g.S, T) || p1 > window;
    for (int i = threadIdx.x; i < p1 - p0; i += kThreads) mass[i] = 0.f;
    struct Batch {
      uint2 words[Dg][4];
      uint32_t sz[Dg][4];
    };
    const uint8_t* my_codes = codes + 8 * col;
    auto load = [&](Batch& x, int p) {
      const int at = p + row8 - g.S;
      if (p + kBatch <= i1) {  // positions 8 apart are constants apart
        const uint8_t *c = my_codes + int64_t(at) * (D / 4), *z = sz + int64_t(at) * (Dg * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < Dg; ++j) {
            x.words[j][i] = __ldg(reinterpret_cast<const uint2*>(c + i * 8 * (D / 4) + 32 * j));
            x.sz[j][i] = __ldg(reinterpret_cast<const uint32_t*>(z + i * 8 * (Dg * 4) + 4 * j));
          }
      } else if (p < i1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t last = min(at + 8 * i, i1 - 1 - g.S);
#pragma unroll
          for (int j = 0; j < Dg; ++j) {
            x.words[j][i] = __ldg(reinterpret_cast<const uint2*>(my_codes + last * (D / 4) + 32 * j));
            x.sz[j][i] = __ldg(reinterpret_cast<const uint32_t*>(sz + last * (Dg * 4) + 4 * j));
          }
        }
      }
    };
    constexpr int kStep = kBatch * kWarps;
    constexpr bool kAhead = D == 128 && NB < 4;  // two batches under way where the registers allow
    for (int r0 = 0; r0 < rows; r0 += R) {
      int p = i0 + kBatch * warp;
      Batch x0, x1;
      load(x0, p);
      if (kAhead) load(x1, p + kStep);
      // ----------------- the rows' fragments, factors and references ------------------
      __syncthreads();
      for (int r = warp; r < R; r += kWarps) {
        const int row = r0 + r;
        const bool on = row < rows;
        const int64_t at = int64_t(b * a.n + row / g.G) * g.Hq + h * g.G + row % g.G;
        const float* q = a.qrot + (on ? at : 0) * D;
        uint32_t most = 0;
        float v[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          v[i] = on ? q[lane + 32 * i] : 0.f;
          if (isfinite(v[i])) most = max(most, __float_as_uint(fabsf(v[i])));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        // the largest finite component lands in [2^14, 2^15)
        const int e = max(-100, (int(most) >> 23) - 126 - 15);
        const float up = pow2i(min(126, -e));
        float sums[Dg];
#pragma unroll
        for (int j = 0; j < Dg; ++j) sums[j] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int ch = lane + 32 * i;
          // fp16 parts: group j = ch / 128, k step (ch % 128) / 16 of it, the fragment's half and lane by ch % 16
          const float x = v[i] * up;
          const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
          sums[i / 4] += __half2float(hi) + __half2float(lo);
          const int k = ch & 15, c = (k & 7) >> 1, reg = k >> 3, part = k & 1;
          __half* f = reinterpret_cast<__half*>(f16 + ((r >> 2) * KS + (ch >> 4)) * 32 + (2 * (r & 3)) * 4 + c);
          f[2 * reg + part] = hi;
          f[16 + 2 * reg + part] = lo;  // the next column: four lanes on
          if (wide) {
            uint32_t w[3];
            split3_bf16(v[i], w);
            // piece ch / 8 = col + 4 m: registers x, y are step 2 m, z, w step 2 m + 1
            const int piece = ch >> 3, cc = piece & 3, m = piece >> 2, in = ch & 7;
            const int step = 2 * m + (in >> 2), rg = (in >> 1) & 1;
            uint16_t* s0 = reinterpret_cast<uint16_t*>(fbf + (((r >> 2) * 2) * KS + step) * 32 + (2 * (r & 3)) * 4 + cc);
            uint16_t* s1 = reinterpret_cast<uint16_t*>(fbf + (((r >> 2) * 2 + 1) * KS + step) * 32 + (2 * (r & 3)) * 4 + cc);
            s0[2 * rg + (in & 1)] = uint16_t(w[0]);
            s0[16 + 2 * rg + (in & 1)] = uint16_t(w[1]);
            s1[2 * rg + (in & 1)] = uint16_t(w[2]);
            s1[16 + 2 * rg + (in & 1)] = 0;
          }
        }
#pragma unroll
        for (int j = 0; j < Dg; ++j) {
#pragma unroll
          for (int o = 16; o; o >>= 1) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
          if (lane == 0) qsum[r * Dg + j] = sums[j] * pow2i(max(-126, e));
        }
        if (lane == 0) {
          const float x = on ? a.lse[at] : -INFINITY;
          float hi = x * 1.4426950408889634f;
          // the product's rounding and what the constant leaves out
          float lo = fmaf(x, 1.4426950408889634f, -hi) + x * 1.9259629911266175e-8f;
          if (!isfinite(hi)) hi = x == -INFINITY ? INFINITY : hi, lo = 0.f;  // a row without weight
          rowc[r] = make_float4(pow2i(min(127, max(-126, e + 16))), hi, lo, __int_as_float(on ? T - ql + row / g.G : -1));
        }
      }
      __syncthreads();
      float fac[NB], ref[NB], ref2[NB], sums[NB][Dg];
      int last[NB];
#pragma unroll
      for (int t = 0; t < NB; ++t) {
        const float4 x = rowc[4 * t + col];
        fac[t] = x.x, ref[t] = x.y, ref2[t] = x.z, last[t] = __float_as_int(x.w);
#pragma unroll
        for (int j = 0; j < Dg; ++j) sums[t][j] = qsum[(4 * t + col) * Dg + j];
      }
      const int seen = T - ql;  // every row sees the positions up to this one
      // scores of four positions (0, 8, 16, 24 and row8 on) against this lane's rows: their weights, summed over the rows
      auto weigh = [&](const float (&s)[NB][4], int p, int end) {
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = ex2z((s[t][i] - ref[t]) - ref2[t]);
            w[i] += p + 8 * i + row8 <= max(seen, last[t]) ? x : 0.f;
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
          w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
        }
        // column i of the quad writes position 8 i + row8
        const float x = col == 0 ? w[0] : col == 1 ? w[1] : col == 2 ? w[2] : w[3];
        const int at = p + 8 * col + row8;
        if (at < end) mass[at - p0] += x;
      };

      // ------------------------------- INT2 rows --------------------------------------
      auto take = [&](const Batch& now, int p) {
        float s[NB][4];
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
        for (int j = 0; j < Dg; ++j) {
          float acc[NB][2][4], high[NB][2][4];
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[t][m][i] = 0.f, high[t][m][i] = 0.f;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int level = 0; level < (LM ? 2 : 1); ++level) {
              uint32_t r[4][8];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t w = i ? now.words[j][x].y : now.words[j][x].x;
                if (level) codes_of<0x02000200u>(w, r[x]);
                else codes_of<0x03000300u>(w, r[x]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                  const uint2 f = f16[(t * KS + 8 * j + 4 * i + k) * 32 + lane];
                  mma_f16(level ? high[t][0] : acc[t][0], r[0][2 * k], r[1][2 * k], r[0][2 * k + 1], r[1][2 * k + 1], f.x, f.y);
                  mma_f16(level ? high[t][1] : acc[t][1], r[2][2 * k], r[3][2 * k], r[2][2 * k + 1], r[3][2 * k + 1], f.x, f.y);
                }
            }
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&now.sz[j][x]));
#pragma unroll
            for (int t = 0; t < NB; ++t) {
              float dot = acc[t][x >> 1][2 * (x & 1)] + acc[t][x >> 1][2 * (x & 1) + 1];
              if (LM) dot = fmaf(kLmRho, dot, kLmHi * (high[t][x >> 1][2 * (x & 1)] + high[t][x >> 1][2 * (x & 1) + 1]));
              s[t][x] = fmaf(z.x * fac[t], dot, fmaf(z.y, sums[t][j], s[t][x]));
            }
          }
        }
        weigh(s, p, i1);
      };
#pragma unroll 1
      while (p < i1) {
        if (kAhead) {
          take(x0, p);
          load(x0, p + 2 * kStep);
          p += kStep;
          if (p >= i1) break;
          take(x1, p);
          load(x1, p + 2 * kStep);
        } else {
          x1 = x0;
          load(x0, p + kStep);
          take(x1, p);
        }
        p += kStep;
      }

      // ------------------------------- BF16 rows --------------------------------------
      if (wide) {
        auto region = [&](int from, int to, bool is_ring) {
          for (int q = from + kBatch * warp; q < to; q += kBatch * kWarps) {
            const uint4* src[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = min(q + 8 * i + row8, to - 1);
              src[i] = reinterpret_cast<const uint4*>(is_ring ? ring + int64_t(at % g.W) * (2 * D) : sink + int64_t(at) * (2 * D)) + col;
            }
            float acc[NB][2][2][4];
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[t][0][m][i] = 0.f, acc[t][1][m][i] = 0.f;
#pragma unroll 2
            for (int m = 0; m < D / 32; ++m) {
              uint4 x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i] = __ldg(src[i] + 4 * m);
#pragma unroll
              for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                  const uint2 f = fbf[((2 * t + part) * KS + 2 * m) * 32 + lane], f1 = fbf[((2 * t + part) * KS + 2 * m + 1) * 32 + lane];
                  mma_bf16(acc[t][part][0], x[0].x, x[1].x, x[0].y, x[1].y, f.x, f.y);
                  mma_bf16(acc[t][part][0], x[0].z, x[1].z, x[0].w, x[1].w, f1.x, f1.y);
                  mma_bf16(acc[t][part][1], x[2].x, x[3].x, x[2].y, x[3].y, f.x, f.y);
                  mma_bf16(acc[t][part][1], x[2].z, x[3].z, x[2].w, x[3].w, f1.x, f1.y);
                }
            }
            float s[NB][4];
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[t][i] = (acc[t][0][i >> 1][2 * (i & 1)] + acc[t][0][i >> 1][2 * (i & 1) + 1]) + acc[t][1][i >> 1][2 * (i & 1)];
            weigh(s, q, to);
          }
        };
        region(p0, min(p1, min(g.S, T)), false);
        region(max(p0, window), p1, true);
      }
    }
    __syncthreads();
    const int64_t to = int64_t(unit) * g.cap + p0;
    for (int i = threadIdx.x; i < p1 - p0; i += kThreads) a.mass_out[to + i] = mass[i] + (a.mass_in ? a.mass_in[to + i] : 0.f);
    __syncthreads();
  }
}

template <int D, int NB, bool LM>
int launch_l(const MassArgs& a, dim3 grid, cudaStream_t stream) {
  constexpr int smem = Mass<D, NB>::kBytes;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_mass_kernel<D, NB, LM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  return row_launch(a.n > 0, attn_mass_kernel<D, NB, LM>, grid, kThreads, smem, stream, a);
}
template <int D, int NB>
int launch_n(const MassArgs& a, dim3 grid, cudaStream_t stream) {
  return a.g.lm ? launch_l<D, NB, true>(a, grid, stream) : launch_l<D, NB, false>(a, grid, stream);
}
template <int D>
int launch_d(const MassArgs& a, dim3 grid, cudaStream_t stream) {
  const int64_t rows = int64_t(a.n) * a.g.G;
  return rows <= 4 ? launch_n<D, 1>(a, grid, stream) : rows <= 8 ? launch_n<D, 2>(a, grid, stream) : launch_n<D, 4>(a, grid, stream);
}

}  // namespace

int launch_attn_mass(const MassArgs& args, cudaStream_t stream) {
  MassArgs a = args;
  const int64_t units = int64_t(a.g.B) * a.g.Hkv;
  int dev = 0, sms = 0;
  if (units > 65535 || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_LAUNCH;
  // positions of a block: enough blocks for every SM to have eight, no more than its masses' shared memory holds
  const int64_t even = (int64_t(a.top) * units + 8 * sms - 1) / (8 * sms);
  a.chunk = int(std::min<int64_t>(kMostChunk, std::max<int64_t>(kBatch * kWarps, (even + 127) / 128 * 128)));
  const dim3 grid(unsigned((a.top + a.chunk - 1) / a.chunk), unsigned(units));
  switch (a.g.D) {
    case 128: return launch_d<128>(a, grid, stream);
    case 256: return launch_d<256>(a, grid, stream);
    default: return launch_d<512>(a, grid, stream);
  }
}

}  // namespace oscar
