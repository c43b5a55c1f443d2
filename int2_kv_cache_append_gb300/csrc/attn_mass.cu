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
// written.  A warp works for itself, without shared memory: 32 positions at a
// time, the next ones' loads under way.  A lane's two code words of a row are
// exactly its A fragments of the group (the header's K layout), unpacked by a
// shift and an AND each into fp16 subnormals, code * 2^-16, at the top of the
// mantissa, where the products lose nothing (common.cuh).  The columns are four
// query rows' high and low fp16 parts, 22 bits in all, scaled by a power of two
// per row; a lane then has its row's whole score in two accumulators, and the sum
// over the rows is two shuffles.  BF16 rows take the same path with three bf16
// parts; a lane's 16-byte pieces of a row are its fragments, channels in an order
// of their own.
//
// What bounds it: instructions, about 300 a batch of 32 positions, over half of them
// the codes' unpacking and the products (32 ragged sequences of up to 32K, 8 KV heads
// of 4 rows: 103 us, 2.5 TB/s of K and masses); with many rows of head_dim 256 or 512 the
// mma.sync pipe and its latency.  Many rows of head_dim 128: attn_mass_tc.cu.
//
// The rows' fragments are written once by a kernel of their own behind the query
// rotation: built by every block they cost as much as the positions themselves.
#include <algorithm>

#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kBatch = 32;          // positions of a warp's turn
constexpr int kMostPiece = 256;     // positions of a warp

// The codes at bits 2 p and 16 + 2 p of a word as fp16 values: code * 2^-16 for odd p, whose shift to the top of the
// mantissa leaves the even one below it, code * 2^-18.  (A shift for each would cost a quarter more of what the kernel has
// most of, logic instructions.)  The query's fragments are four times larger there.  bits: 3, or 2 for the high bit alone.
template <uint32_t bits>
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&r)[8]) {
#pragma unroll
  for (int p = 0; p < 8; p += 2) {
    const uint32_t x = p < 4 ? w << (6 - 2 * p) : w >> (2 * p - 6);
    r[p] = x & (bits * 0x00400040u);
    r[p + 1] = x & (bits * 0x01000100u);
  }
}

// What the fragment kernel leaves, per (sequence, KV head), for tiles of four rows: fp16 fragments [tiles][D / 16][32] and
// bf16 fragments [tiles][2][D / 16][32] of 8 bytes; per row (factor, reference high and low, last position) and the sums of
// its groups [D / 128].
struct Frags {
  uint2 *f16, *fbf;
  float4* row;
  float* sum;
};
template <int D>
__host__ __device__ inline Frags frags_of(const MassArgs& a, int64_t unit) {
  const int64_t units = int64_t(a.g.B) * a.g.Hkv, piece = int64_t(a.tiles) * (D / 16) * 32;
  uint8_t* at = a.frags;
  Frags f;
  f.f16 = reinterpret_cast<uint2*>(at) + unit * piece;
  at += units * piece * 8;
  f.fbf = reinterpret_cast<uint2*>(at) + unit * piece * 2;
  at += units * piece * 16;
  f.row = reinterpret_cast<float4*>(at) + unit * a.tiles * 4;
  at += units * a.tiles * 64;
  f.sum = reinterpret_cast<float*>(at) + unit * a.tiles * 4 * (D / kGroup);
  return f;
}

template <int D>
__global__ void __launch_bounds__(kThreads) mass_frags_kernel(const MassArgs a) {
  constexpr int Dg = D / kGroup, KS = D / 16;
  const Geom& g = a.g;
  const int lane = threadIdx.x & 31;
  const int64_t at_row = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5), units = int64_t(g.B) * g.Hkv;
  const int64_t unit = at_row / (4 * a.tiles);
  pdl_wait();  // the rotated queries
  if (unit >= units) return;
  const int row = int(at_row - unit * 4 * a.tiles), b = int(unit / g.Hkv), h = int(unit % g.Hkv);
  const int T = max(0, min(a.seq_lens[b], g.cap)), ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n);
  const bool on = row < ql * g.G;
  const Frags f = frags_of<D>(a, unit);
  const int64_t at = (int64_t(b) * a.n + row / g.G) * g.Hq + h * g.G + row % g.G;
  const float* q = a.qrot + (on ? at : 0) * D;
  const float lse = on ? a.lse[at] : -INFINITY;
  const bool weighs = lse != -INFINITY;  // else the query may be anything
  uint32_t most = 0;
  float v[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    v[i] = weighs ? q[lane + 32 * i] : 0.f;
    if (isfinite(v[i])) most = max(most, __float_as_uint(fabsf(v[i])));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  // the largest finite component lands in [2^12, 2^13)
  const int e = max(-100, (int(most) >> 23) - 126 - 13);
  const float up = pow2i(min(126, -e));
  const int tile = row >> 2, lead = (2 * (row & 3)) * 4;  // the first lane of the row's column
  float sums[Dg];
#pragma unroll
  for (int j = 0; j < Dg; ++j) sums[j] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int ch = lane + 32 * i;
    // fp16 parts: k step ch / 16, the fragment's register and lane by ch % 16
    const int k = ch & 15, c = (k & 7) >> 1, in = 2 * (k >> 3) + (k & 1);
    const float x = v[i] * up * (k < 8 ? 4.f : 1.f);
    const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
    sums[i / 4] += (__half2float(hi) + __half2float(lo)) * (k < 8 ? 0.25f : 1.f);
    __half* to = reinterpret_cast<__half*>(f.f16 + (int64_t(tile) * KS + (ch >> 4)) * 32 + lead + c);
    to[in] = hi;
    to[16 + in] = lo;  // the next column: four lanes on
    uint32_t w[3];
    split3_bf16(v[i], w);
    // piece ch / 8 = c + 4 m: registers x, y are step 2 m, z, w step 2 m + 1
    const int piece = ch >> 3, cc = piece & 3, step = 2 * (piece >> 2) + ((ch & 7) >> 2), at2 = ch & 3;
    uint16_t* s0 = reinterpret_cast<uint16_t*>(f.fbf + (int64_t(tile) * 2 * KS + step) * 32 + lead + cc);
    uint16_t* s1 = s0 + KS * 32 * 4;
    s0[at2] = uint16_t(w[0]);
    s0[16 + at2] = uint16_t(w[1]);
    s1[at2] = uint16_t(w[2]);
    s1[16 + at2] = 0;
  }
#pragma unroll
  for (int j = 0; j < Dg; ++j) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sums[j] += __shfl_xor_sync(0xffffffffu, sums[j], o);
    if (lane == 0) f.sum[row * Dg + j] = sums[j] * pow2i(max(-126, e));
  }
  if (lane == 0) {
    float hi = lse * 1.4426950408889634f;
    // the product's rounding and what the constant leaves out
    float lo = fmaf(lse, 1.4426950408889634f, -hi) + lse * 1.9259629911266175e-8f;
    if (!isfinite(hi)) hi = weighs ? hi : INFINITY, lo = 0.f;
    f.row[row] = make_float4(pow2i(min(127, max(-126, e + 16))), hi, lo, __int_as_float(on ? T - ql + row / g.G : -1));
  }
}

// Blocks on an SM at least, for the registers.
template <int D, int NB>
constexpr int resident() { return D == 128 ? (NB == 1 ? 4 : 3) : 2; }

// NB tiles of four rows at a time; ONE: there are no more.
template <int D, int NB, bool LM, bool ONE>
__global__ void __launch_bounds__(kThreads, (resident<D, NB>())) attn_mass_kernel(const MassArgs a) {
  constexpr int Dg = D / kGroup, KS = D / 16;
  constexpr bool kHold = ONE && NB * KS <= 16;  // the fragments stay in registers
  constexpr bool kAhead = D == 128;             // as does a second batch; of longer rows one is enough under way
  const Geom& g = a.g;
  const int unit = blockIdx.y, b = unit / g.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row8 = lane >> 2, col = lane & 3;
  const int given = a.seq_lens[b], T = max(0, min(given, g.cap));
  if (given > g.cap && blockIdx.x == 0 && threadIdx.x == 0) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
  const int ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n), tiles = (ql * g.G + 3) / 4;
  const int seen = T - ql;                // every row sees the positions up to this one
  const int window = max(g.S, T - g.W);   // the ring's first position
  const uint8_t* base = a.layer_base;
  const uint8_t* codes = base + g.sink_bytes + g.ring_bytes + int64_t(unit) * g.ncap * (D / 4) + 8 * col;
  const uint8_t* sz = base + g.sink_bytes + g.ring_bytes + g.codes_bytes + int64_t(unit) * g.ncap * (Dg * 4);
  const uint8_t* sink = base + int64_t(unit) * g.S * (2 * D);
  const uint8_t* ring = base + g.sink_bytes + int64_t(unit) * g.W * (2 * D);
  const Frags f = frags_of<D>(a, unit);
  const float* mass_in = a.mass_in ? a.mass_in + int64_t(unit) * g.cap : nullptr;
  float* mass_out = a.mass_out + int64_t(unit) * g.cap;

  struct Batch {
    uint2 words[Dg][4];
    uint32_t sz[Dg][4];
    float mass;  // of the position that this lane writes
  };
  // INT2 positions p + row8 + 8 i below end
  auto load = [&](Batch& x, int p, int end) {
    const int at = p + row8 - g.S;
    if (p + kBatch <= end) {  // positions 8 apart are constants apart
      const uint8_t *c = codes + int64_t(at) * (D / 4), *z = sz + int64_t(at) * (Dg * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < Dg; ++j) {
          x.words[j][i] = __ldg(reinterpret_cast<const uint2*>(c + i * 8 * (D / 4) + 32 * j));
          x.sz[j][i] = __ldg(reinterpret_cast<const uint32_t*>(z + i * 8 * (Dg * 4) + 4 * j));
        }
    } else if (p < end) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t last = min(at + 8 * i, end - 1 - g.S);
#pragma unroll
        for (int j = 0; j < Dg; ++j) {
          x.words[j][i] = __ldg(reinterpret_cast<const uint2*>(codes + last * (D / 4) + 32 * j));
          x.sz[j][i] = __ldg(reinterpret_cast<const uint32_t*>(sz + last * (Dg * 4) + 4 * j));
        }
      }
    }
    x.mass = mass_in && p + 8 * col + row8 < end ? mass_in[p + 8 * col + row8] : 0.f;
  };
  struct Rows {  // this lane's row of each tile
    float fac[NB], ref[NB], ref2[NB], sum[NB][Dg];
    int last[NB];
  };
  auto rows_of = [&](Rows& r, int t0) {
#pragma unroll
    for (int t = 0; t < NB; ++t) {
      const int row = 4 * min(t0 + t, tiles - 1) + col;
      const float4 x = f.row[row];
      r.fac[t] = x.x, r.ref[t] = t0 + t < tiles ? x.y : INFINITY, r.ref2[t] = x.z, r.last[t] = __float_as_int(x.w);
#pragma unroll
      for (int j = 0; j < Dg; ++j) r.sum[t][j] = f.sum[row * Dg + j];
    }
  };
  // scores of four positions (0, 8, 16, 24 and row8 on) against this lane's rows: their weights
  auto weigh = [&](const Rows& r, const float (&s)[NB][4], int p, float (&w)[4]) {
    if (p + kBatch - 1 <= seen) {
#pragma unroll
      for (int t = 0; t < NB; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] += ex2z((s[t][i] - r.ref[t]) - r.ref2[t]);
      return;
    }
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = ex2z((s[t][i] - r.ref[t]) - r.ref2[t]);
        w[i] += p + 8 * i + row8 <= r.last[t] ? x : 0.f;
      }
  };
  // the rows' sum; column i of the quad writes position 8 i + row8
  auto write = [&](float (&w)[4], int p, int end, float before) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 1);
      w[i] += __shfl_xor_sync(0xffffffffu, w[i], 2);
    }
    const float x = col == 0 ? w[0] : col == 1 ? w[1] : col == 2 ? w[2] : w[3];
    const int at = p + 8 * col + row8;
    if (at < end) mass_out[at] = x + before;
  };

  const int64_t first = (int64_t(blockIdx.x) * kWarps + warp) * a.piece;
  Batch x0;
  if (kAhead && first < T) load(x0, max(int(first), g.S), min(min(T, int(first) + a.piece), window));
  pdl_wait();  // the fragments; every block, also one without positions
  Rows held;
  uint2 frag[kHold ? NB : 1][kHold ? KS : 1];
  if (ONE && first < T && tiles) {
    rows_of(held, 0);
    if (kHold) {
#pragma unroll
      for (int t = 0; t < NB; ++t)
#pragma unroll
        for (int k = 0; k < KS; ++k) frag[kHold ? t : 0][kHold ? k : 0] = f.f16[(int64_t(min(t, tiles - 1)) * KS + k) * 32 + lane];
    }
  }

  for (int64_t c0 = first; c0 < T; c0 += int64_t(gridDim.x) * kWarps * a.piece) {
    const int p0 = int(c0), p1 = min(T, p0 + a.piece);
    const int i0 = max(p0, g.S), i1 = min(p1, window);  // INT2 positions
    if (kAhead && c0 != first) load(x0, i0, i1);
#pragma unroll 1
    for (int p = i0; p < i1; p += kBatch) {
      Batch now;
      if (kAhead) {
        now = x0;
        if (p + kBatch < i1) load(x0, p + kBatch, i1);
      } else {
        load(now, p, i1);
      }
      float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int t0 = 0; t0 < (ONE ? min(tiles, 1) : tiles); t0 += NB) {
        if (!ONE) rows_of(held, t0);
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
                uint32_t word = i ? now.words[j][x].y : now.words[j][x].x;
                // unpacked again for every block of rows: all of a batch's codes do not fit the registers
                if (!ONE) asm volatile("" : "+r"(word));
                if (level) codes_of<2>(word, r[x]);
                else codes_of<3>(word, r[x]);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int t = 0; t < NB; ++t) {
                  const int ks = 8 * j + 4 * i + k;
                  const uint2 q = kHold ? frag[kHold ? t : 0][kHold ? ks : 0] : f.f16[(int64_t(min(t0 + t, tiles - 1)) * KS + ks) * 32 + lane];
                  mma_f16(level ? high[t][0] : acc[t][0], r[0][2 * k], r[1][2 * k], r[0][2 * k + 1], r[1][2 * k + 1], q.x, q.y);
                  mma_f16(level ? high[t][1] : acc[t][1], r[2][2 * k], r[3][2 * k], r[2][2 * k + 1], r[3][2 * k + 1], q.x, q.y);
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
              s[t][x] = fmaf(z.x * held.fac[t], dot, fmaf(z.y, held.sum[t][j], s[t][x]));
            }
          }
        }
        weigh(held, s, p, w);
      }
      write(w, p, i1, now.mass);
    }

    // --------------------------------- BF16 rows ----------------------------------------
    auto region = [&](int from, int to, bool is_ring) {
#pragma unroll 1
      for (int p = from; p < to; p += kBatch) {
        const uint4* src[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = min(p + 8 * i + row8, to - 1);
          src[i] = reinterpret_cast<const uint4*>(is_ring ? ring + int64_t(at % g.W) * (2 * D) : sink + int64_t(at) * (2 * D)) + col;
        }
        const float before = mass_in && p + 8 * col + row8 < to ? mass_in[p + 8 * col + row8] : 0.f;
        float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int t0 = 0; t0 < tiles; t0 += NB) {
          if (!ONE) rows_of(held, t0);
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
                const uint2* q = f.fbf + ((2 * int64_t(min(t0 + t, tiles - 1)) + part) * KS + 2 * m) * 32 + lane;
                const uint2 u = q[0], v = q[32];
                mma_bf16(acc[t][part][0], x[0].x, x[1].x, x[0].y, x[1].y, u.x, u.y);
                mma_bf16(acc[t][part][0], x[0].z, x[1].z, x[0].w, x[1].w, v.x, v.y);
                mma_bf16(acc[t][part][1], x[2].x, x[3].x, x[2].y, x[3].y, u.x, u.y);
                mma_bf16(acc[t][part][1], x[2].z, x[3].z, x[2].w, x[3].w, v.x, v.y);
              }
          }
          float s[NB][4];
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[t][i] = (acc[t][0][i >> 1][2 * (i & 1)] + acc[t][0][i >> 1][2 * (i & 1) + 1]) + acc[t][1][i >> 1][2 * (i & 1)];
          weigh(held, s, p, w);
        }
        write(w, p, to, before);
      }
    };
    region(p0, min(p1, min(g.S, T)), false);
    region(max(p0, window), p1, true);
  }
}

template <int D, int NB, bool LM, bool ONE>
int launch_one(const MassArgs& a, cudaStream_t stream) {
  const int64_t rows = int64_t(a.g.B) * a.g.Hkv * a.tiles * 4;
  if (rows > 0) {
    const int rc = row_launch(true, mass_frags_kernel<D>, dim3(unsigned((rows + kWarps - 1) / kWarps)), kThreads, 0, stream, a);
    if (rc != OSCAR_OK) return rc;
  }
  const int64_t block = int64_t(kWarps) * a.piece;
  const dim3 grid(unsigned((a.top + block - 1) / block), unsigned(a.g.B * a.g.Hkv));
  return row_launch(rows > 0, attn_mass_kernel<D, NB, LM, ONE>, grid, kThreads, 0, stream, a);
}
template <int D, int NB, bool ONE>
int launch_n(const MassArgs& a, cudaStream_t stream) {
  return a.g.lm ? launch_one<D, NB, true, ONE>(a, stream) : launch_one<D, NB, false, ONE>(a, stream);
}
template <int D>
int launch_d(const MassArgs& a, cudaStream_t stream) {
  // One or two tiles of rows: their fragments stay in registers.  Against the form for more, 4 rows of each of 64 units over
  // 32,768 positions 51 us instead of 116, 8 rows of 64 units over 16,384 38 us instead of 57.
  return a.tiles <= 1 ? launch_n<D, 1, true>(a, stream) : a.tiles == 2 ? launch_n<D, 2, true>(a, stream)
                                                                       : launch_n<D, 4, false>(a, stream);
}

// Query rows of a (sequence, KV head) that take the form with positions in the TMEM lanes (attn_mass_tc.cu).  us here / there
// with 4, 8, 16, 24, 64 rows: 256 ragged units of up to 32,768 positions 101 / 327, 160 / 328, 273 / 334, 390 / 335, 658 / 381;
// 256 of 32,768 139 / 510, 229 / 511, 408 / 516, 588 / 517, 1001 / 593; 32 ragged ones 24 / 55, 30 / 55, 45 / 56, 65 / 56, 111 / 65;
// 8 of 16,384 12 / 18, 15 / 18, 17 / 18, 22 / 18, 32 / 19; 128 ragged ones of up to 2000 15 / 31, 19 / 31, 25 / 33, 35 / 35,
// 54 / 40.  (17 rows cost here what 32 do: four tiles of four at a time.)  Longer heads' keys do not fit beside the scores.
bool many_rows(const Geom& g, int n) { return g.D == 128 && int64_t(n) * g.G > 16; }

}  // namespace

uint64_t mass_frag_bytes(const Geom& g, int n) {
  if (many_rows(g, n)) return mass_image_bytes(g, n);
  const uint64_t rows = uint64_t(g.B) * g.Hkv * ((int64_t(n) * g.G + 3) / 4) * 4;
  return rows * (uint64_t(g.D) * 12 + 16 + g.Dg * 4);
}

int launch_attn_mass(const MassArgs& args, cudaStream_t stream) {
  if (many_rows(args.g, args.n)) return launch_attn_mass_tc(args, stream);
  MassArgs a = args;
  a.tiles = int((int64_t(a.n) * a.g.G + 3) / 4);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_LAUNCH;
  // Positions of a warp: few enough for every SM to have 32 warps in turn.  us a call with 32 / 64 / 128 / 256: 64 units of
  // 32,768 positions 63 / 51 / 47 / 51, 256 of 8192 69 / 55 / 52 / 55, 8 of 32,768 15 / 14 / 15 / 20; 256 ragged ones of up to
  // 32,768 107 with 128, 103 with 256.
  const int64_t even = int64_t(a.top) * a.g.B * a.g.Hkv / (32 * sms);
  a.piece = even >= 4 * kMostPiece ? kMostPiece : int(std::min<int64_t>(kMostPiece / 2, std::max<int64_t>(kBatch, even / kBatch * kBatch)));
  return a.g.D == 128 ? launch_d<128>(a, stream) : a.g.D == 256 ? launch_d<256>(a, stream) : launch_d<512>(a, stream);
}

}  // namespace oscar
