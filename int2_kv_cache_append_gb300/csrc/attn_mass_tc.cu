// attn_mass of many query rows, head_dim 128, on the 5th-generation tensor cores
// (the mathematics and the form for few rows: attn_mass.cu).
//
// Positions are the TMEM lanes and query rows the columns, so the sum over rows is
// a thread's own, without exchanges, and a position's scale and zero are two of its
// registers.  Keys are expanded once per tile of 256 positions, into TMEM, to exact
// fp16 values (code - 1, or 150 times a Lloyd-Max level's distance from the middle;
// what that leaves out joins the zero); the rows pass by 96 at a time as two fp16
// parts, 22 bits.  BF16 positions take the same way with three bf16 parts.  The order
// of the channels is that of the code words: the rows' parts are written in it, and
// in the swizzled form in which a bulk copy brings them, by a kernel of their own.
//
// TMEM holds a tile's keys (2 x 64 columns) and two buffers of scores (2 x 2 x 96): the
// products of one block of rows run under the exponentials of the other.  With the keys
// in shared memory and blocks of 128 rows, every product reads twice the bytes there:
// 97 instead of 85 us below.
//
// What bounds it: the way of the scores out of TMEM (100 KB a block of rows) and the
// constants of a row, a broadcast of 16 bytes for each; a block of rows takes 1.5 us, its
// products 0.8.  8 KV heads over 16,384 positions, us with 32 / 64 / 128 / 256 / 1024 rows
// each: 20 / 21 / 27 / 36 / 85 (attn_mass.cu 24 / 34 / 58 / 97 / 358), of which the
// rotation and the parts are 10.  Sixteen warps instead of eight, all of a thread's scores
// read before the first exponential, the constants brought by bulk copies: no change.
#include <algorithm>
#include <type_traits>

#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int D = 128;
constexpr int kTile = 256;                    // positions: two accumulators
constexpr int kRows = 96;                     // query rows of a block of them
constexpr int kPiece = kRows * 128;           // bytes of half of their channels
constexpr int kSoftWarps = 8, kMma = kSoftWarps, kCopy = kMma + 1, kThreads = (kCopy + 1) * 32;
constexpr int kImage16 = 4 * kPiece, kImageBf = 6 * kPiece;  // parts x channel halves
constexpr uint32_t cKeys = 0, cScores = 128, kScores = 2 * kRows;  // TMEM columns: 64 per accumulator; two buffers
constexpr int oB = 0;                         // [2 buffers]
constexpr int oTable = oB + 2 * kImageBf;     // [2][pairs of rows][factor, sum, -reference high, low][2]
constexpr int oJoin = oTable + 2 * kRows * 16;  // [256] sums over the upper half of the columns
constexpr int oBar = oJoin + kTile * 4;
struct Bars {
  uint32_t b_full, b_free, a_full, d_full, d_free, drained;
  __device__ explicit Bars(uint32_t at)
      : b_full(at), b_free(at + 16), a_full(at + 32), d_full(at + 40), d_free(at + 56), drained(at + 72) {}
};
constexpr int kBytes = oBar + 10 * 8 + 16 + 1024;  // + TMEM address, alignment slack
static_assert(oBar % 8 == 0 && kBytes <= 232448, "shared memory");

// What mass_images_kernel leaves per (sequence, KV head), by blocks of kRows rows
struct Images {
  uint8_t *f16, *bf;
  float4* row;  // factor, reference high and low
  float* sum;
};
__host__ __device__ inline Images images_of(const MassArgs& a, int64_t unit) {
  const int64_t units = int64_t(a.g.B) * a.g.Hkv;
  uint8_t* at = a.frags;
  Images f;
  f.f16 = at + unit * a.tiles * kImage16;
  at += units * a.tiles * kImage16;
  f.bf = at + unit * a.tiles * kImageBf;
  at += units * a.tiles * kImageBf;
  f.row = reinterpret_cast<float4*>(at) + unit * a.tiles * kRows;
  at += units * a.tiles * (kRows * 16);
  f.sum = reinterpret_cast<float*>(at) + unit * a.tiles * kRows;
  return f;
}

// a warp per row
__global__ void __launch_bounds__(128) mass_images_kernel(const MassArgs a) {
  const Geom& g = a.g;
  const int lane = threadIdx.x & 31;
  const int64_t at_row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5), units = int64_t(g.B) * g.Hkv;
  const int64_t unit = at_row / (kRows * a.tiles);
  pdl_wait();  // the rotated queries
  if (unit >= units) return;
  const int row = int(at_row - unit * kRows * a.tiles), b = int(unit / g.Hkv), h = int(unit % g.Hkv);
  const int ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n);
  const bool on = row < ql * g.G;
  const Images f = images_of(a, unit);
  const int64_t at = (int64_t(b) * a.n + row / g.G) * g.Hq + h * g.G + row % g.G;
  const float* q = a.qrot + (on ? at : 0) * D;
  const float lse = on ? a.lse[at] : -INFINITY;
  const bool weighs = lse != -INFINITY;  // else the query may be anything
  // columns k = 4 lane .. + 3 of the codes' order: word k / 16 holds channels 64 (w & 1) + 16 (p / 2) + 8 (p & 1) + 2 (w / 2)
  // and the next one as pair p
  const int w = lane >> 2, c0 = 64 * (w & 1) + 16 * (lane & 3) + 2 * (w >> 1);
  float2 u = make_float2(0.f, 0.f), v = u;
  float4 n4 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (weighs) {
    u = *reinterpret_cast<const float2*>(q + c0);
    v = *reinterpret_cast<const float2*>(q + c0 + 8);
    n4 = *reinterpret_cast<const float4*>(q + 4 * lane);  // the BF16 rows' order
  }
  const float x[4] = {u.x, u.y, v.x, v.y}, y[4] = {n4.x, n4.y, n4.z, n4.w};
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (isfinite(x[i])) most = max(most, __float_as_uint(fabsf(x[i])));
#pragma unroll
  for (int o = 16; o; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  // the largest finite component lands in [2^6, 2^7): products with 249 stay far from float32's end, low parts above fp16's
  const int e = max(-100, (int(most) >> 23) - 126 - 7);
  const float up = pow2i(min(126, -e));
  uint32_t hi[2], lo[2];
  float sum = split_pair(x[0] * up, x[1] * up, hi[0], lo[0]);
  sum += split_pair(x[2] * up, x[3] * up, hi[1], lo[1]);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  // half of the channels, then a row's swizzled 16-byte pieces
  const int r = row % kRows;
  const int64_t off = (lane >> 4) * kPiece + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + 8 * (lane & 1);
  uint8_t* to = f.f16 + int64_t(row / kRows) * kImage16 + off;
  *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(to + 2 * kPiece) = make_uint2(lo[0], lo[1]);
  uint32_t s[4][3];
#pragma unroll
  for (int i = 0; i < 4; ++i) split3_bf16(y[i], s[i]);
  to = f.bf + int64_t(row / kRows) * kImageBf + off;
#pragma unroll
  for (int part = 0; part < 3; ++part)
    *reinterpret_cast<uint2*>(to + part * 2 * kPiece) = make_uint2(s[0][part] | s[1][part] << 16, s[2][part] | s[3][part] << 16);
  if (lane == 0) {
    float high = lse * 1.4426950408889634f;
    // the product's rounding and what the constant leaves out
    float low = fmaf(lse, 1.4426950408889634f, -high) + lse * 1.9259629911266175e-8f;
    if (!isfinite(high)) high = weighs ? high : INFINITY, low = 0.f;
    f.row[row] = make_float4(pow2i(min(127, max(-126, e))), high, low, 0.f);
    f.sum[row] = sum * pow2i(min(127, max(-126, e)));
  }
}

// A tile: 256 of the positions of one kind
struct Tile {
  bool bf;
  int i0;  // first of them
};

__global__ void __launch_bounds__(kThreads, 1) attn_mass_tc_kernel(const MassArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const Geom& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = blockIdx.y, b = unit / g.Hkv;
  const int given = a.seq_lens[b], T = max(0, min(given, g.cap));
  if (given > g.cap && blockIdx.x == 0 && threadIdx.x == 0) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
  const int ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n), rows = ql * g.G;
  const int seen = T - ql;                // every row sees the positions up to this one
  const int window = max(g.S, T - g.W);   // the ring's first position
  const int sinks = min(g.S, T), packed = max(0, min(T, window) - g.S), ints = (packed + kTile - 1) / kTile;
  const int bfs = sinks + max(0, T - window), tiles = ints + (bfs + kTile - 1) / kTile;
  const float* mass_in = a.mass_in ? a.mass_in + int64_t(unit) * g.cap : nullptr;
  float* mass_out = a.mass_out + int64_t(unit) * g.cap;
  if (rows == 0) {
    pdl_wait();
    for (int64_t p = int64_t(blockIdx.x) * kThreads + threadIdx.x; p < T; p += int64_t(gridDim.x) * kThreads)
      mass_out[p] = mass_in ? mass_in[p] : 0.f;
    return;
  }
  if (int(blockIdx.x) >= tiles) {
    pdl_wait();
    return;
  }
  const Images f = images_of(a, unit);
  auto tile_of = [&](int t) { return Tile{t >= ints, (t >= ints ? t - ints : t) * kTile}; };
  const int chunks = (rows + kRows - 1) / kRows;
  auto width = [&](int c) { return min(kRows, (rows - c * kRows + 31) & ~31); };  // rows of a block, padded

  const Bars bar(base + oBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + oBar + 80);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.b_full + 8 * i, 1);
      mbar_init(bar.b_free + 8 * i, 1);
      mbar_init(bar.d_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
      mbar_init(bar.d_free + 8 * i, kSoftWarps);
    }
    mbar_init(bar.a_full, kSoftWarps);
    mbar_init(bar.drained, 1);
    mbar_fence_init();
  }
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() { status_or(a.status, OSCAR_DEV_TIMEOUT); };

  if (warp < kSoftWarps) {
    // ------------------------- keys and exponentials --------------------------
    // A thread has two positions, a lane of either accumulator, so that a row's constants are read once for both; of the keys
    // it expands half of the channels, of a block's rows it takes half.
    const int r = threadIdx.x & 127, half = warp >> 2;
    const uint32_t lanes = tmem + (uint32_t(32 * (warp & 3)) << 16);
    float* table = reinterpret_cast<float*>(sm + oTable);
    float* join = reinterpret_cast<float*>(sm + oJoin) + r;
    const uint8_t* codes = a.layer_base + g.sink_bytes + g.ring_bytes;
    const uint8_t* sz = codes + g.codes_bytes + int64_t(unit) * g.ncap * 4;
    codes += int64_t(unit) * g.ncap * (D / 4);
    const uint8_t* sink = a.layer_base + int64_t(unit) * g.S * (2 * D);
    const uint8_t* ring = a.layer_base + g.sink_bytes + int64_t(unit) * g.W * (2 * D);

    struct Key {
      uint4 w;
      uint32_t sz;
      int p;  // the position; its complement behind the last
    };
    struct Keys {
      Key of[2];
    };
    auto load = [&](Keys& y, const Tile& t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        Key& x = y.of[e];
        const int i = t.i0 + 128 * e + r, n = t.bf ? bfs : packed, at = min(i, n - 1);
        x.p = t.bf ? (at < sinks ? at : window + at - sinks) : g.S + at;
        if (!t.bf) {
          x.w = __ldg(reinterpret_cast<const uint4*>(codes + int64_t(at) * (D / 4)) + half);
          x.sz = __ldg(reinterpret_cast<const uint32_t*>(sz) + at);
        }
        if (i >= n) x.p = ~x.p;
      }
    };
    auto expand = [&](const Keys& y, const Tile& t) {
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const Key x = e ? y.of[1] : y.of[0];
        const uint32_t to = lanes + cKeys + 64 * e + 32 * half;
        const int p = x.p < 0 ? ~x.p : x.p;
        const uint4* src = reinterpret_cast<const uint4*>(p < g.S ? sink + int64_t(p) * (2 * D) : ring + int64_t(p % max(g.W, 1)) * (2 * D));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[16];
          if (t.bf) {
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const uint4 u = __ldg(src + 8 * half + 4 * c + m);
              v[4 * m] = u.x, v[4 * m + 1] = u.y, v[4 * m + 2] = u.z, v[4 * m + 3] = u.w;
            }
          } else {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t word = c == 0 ? (w ? x.w.y : x.w.x) : (w ? x.w.w : x.w.z);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t s = code_shift(word, q);
                uint32_t even = less_one_even(s), odd = less_one_odd(s);
                if (g.lm) even = lm_value(even), odd = lm_value(odd);
                v[8 * w + 2 * q] = even, v[8 * w + 2 * q + 1] = odd;
              }
            }
          }
          tmem_st16(to + 16 * c, v);
        }
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      mbar_arrive_if(bar.a_full, lane == 0);
    };
    // the constants of a block's row, by a thread each
    const int own = threadIdx.x;
    auto constants = [&](const Tile& t, int c, float4& x, float& sum) {
      if (own >= width(c)) return;
      const int at = c * kRows + own;
      x = f.row[at];
      sum = t.bf ? 0.f : f.sum[at];
      if (t.bf) x.x = 1.f;
    };

    Tile t = tile_of(blockIdx.x);
    Keys key;
    load(key, t);
    pdl_wait();  // the rows' parts
    float4 rc = make_float4(0.f, 0.f, 0.f, 0.f);
    float rs = 0.f;
    constants(t, 0, rc, rs);
    expand(key, t);
    bool ok = true;
    uint32_t k = 0;
#pragma unroll 1
    for (int at = blockIdx.x; at < tiles; at += gridDim.x) {
      const bool more = at + int(gridDim.x) < tiles;
      const Tile then = more ? tile_of(at + gridDim.x) : t;
      Keys key2 = key;
      if (more) load(key2, then);
      uint64_t sc2[2], zero2[2], sum[2][2];
      int first[2];  // the first row that sees the position
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sc = 1.f, zero = 0.f;
        if (!t.bf) {
          const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&key.of[e].sz));
          sc = g.lm ? z.x * (1.f / 150.f) : z.x;
          zero = g.lm ? fmaf(z.x, kLmMiddle, z.y) : z.x + z.y;
        }
        sc2[e] = splat_x2(sc), zero2[e] = splat_x2(zero);
        sum[e][0] = sum[e][1] = 0;
        const int p = key.of[e].p;
        first[e] = max(0, (p < 0 ? ~p : p) - seen) * g.G;
      }
      // the position that this thread writes
      const int p = half ? key.of[1].p : key.of[0].p;
      const float before = p >= 0 && mass_in ? mass_in[p] : 0.f;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++k) {
        const int n = width(c);
        float* tab = table + (k & 1) * (kRows * 4);
        if (own < n) {
          float* to = tab + (own >> 1) * 8 + (own & 1);
          to[0] = rc.x, to[2] = rs, to[4] = -rc.y, to[6] = -rc.z;
        }
        const bool last = c + 1 == chunks;
        if (!last || more) constants(last ? then : t, last ? 0 : c + 1, rc, rs);
        ok = wait_warp(bar.d_full + 8 * (k & 1), (k >> 1) & 1, a.wait_turns);
        if (any256(3, !ok)) {
          ok = false;
          break;
        }
        fence_after();
        if (last && more) expand(key2, then);  // the products have read the keys before
        const int hidden0 = first[0] - c * kRows, hidden1 = first[1] - c * kRows;  // rows that do not see the position
        const bool masked = __any_sync(0xffffffffu, max(hidden0, hidden1) > 0);
        const uint32_t from = lanes + cScores + (k & 1) * kScores;
#pragma unroll 1
        for (int j0 = half * (n / 2); j0 < (half + 1) * (n / 2); j0 += 16) {
          uint32_t s0[16], s1[16];
          tmem_ld16(from + j0, s0);
          tmem_ld16(from + kRows + j0, s1);
          tmem_wait16(s0);
          tmem_wait16(s1);
          const ulonglong2* row = reinterpret_cast<const ulonglong2*>(tab + j0 * 4);
          auto weights = [&](auto hide) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const ulonglong2 x = row[2 * j], y = row[2 * j + 1];
              auto weight = [&](const uint32_t (&s)[16], uint64_t scale, uint64_t zero, int hidden) {
                const uint64_t d = mul2(pack2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), x.x);
                float u, v;
                unpack2(add2(fma2(scale, d, fma2(zero, x.y, y.x)), y.y), u, v);
                u = ex2z(u), v = ex2z(v);
                if (decltype(hide)::value) {
                  u = j0 + 2 * j >= hidden ? u : 0.f;
                  v = j0 + 2 * j + 1 >= hidden ? v : 0.f;
                }
                return pack2(u, v);
              };
              sum[0][j & 1] = add2(sum[0][j & 1], weight(s0, sc2[0], zero2[0], hidden0));
              sum[1][j & 1] = add2(sum[1][j & 1], weight(s1, sc2[1], zero2[1], hidden1));
            }
          };
          if (masked) weights(std::true_type());
          else weights(std::false_type());
        }
        fence_before();
        __syncwarp();
        mbar_arrive_if(bar.d_free + 8 * (k & 1), lane == 0);
      }
      if (!ok) break;  // in all of the warps or none
      float x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float u, v;
        unpack2(add2(sum[e][0], sum[e][1]), u, v);
        x[e] = u + v;
      }
      join[half ? 0 : 128] = half ? x[0] : x[1];
      asm volatile("bar.sync 2, 256;" ::: "memory");
      if (p >= 0) mass_out[p] = (half ? join[128] + x[1] : x[0] + join[0]) + before;
      t = then, key = key2;
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kMma) {
    // ------------------------------- products ---------------------------------
    const uint32_t leader = elect_one();
    const uint32_t dB = desc_of(base + oB, 16);
    Waits waits{a.wait_turns};
    waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
    uint32_t k = 0, a_phase = 0;
    // the low parts first: their sum enters while the total is small
    auto products = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t id, int parts) {
#pragma unroll 1
      for (int part = parts - 1; part >= 0; --part)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_f16_ts(d, x + 8 * j, y + (2 * part + (j >> 2)) * (kPiece >> 4) + 2 * (j & 3), id, part < parts - 1 || j > 0, leader);
    };
#pragma unroll 1
    for (int at = blockIdx.x; at < tiles && __all_sync(0xffffffffu, waits.ok); at += gridDim.x) {
      const Tile t = tile_of(at);
      waits.on(bar.a_full, a_phase);
      a_phase ^= 1;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++k) {
        const uint32_t buf = k & 1;
        waits.on(bar.b_full + 8 * buf, (k >> 1) & 1);
        if (k >= 2) waits.on(bar.d_free + 8 * buf, ((k >> 1) & 1) ^ 1);
        fence_after();
        if (!__all_sync(0xffffffffu, waits.ok)) break;
        const uint32_t id = idesc_of(width(c), false, false) | (t.bf ? kBf16 : 0u);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          products(cScores + buf * kScores + x * kRows, cKeys + 64 * x, dB + buf * (kImageBf >> 4), id, t.bf ? 3 : 2);
        mma_commit(bar.b_free + 8 * buf, leader);
        mma_commit(bar.d_full + 8 * buf, leader);
      }
    }
    if (!__all_sync(0xffffffffu, waits.ok) && lane == 0) fail();
    mma_commit(bar.drained, leader);  // every product issued is complete before TMEM is freed
    mbar_wait(bar.drained, 0);
    __syncwarp();
  } else {
    // --------------------------------- rows -----------------------------------
    pdl_wait();
    if (lane == 0) {
      const uint64_t limit = a.wait_turns * 1000ull;
      uint32_t k = 0;
      bool ok = true;
#pragma unroll 1
      for (int at = blockIdx.x; at < tiles && ok; at += gridDim.x) {
        const Tile t = tile_of(at);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const uint32_t buf = k & 1, to = base + oB + buf * kImageBf, br = bar.b_full + 8 * buf;
          if (k >= 2) ok = mbar_wait(bar.b_free + 8 * buf, ((k >> 1) & 1) ^ 1, limit);
          if (!ok) break;
          const uint8_t* src = t.bf ? f.bf + int64_t(c) * kImageBf : f.f16 + int64_t(c) * kImage16;
          const int pieces = t.bf ? 6 : 4;
          const uint32_t bytes = width(c) * 128;
          mbar_arrive_expect_tx(br, pieces * bytes);
          for (int i = 0; i < pieces; ++i) bulk_g2s(to + i * kPiece, src + i * kPiece, bytes, br);
          ++k;
        }
      }
      if (!ok) fail();
      // what was issued lands before the block ends, also where a wait ran out
      for (uint32_t i = k >= 2 ? k - 2 : 0; i < k; ++i) mbar_wait(bar.b_full + 8 * (i & 1), (i >> 1) & 1);
    }
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (warp == kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

uint64_t mass_image_bytes(const Geom& g, int n) {
  const uint64_t blocks = uint64_t(g.B) * g.Hkv * ((int64_t(n) * g.G + kRows - 1) / kRows);
  return blocks * (kImage16 + kImageBf + kRows * 20);
}

int launch_attn_mass_tc(const MassArgs& args, cudaStream_t stream) {
  MassArgs a = args;
  a.tiles = int((int64_t(a.n) * a.g.G + kRows - 1) / kRows);
  static int known[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!known[dev]) {
    int n = 0;
    if (cudaFuncSetAttribute(attn_mass_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    known[dev] = n;
  }
  const int64_t units = int64_t(a.g.B) * a.g.Hkv, rows = units * a.tiles * kRows, sms = known[dev];
  const int rc = row_launch(true, mass_images_kernel, dim3(unsigned((rows + 3) / 4)), 128, 0, stream, a);
  if (rc != OSCAR_OK) return rc;
  // Blocks of a unit: the rounds of the SMs times a block's tiles, a tile's time for its start and end; of many units as many
  // that a block has 16 tiles at most, for ragged lengths.  us with 1 / 2 / 4 / 8 / 16 / 32: 256 units of up to 32,768
  // positions, 32 rows each, 404 / 337 / 299 / 286 / 298 / 330, 256 rows 915 / 770 / 681 / 641 / 654 / 690; 200 of up to 9000
  // 124 / 105 / 97 / 99 / 114 / 138.
  const int64_t tiles = (a.top + kTile - 1) / kTile + 1;
  int64_t best = 1, cost = INT64_MAX;
  for (int64_t x = 1; x <= std::min<int64_t>(tiles, std::max<int64_t>(1, 4 * sms / units)); ++x) {
    const int64_t c = (units * x + sms - 1) / sms * ((tiles + x - 1) / x + 1);
    if (c < cost) cost = c, best = x;
  }
  best = std::max(best, (tiles + 15) / 16);
  return row_launch(true, attn_mass_tc_kernel, dim3(unsigned(best), unsigned(units)), kThreads, kBytes, stream, a);
}

}  // namespace oscar
