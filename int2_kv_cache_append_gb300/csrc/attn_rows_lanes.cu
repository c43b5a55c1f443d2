// Attention of blocks of query rows over one cache on the 5th-generation tensor
// cores, head_dim 128, query rows in the TMEM lanes: the kernel behind
// attn_extend and attn_decode_prefix for a bf16 output and more than 32 query
// rows per (sequence, KV head).
//
// A CTA holds 128 rotated query rows and walks its share of the positions 128 at
// a time:
//
//   S [128 rows x 128 tokens] = Q K^T,   O [128 rows x 128 channels] += P V
//
// The arithmetic is that of the token-lane kernel (attn_rows_tc.cu): INT2 keys
// as exact fp16 values and a rank-one term, queries as two fp16 values, value
// rows with an exponent of their own that joins the score.  A row's reference M
// lies 8 below its maximum when it is chosen and follows it only when that has
// grown by 2^7 (P is fp16), and then its warps rescale their rows of O.
//
// Eight softmax warps: warp w has rows 32 (w mod 4) .. + 31 and the tokens of
// half w / 4; the two threads of a row exchange their maxima once per tile.  Two
// score tiles alternate, so the products of one run under the softmax of the
// other.  Both left operands come from TMEM: Q's two parts stay there, and P
// overwrites the scores that it was made from.  In shared memory they would
// take 96 KB of reads per tile from a budget (128 bytes per clock) that K, V
// and their expansion already use.
//
// What bounds it: the hand-overs from the products to the softmax to the next
// products, and beside them the V expanders, busy all the time.  A tile takes
// about 2850 cycles, of which the tensor cores need 1600; without the expansion,
// or without the softmax, it would still take three quarters of that.  A chunk of 2048 tokens x 64
// heads over 16,384 positions (one sequence, 8 KV heads): 1.28 ms, 0.8 PFLOP/s
// of products that the operator needs (the low part of Q doubles those of the
// scores).
#include <algorithm>

#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int N = 128;                  // query rows per CTA
constexpr int D = 128;
constexpr int kSoftWarps = 8;
constexpr int kThreads = (kSoftWarps + 4 + 4 + 1) * 32;
constexpr float kNone = -1e30f;         // M before the first visible position
constexpr float kTop = 15.f;            // log2 of the largest P (fp16 below 2^16)
constexpr float kBelow = 8.f;           // a new M lies this far below its row's maximum
constexpr int KU = 4, VU = 4, CB = 4, kStages = 4;  // two tiles of K and of V units
constexpr int oK = 0;
constexpr int oV = oK + KU * kUnit;
constexpr int oRawK = oV + VU * kUnit;
constexpr int oRawV = oRawK + kStages * kRawStage;
constexpr int oRank = oRawV + kStages * kRawStage;  // the keys' two and the queries' rank-one operands
constexpr int oConst = oRank + 3 * kRank;
constexpr int oRow = oConst + CB * TileConsts<true>::kBytes;
constexpr int kRow = N * 4 + 4 * N * 4;             // row index; exchange [2][2][N]
constexpr int oBar = oRow + kRow;
constexpr int kBars = 2 * KU + 2 * VU + 2 * CB + 2 + 1 + 1 + 2;
constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;  // + alignment slack
static_assert(oBar % 8 == 0 && kBytes <= 232448, "shared memory");
constexpr uint32_t cS = 0, cO = 256, cQ = 384;        // TMEM columns: two score tiles, O, Q's two parts

// 64 consecutive columns of the thread's TMEM lane
__device__ __forceinline__ void tmem_ld64(uint32_t a, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(a));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]),
                 "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]), "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]),
                 "+r"(r[40]), "+r"(r[41]), "+r"(r[42]), "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]),
                 "+r"(r[48]), "+r"(r[49]), "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]),
                 "+r"(r[56]), "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
               :
               : "memory");
}

__global__ void __launch_bounds__(kThreads, 1) attn_rows_lanes_kernel(const RowsArgs a) {
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

  int* outr = reinterpret_cast<int*>(sm + oRow);            // a row's index among all query rows, -1 = none
  float* swap = reinterpret_cast<float*>(outr + N);         // [2][2][N]
  const uint32_t bar = base + oBar;
  const uint32_t k_full = bar, k_empty = k_full + 8 * KU, v_full = k_empty + 8 * KU, v_empty = v_full + 8 * VU,
                 c_full = v_empty + 8 * VU, c_empty = c_full + 8 * CB, s_full = c_empty + 8 * CB, p_full = s_full + 16,
                 p_done = p_full + 8, q_full = p_done + 8, drained = q_full + 8;
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + oBar + kBars * 8);
  uint32_t* tmem_slot = words;

  for (int c = threadIdx.x; c < N; c += kThreads) {
    const int row = rt * N + c, t = row / g.G;
    const bool live = row < rows && t < ql;
    outr[c] = live ? (b * a.n + t) * g.Hq + h * g.G + row % g.G : -1;
    if (nt <= 0 && live) *reinterpret_cast<float2*>(a.ml + (int64_t(outr[c]) * a.ns + s) * 2) = make_float2(kNone, 0.f);
  }
  if (nt <= 0) {  // nothing visible in this share
    rows_wait(a);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < KU; ++i) mbar_init(k_full + 8 * i, 4), mbar_init(k_empty + 8 * i, 1);
    for (int i = 0; i < VU; ++i) mbar_init(v_full + 8 * i, 4), mbar_init(v_empty + 8 * i, 1);
    for (int i = 0; i < CB; ++i) mbar_init(c_full + 8 * i, 8), mbar_init(c_empty + 8 * i, kSoftWarps);
    for (int i = 0; i < 2; ++i) mbar_init(s_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
    mbar_init(p_full, kSoftWarps);
    mbar_init(p_done, 1);
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
    const int half = warp >> 2, row = threadIdx.x & 127;     // the thread's tokens of a tile and row (TMEM lane)
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;  // the warp's TMEM lanes
    float qscale;  // power of two that undoes the row's scaling
    // Q: this thread's 64 channels of its row, scaled (query_exponent) and split into two fp16 parts.  Plain loads: the
    // rotation may still be writing when this kernel starts (row_launch).
    {
      const int r = outr[row];
      const float4* src = reinterpret_cast<const float4*>(a.qrot + int64_t(max(r, 0)) * D + 64 * half);
      uint32_t mx = 0;
      if (r >= 0) {
#pragma unroll 8
        for (int j = 0; j < 16; ++j) {
          const float4 v = src[j];
          const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (isfinite(f[e])) mx = max(mx, __float_as_uint(fabsf(f[e])));
        }
      }
      uint32_t* both = reinterpret_cast<uint32_t*>(swap + 2 * N);  // the row's two threads
      both[half * N + row] = mx;
      asm volatile("bar.sync 3, 256;" ::: "memory");
      const int fe = query_exponent(max(mx, both[(half ^ 1) * N + row]));
      const float inv = pow2i(-fe);
      qscale = pow2i(fe);
      float sum = 0.f;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (r >= 0) v = src[8 * c + j];
          sum += split_pair(v.x * inv, v.y * inv, hi[2 * j], lo[2 * j]);
          sum += split_pair(v.z * inv, v.w * inv, hi[2 * j + 1], lo[2 * j + 1]);
        }
        tmem_st16(tmem + lanes + cQ + 32 * half + 16 * c, hi);
        tmem_st16(tmem + lanes + cQ + 64 + 32 * half + 16 * c, lo);
      }
      swap[half * N + row] = sum;
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("bar.sync 3, 256;" ::: "memory");
      if (half == 0) {
        const uint2 q = rank_query(swap[row] + swap[N + row]);
        uint8_t* rank = sm + oRank + 2 * kRank;
        *reinterpret_cast<uint4*>(rank + rank_offset(row, 0)) = make_uint4(q.x, q.y, 0, 0);
        *reinterpret_cast<uint4*>(rank + rank_offset(row, 8)) = make_uint4(0, 0, 0, 0);
      }
      fence_async();
      fence_before();
      __syncwarp();
      mbar_arrive_if(q_full, lane == 0);
      asm volatile("bar.sync 3, 256;" ::: "memory");  // the sums have been read
    }
    const int t_row = (rt * N + row) / g.G;
    const int lim = outr[row] < 0 ? -1 : a.causal ? T - ql + t_row : T - 1;  // last position that the row sees
    const uint32_t O = tmem + lanes + cO + 64 * half;
    float M = kNone;
    uint64_t l2 = 0;
    bool ok = true;
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      const int cb = i % CB, base_pos = p0 + i * kTok;
      ok = ok && wait(c_full + 8 * cb, (i / CB) & 1);
      ok = ok && wait(s_full + 8 * (i & 1), (i >> 1) & 1);
      fence_after();
      const uint32_t S = tmem + lanes + cS + (i & 1) * 128 + 64 * half;
      const TileConsts<true> tc(sm + oConst, cb);
      float phi = kKeyEven * qscale;
      const bool masked = base_pos + kTok - 1 > see_all;  // some row does not see some position of the tile
      const bool plain = !masked && *tc.uneven() == 0;
      const int see = lim - base_pos - 64 * half;          // the thread's columns j <= see are visible
      const float* ev = tc.e() + 64 * half;
      const float* rv = tc.rv() + 64 * half;
      // the scores of this thread's 64 tokens; with exponents or hidden positions, u = phi S + e or -inf instead
      uint32_t r[64];
      tmem_ld64(S, r);
      if (*tc.k_uneven()) {  // some key row has a factor of its own
        phi = 1.f;
        const float* kf = tc.k() + 64 * half;
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(kf + j);
          r[j] = __float_as_uint(__uint_as_float(r[j]) * (f.x * qscale));
          r[j + 1] = __float_as_uint(__uint_as_float(r[j + 1]) * (f.y * qscale));
          r[j + 2] = __float_as_uint(__uint_as_float(r[j + 2]) * (f.z * qscale));
          r[j + 3] = __float_as_uint(__uint_as_float(r[j + 3]) * (f.w * qscale));
        }
      }
      float top = -INFINITY, top1 = -INFINITY;
      if (plain) {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          top = max3(top, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
          top1 = max3(top1, __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
        }
        top = fmaxf(top, top1) * phi;
      } else {
#pragma unroll
        for (int j = 0; j < 64; j += 4) {
          const float4 e = *reinterpret_cast<const float4*>(ev + j);
          const float x[4] = {fmaf(__uint_as_float(r[j]), phi, e.x), fmaf(__uint_as_float(r[j + 1]), phi, e.y),
                              fmaf(__uint_as_float(r[j + 2]), phi, e.z), fmaf(__uint_as_float(r[j + 3]), phi, e.w)};
#pragma unroll
          for (int q = 0; q < 4; ++q) r[j + q] = __float_as_uint(j + q <= see ? x[q] : -INFINITY);
          top = max3(top, __uint_as_float(r[j]), __uint_as_float(r[j + 1]));
          top1 = max3(top1, __uint_as_float(r[j + 2]), __uint_as_float(r[j + 3]));
        }
        top = fmaxf(top, top1);
      }
      swap[(i & 1) * 2 * N + half * N + row] = top;
      if (any256(3, !ok)) {
        ok = false;
        break;
      }
      top = fmaxf(top, swap[(i & 1) * 2 * N + (half ^ 1) * N + row]);
      const bool grow = top > M + kTop;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2f(M - (top - kBelow)) : 1.f;
        if (grow) M = top - kBelow;
        l2 = mul2(l2, splat_x2(f));
        if (i > 0) {
          ok = wait(p_done, (i - 1) & 1);  // O is not in use
          fence_after();
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t o[16];
            tmem_ld16(O + c, o);
            tmem_wait16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(O + c, o);
          }
        }
      }
      // P, over the scores
      const uint64_t n2 = splat_x2(-M);
      uint64_t sum = 0, sum1 = 0;  // of this tile, so that l takes one rounding a tile
      if (plain) {
        const uint64_t phi2 = splat_x2(phi);
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float v, w;
            unpack2(fma2(pack2(__uint_as_float(r[c + 2 * j]), __uint_as_float(r[c + 2 * j + 1])), phi2, n2), v, w);
            v = ex2z(v);
            w = ex2z(w);
            p[j] = half2_of(v, w);
            if (j & 1) sum = add2(sum, pack2(v, w));
            else sum1 = add2(sum1, pack2(v, w));
          }
          tmem_st16(S + c / 2, p);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(rv + c + 2 * j);
            float v[4];
            unpack2(add2(pack2(__uint_as_float(r[c + 2 * j]), __uint_as_float(r[c + 2 * j + 1])), n2), v[0], v[1]);
            unpack2(add2(pack2(__uint_as_float(r[c + 2 * j + 2]), __uint_as_float(r[c + 2 * j + 3])), n2), v[2], v[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = ex2z(v[q]);
            p[j] = half2_of(v[0], v[1]);
            p[j + 1] = half2_of(v[2], v[3]);
            sum1 = fma2(pack2(v[0], v[1]), y.x, sum1);
            sum = fma2(pack2(v[2], v[3]), y.y, sum);
          }
          tmem_st16(S + c / 2, p);
        }
      }
      l2 = add2(l2, add2(sum, sum1));
      // every warp sees every phase of p_done: the next one cannot complete before this warp's arrival below
      if (i > 0) ok = ok && wait(p_done, (i - 1) & 1);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      mbar_arrive_if(p_full, lane == 0);
      mbar_arrive_if(c_empty + 8 * cb, lane == 0);
    }
    // the sums of a row's two threads, then O
    ok = ok && wait(p_done, (nt - 1) & 1);
    float l, l1;
    unpack2(l2, l, l1);
    l += l1;
    float* sums = swap + (nt & 1) * 2 * N;  // not the last tile's maxima, which may still be read
    sums[half * N + row] = l;
    if (!any256(3, !ok)) {
      fence_after();
      const int r = outr[row];
      if (r >= 0 && half == 0)
        *reinterpret_cast<float2*>(a.ml + (int64_t(r) * a.ns + s) * 2) = make_float2(M, l + sums[N + row]);
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        uint32_t v[16];
        tmem_ld16(O + c, v);
        tmem_wait16(v);
        if (r >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(a.acc + (int64_t(r) * a.ns + s) * D + 64 * half + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        }
      }
    } else if (lane == 0) {
      fail();
    }
  } else if (warp < kSoftWarps + 8) {
    Share x{&a, u, T, p0, p1, nt, sm, base, k_full, k_empty, v_full, v_empty, c_full, c_empty,
            oK, oV, oRawK, oRawV, oConst, oRank};
    const int tok = threadIdx.x - kSoftWarps * 32;
    const bool ok = warp < kSoftWarps + 4 ? (g.lm ? expand_k<1, KU, CB, kStages, 4, true, true>(x, tok, lane) : expand_k<1, KU, CB, kStages, 4, false, true>(x, tok, lane))
                                          : (g.lm ? expand_v<1, VU, CB, kStages, 4, true, true>(x, warp & 3, lane) : expand_v<1, VU, CB, kStages, 4, false, true>(x, warp & 3, lane));
    cp_async_wait<0>();  // also where a wait ran out
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------ MMA issuer --------------------------------
    // One warp issues every product; its instructions, not the tensor cores, would be the kernel's bound if it computed
    // buffer indices and looked at the outcome of every wait.
    const uint32_t leader = elect_one();
    constexpr uint32_t id_qk = idesc_of(kTok, false, false), id_pv = idesc_of(D, false, true);
    const uint32_t dK = desc_of(base + oK, 16), dV = desc_of(base + oV, kUnit / 2), dRank = rank_desc(base + oRank);
    Waits waits{a.wait_turns};
    Ring<KU> kr;
    Ring<VU> vr;
    auto product_qk = [&](uint32_t odd) {
      const uint32_t d = cS + odd * 128;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        waits.on(k_full + 8 * kr.at, kr.phase);
        fence_after();
        const uint32_t k = dK + kr.at * (kUnit >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)  // Q's high, then its low part; descriptors count 16 bytes
          mma_f16_ts(d, cQ + 64 * (j >> 2) + 32 * half + 8 * (j & 3), k + 2 * (j & 3), id_qk, half | j, leader);
        if (half == 0) mma_f16_ss<kDescRank>(d, dRank + (2 * kRank >> 4), dRank + odd * (kRank >> 4), id_qk, 1, leader);
        mma_commit(k_empty + 8 * kr.at, leader);
        kr.next();
        if (g.lm) {
          waits.on(k_full + 8 * kr.at, kr.phase);
          fence_after();
          const uint32_t x = dK + kr.at * (kUnit >> 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16_ts(d, cQ + 32 * half + 8 * j, x + 2 * j, id_qk, 1, leader);
          mma_commit(k_empty + 8 * kr.at, leader);
          kr.next();
        }
      }
      mma_commit(s_full + 8 * odd, leader);
    };
    auto product_pv = [&](uint32_t odd, uint32_t acc) {
      waits.on(p_full, odd);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        waits.on(v_full + 8 * vr.at, vr.phase);
        fence_after();
        const uint32_t v = dV + vr.at * (kUnit >> 4);
        const uint32_t p = cS + odd * 128 + 64 * k;  // 64 tokens of P in 32 columns
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16_ts(cO, p + 8 * j, v + 128 * j, id_pv, k | j ? 1 : acc, leader);
        mma_commit(v_empty + 8 * vr.at, leader);
        vr.next();
      }
      mma_commit(p_done, leader);
    };
    waits.on(q_full, 0);
    waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
    fence_after();
    if (__all_sync(0xffffffffu, waits.ok)) {
      product_qk(0);
      if (nt > 1) product_qk(1);
    }
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      if (!__all_sync(0xffffffffu, waits.ok)) break;
      product_pv(i & 1, i > 0);
      if (i + 2 < nt) {
        waits.on(p_done, i & 1);  // the scores of tile i + 2 overwrite P
        fence_after();
        product_qk(i & 1);
      }
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

}  // namespace

int launch_attn_rows_lanes(const RowsArgs& a, cudaStream_t stream) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_rows_lanes_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int64_t tiles = (int64_t(a.n) * a.g.G + N - 1) / N;
  const int64_t items = tiles * a.g.B * a.g.Hkv * a.ns;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  return row_launch(true, attn_rows_lanes_kernel, dim3(unsigned(items)), kThreads, kBytes, stream, a);
}

}  // namespace oscar
