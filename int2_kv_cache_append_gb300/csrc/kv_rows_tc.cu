// Products of many rows with a layer's rotation on the 5th-generation tensor
// cores: kv_read, the query rotation and the un-rotation of the merged rows for
// larger calls (kv_rows.cu has the float32 form and the merge).
//
//   out [128 rows x NC columns] = X [128 x D] B^T,  B [NC x D] = rows of R (or of R^T)
//
// A CTA keeps its NC columns of the matrix in shared memory as fp16 values,
// split into two parts where the result is float32 or a query, and walks the
// row tiles.  X is expanded to fp16 operands in units of 64 channels: cached
// INT2 rows as s (c - 1) with the middles as a rank-one term (see expand_k), every
// row scaled by a power of two of its own, with a second set of units for the
// rounding residues where the result is float32 and there are any; merged rows are
// such operands already.  A bf16 result takes one product, R and X rounded to
// fp16 (2^-11 each, against 2^-8 of the output); a query from bf16 two; a
// float32 result two or three, 2^-22.
//
// Two groups of four warps expand alternate tiles, one warp issues the
// products, four warps scale and store the result of the previous tile.
//
// What bounds it: at D = 128 the expansion and the stores (kv_read of 4 x 8192
// positions, 8 KV heads: 64 us, 2.5 TB/s, a third of the copy rate).  At larger
// D a row is expanded again for every NC columns, up to 8 times at D = 512, and
// the latency of BF16 rows counts, which are read once more for their largest
// value: 4 x 4099 positions at D = 512 take 208 us as INT2 rows into bf16, 490
// us into float32, and 486 us and 1.05 ms with 2560 BF16 rows among them.  Reading those
// rows by whole warps, line by line, was slower (1.33 ms).  Every wait is
// bounded, as in the attention kernels.
#include <algorithm>

#include "rows_tc.cuh"

namespace oscar {
namespace {

enum { kQuery, kFinish, kRead };

struct MmArgs {
  QrotRowsArgs q;
  FinishArgs f;
  ReadArgs r;
  int64_t tiles;
  int xl;  // the rows' low parts take part
  FastDiv div_hkv, div_n;  // of kv_read
  uint32_t wait_turns;     // limit of every barrier wait, a microsecond each at most
  int wait_poison;         // test hook: above 0, CTA 0's first accumulator expects an arrival that never comes
};

// The matrix enters times this: elements of a rotation are below 1, most far below, and the low part of a small one would
// be a subnormal fp16 number with few bits (float32 results were off by 1.4e-6 of their norm without it).
constexpr float kMatrixScale = 128.0f;
constexpr int kExpandWarps = 8, kStoreWarps = 4;
constexpr int kThreads = (kExpandWarps + kStoreWarps + 1) * 32;

template <int DG, bool RL>  // RL: the matrix's low part takes part
struct Plan {
  static constexpr int D = 128 * DG;
  static constexpr int NC = DG == 1 ? 128 : (RL ? 256 : 512) / DG;  // columns of a CTA
  static constexpr int PU = DG == 1 ? 3 : 2;                // units of an expanding group
  // The tensor cores cut every addition off: the 64 of two products over D = 512 in one sum make it 1e-6 too small.  So the
  // products with the low part have an accumulator of their own, and at D = 512 either half of the channels has one, too.
  static constexpr int kParts = !RL ? 1 : DG == 4 ? 3 : 2;
  static constexpr int kAcc = DG == 4 && !RL ? 4 : 2;        // tiles that have accumulators
  static constexpr int kCols = kAcc * kParts * NC > 256 ? 512 : 256;  // of TMEM
  static constexpr int kB = NC * D * 2;                     // one part of the matrix
  static constexpr int oB = 0;
  static constexpr int oX = (RL ? 2 : 1) * kB;
  static constexpr int oRank = oX + 2 * PU * kUnit;          // rows' (two), then the matrix's rank-one operand
  static constexpr int oRow = oRank + 2 * kRank + NC * 32;   // factors of the rows [kAcc][128]; sums of the matrix [NC][DG]
  static constexpr int oBar = oRow + kAcc * 128 * 4 + NC * DG * 4;
  static constexpr int kBars = 4 * PU + 3 * kAcc + 1;
  static constexpr int kBytes = oBar + kBars * 8 + 16 + 1024;
  static_assert(kBytes <= 232448, "shared memory");
};

// 32 bytes of a row, at once where the output is aligned to that
__device__ __forceinline__ void store32(void* dst, const uint32_t (&v)[8], bool aligned) {
  if (!aligned) {
    static_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    return;
  }
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int SRC, int DG, bool RL>
__global__ void __launch_bounds__(kThreads, 1) rows_mm_kernel(const __grid_constant__ MmArgs a) {
  using L = Plan<DG, RL>;
  constexpr int D = L::D, NC = L::NC, PU = L::PU, kAcc = L::kAcc, kParts = L::kParts, kStep = kParts * NC, kCols = L::kCols;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * NC;
  const int role = SRC == kRead && !a.r.k_out ? 1 : blockIdx.z;  // of kv_read: K, V, or the one that is asked for
  const Geom& g = a.r.g;
  const float* R = SRC == kQuery ? a.q.R_K : SRC == kFinish ? a.f.R_V : role ? a.r.R_V : a.r.R_K;
  const bool hadamard = SRC == kQuery ? a.q.hadamard : SRC == kFinish ? a.f.hadamard : a.r.hadamard;
  const bool plain = SRC == kFinish ? a.f.absorb_v : SRC == kRead ? role && a.r.absorb_v : false;  // no matrix
  void* out = SRC == kQuery ? a.q.qrot : SRC == kFinish ? a.f.out : role ? a.r.v_out : a.r.k_out;
  const bool out32 = SRC == kQuery || (SRC == kFinish ? a.f.out_fp32 : a.r.out_fp32);
  int32_t* status = SRC == kQuery ? a.q.status : SRC == kFinish ? a.f.status : a.r.status;
  const int64_t rows = SRC == kQuery ? a.q.rows : SRC == kFinish ? a.f.rows : int64_t(g.B) * a.r.n * g.Hkv;
  if (SRC == kQuery) pdl_trigger();

  float* factor = reinterpret_cast<float*>(sm + L::oRow);      // [kAcc][128]
  float* sums = factor + kAcc * 128;                                  // [NC][DG]
  const uint32_t bar = base + L::oBar;
  auto x_full = [&](int p, int i) { return bar + 8u * (p * PU + i); };
  auto x_empty = [&](int p, int i) { return bar + 8u * (2 * PU + p * PU + i); };
  const uint32_t f_full = bar + 32u * PU, acc_full = f_full + 8 * kAcc, acc_empty = acc_full + 8 * kAcc, drained = acc_empty + 8 * kAcc;
  uint32_t* words = reinterpret_cast<uint32_t*>(sm + L::oBar + L::kBars * 8);
  uint32_t* tmem_slot = words;

  if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) {
    if (SRC == kQuery && a.q.zero_word) *a.q.zero_word = 0;
  }
  if (threadIdx.x == 0) {
    for (int p = 0; p < 2; ++p)
      for (int i = 0; i < PU; ++i) mbar_init(x_full(p, i), 4), mbar_init(x_empty(p, i), 1);
    for (int p = 0; p < kAcc; ++p) {
      mbar_init(f_full + 8 * p, 4);
      mbar_init(acc_full + 8 * p, 1 + (p == 0 && blockIdx.x + blockIdx.y + blockIdx.z == 0 && a.wait_poison > 0));
      mbar_init(acc_empty + 8 * p, kStoreWarps);
    }
    mbar_init(drained, 1);
    mbar_fence_init();
  }
  if (warp == kExpandWarps + kStoreWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "n"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // B: a thread makes 16-byte chunks of 8 k of one column; sums of every column's groups for the rank-one term
  for (int i = threadIdx.x; i < NC * DG; i += kThreads) sums[i] = 0.f;
  __syncthreads();
  for (int i = threadIdx.x; i < NC * (D / 8); i += kThreads) {
    // consecutive threads: consecutive columns of R (query), or consecutive chunks of a row of R
    const int n = SRC == kQuery ? i % NC : i / (D / 8), k0 = (SRC == kQuery ? i / NC : i % (D / 8)) * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (plain) v[e] = c0 + n == k0 + e ? 1.f : 0.f;
      else if (hadamard) v[e] = hadamard_at(c0 + n, k0 + e);
      else v[e] = SRC == kQuery ? __ldg(R + int64_t(k0 + e) * D + c0 + n) : __ldg(R + int64_t(c0 + n) * D + k0 + e);
      v[e] *= kMatrixScale;
    }
    uint32_t hi[4], lo[4];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float both = split_pair(v[2 * e], v[2 * e + 1], hi[e], lo[e]);
      const float2 h = __half22float2(*reinterpret_cast<__half2*>(&hi[e]));
      sum += RL ? both : h.x + h.y;
    }
    uint8_t* dst = sm + L::oB + (k0 >> 6) * (NC * 128) + n * 128 + ((((k0 >> 3) & 7) ^ (n & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if (RL) *reinterpret_cast<uint4*>(dst + L::kB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (SRC == kRead) {
      // the 16 chunks of a (column, group) lie in 16 neighbouring lanes: one fixed order of summation
#pragma unroll
      for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      if ((lane & 15) == 0) sums[n * DG + (k0 >> 7)] = sum;
    }
  }
  if (SRC == kRead) {
    __syncthreads();
    for (int i = threadIdx.x; i < NC * 2; i += kThreads) {
      uint2 q[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int gr = 2 * (i & 1) + e;
        q[e] = gr < DG ? rank_query(sums[(i >> 1) * DG + gr]) : make_uint2(0, 0);
      }
      *reinterpret_cast<uint4*>(sm + L::oRank + 2 * kRank + rank_offset(i >> 1, 8 * (i & 1))) = make_uint4(q[0].x, q[0].y, q[1].x, q[1].y);
    }
    for (int i = threadIdx.x; i < 2 * kRank / 16; i += kThreads)
      *reinterpret_cast<uint4*>(sm + L::oRank + 16 * i) = make_uint4(0, 0, 0, 0);
  }
  fence_async();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  if (SRC == kFinish) pdl_wait();  // the merged rows
  auto fail = [&]() {
    status_or(status, OSCAR_DEV_TIMEOUT);
  };
  auto wait = [&](uint32_t br, uint32_t parity) { return wait_warp(br, parity, a.wait_turns); };
  const int sets = a.xl ? 2 : 1;
  const int mine = int((a.tiles - blockIdx.x + gridDim.x - 1) / gridDim.x);  // this CTA's tiles

  if (warp < kExpandWarps) {
    // ------------------------------ rows of X --------------------------------
    const int p = warp >> 2, r = threadIdx.x & 127;
    bool ok = true;
    int n = 0;  // units written
    auto cached = [&](int64_t row) {  // of kv_read
      RowRef ref{nullptr, nullptr, nullptr};
      if (row >= rows) return ref;
      const uint32_t bt = fastdiv(uint32_t(row), a.div_hkv), b = fastdiv(bt, a.div_n);
      const int h = int(uint32_t(row) - bt * uint32_t(g.Hkv));
      int T = a.r.seq_lens[b];
      if (T > g.cap) {
        status_or(status, OSCAR_DEV_OVER_CAPACITY);
        T = g.cap;
      }
      const int64_t pos = int64_t(a.r.start_pos[b]) + int(bt - b * uint32_t(a.r.n));
      if (pos >= 0 && pos < T) ref = row_ref(g, a.r.layer_base, role, int64_t(b) * g.Hkv + h, T, int(pos));
      return ref;
    };
    // INT2 codes a group ahead, scale / zero pairs a row ahead
    RowRef ref{nullptr, nullptr, nullptr}, next{nullptr, nullptr, nullptr};
    uint4 q0, q1, n0 = make_uint4(0, 0, 0, 0), n1 = n0;
    __half2 pairs[DG], npairs[DG];
    auto fetch_codes = [&](const RowRef& from, int gr) {
      if (!from.codes) return;
      n0 = __ldg(reinterpret_cast<const uint4*>(from.codes) + 2 * gr);
      n1 = __ldg(reinterpret_cast<const uint4*>(from.codes) + 2 * gr + 1);
    };
    auto fetch_pairs = [&](const RowRef& from) {
#pragma unroll
      for (int gr = 0; gr < DG; ++gr) npairs[gr] = from.codes ? __ldg(from.sz + gr) : __half2();
    };
    if (SRC == kRead && p < mine) {
      next = cached((int64_t(blockIdx.x) + int64_t(p) * gridDim.x) * 128 + r);
      fetch_codes(next, 0);
      fetch_pairs(next);
    }
#pragma unroll 1
    for (int j = p; ok && j < mine; j += 2) {
      const int64_t row = (int64_t(blockIdx.x) + int64_t(j) * gridDim.x) * 128 + r;
      // where the row comes from, and the factor that undoes its scaling
      const __nv_bfloat16* b16 = nullptr;
      const float* f32 = nullptr;
      const __half* merged = nullptr;  // scaled already; its residues D further on
      float up = 0.f, down = 0.f;
      if (SRC == kRead) {
        ref = next;
        b16 = ref.wide;
        next = j + 2 < mine ? cached(row + 2 * int64_t(gridDim.x) * 128) : RowRef{nullptr, nullptr, nullptr};
        if (next.wide) prefetch_row<DG>(next.wide);
#pragma unroll
        for (int gr = 0; gr < DG; ++gr) pairs[gr] = npairs[gr];
        fetch_pairs(next);
      } else if (SRC == kQuery) {
        if (row_live(row, rows, a.q.q_lens, a.q.n, a.q.Hq)) {
          if (a.q.in_fp32) f32 = static_cast<const float*>(a.q.q) + row * D;
          else b16 = static_cast<const __nv_bfloat16*>(a.q.q) + row * D;
        }
      } else if (row_live(row, rows, a.f.q_lens, a.f.n, a.f.Hq)) {
        merged = reinterpret_cast<const __half*>(a.f.acc + row * a.f.ns * D);
        up = a.f.ml[row * a.f.ns * 2];
        if (j + 2 < mine && row + 2 * int64_t(gridDim.x) * 128 < rows)
          prefetch_row<DG>(reinterpret_cast<const __nv_bfloat16*>(merged + 2 * int64_t(gridDim.x) * 128 * a.f.ns * (2 * D)));
      }
      // 16 channels from k on of a float32 query
      auto fetch = [&](int k, float (&x)[16]) {
#pragma unroll
        for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(x + e) = __ldg(reinterpret_cast<const float4*>(f32 + k + e));
      };
      bool finite = true;
      if (b16 || f32) {
        uint32_t m = 0;
        if (b16) {
          uint32_t w = 0;
          const uint4* src = reinterpret_cast<const uint4*>(b16);
#pragma unroll 16
          for (int e = 0; e < D / 8; ++e) {
            const uint4 v = __ldg(src + e);
            w = absmax2(absmax2(absmax2(absmax2(w, v.x), v.y), v.z), v.w);
          }
          m = max(w & 0xFFFFu, w >> 16) << 16;
        } else {
#pragma unroll 1
          for (int k = 0; k < D; k += 16) {
            float x[16];
            fetch(k, x);
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(fabsf(x[e])));
          }
        }
        finite = m < 0x7F800000u;
        const int e = max(-104, min(127, int(m >> 23) - 126)) - 7;  // 2^-e times the row's largest value is just below 2^7
        down = pow2i(-e);
        up = pow2i(e);
      }
      if (SRC == kQuery) {
        if (!finite) status_or(status, OSCAR_DEV_NONFINITE);
        up *= a.q.qscale;
      }
      if (SRC == kRead && ref.codes) {  // as expand_k, always scaled: the largest value is just below 2^13
        float m = 0.f;
#pragma unroll
        for (int gr = 0; gr < DG; ++gr) {
          const float2 sz = __half22float2(pairs[gr]);
          m = fmaxf(m, fmaxf(fabsf(sz.y), fabsf(fmaf(sz.x, g.lm ? kLmSpan : 3.0f, sz.y))));
        }
        const int e = isfinite(m) ? (int(__float_as_uint(m)) >> 23) - 126 - 13 : 1;  // -36 .. 6 for fp16 pairs
        down = m > 0.f ? pow2i(-e) : 0.f;
        up = m > 0.f ? pow2i(e) : 0.f;
      }
      const int acc = j % kAcc;
      if (j >= kAcc) ok = ok && wait(acc_empty + 8 * acc, ((j / kAcc) & 1) ^ 1);
      factor[acc * 128 + r] = up * (1.0f / kMatrixScale);
      __syncwarp();
      mbar_arrive_if(f_full + 8 * acc, lane == 0);
#pragma unroll 1
      for (int kb = 0; ok && kb < 2 * DG; ++kb) {
        const int gr = kb >> 1, half = kb & 1;
        uint32_t w[4];
        float2 sz = make_float2(0.f, 0.f);
        if (SRC == kRead && half == 0) {
          q0 = n0, q1 = n1;
          fetch_codes(gr + 1 < DG ? ref : next, gr + 1 < DG ? gr + 1 : 0);
        }
        if (SRC == kRead && ref.codes) {
#pragma unroll
          for (int j = 0; j < DG; ++j)
            if (j == gr) sz = __half22float2(pairs[j]);
          if (role == 0) {  // word 2 c + half: pair c of every 16-byte chunk
            w[0] = half ? q0.y : q0.x, w[1] = half ? q0.w : q0.z, w[2] = half ? q1.y : q1.x, w[3] = half ? q1.w : q1.z;
          } else {          // words 2 m and 2 m + 1, codes 8 half ..: pair m
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            w[0] = prmt(q0.x, q0.y, sel), w[1] = prmt(q0.z, q0.w, sel), w[2] = prmt(q1.x, q1.y, sel), w[3] = prmt(q1.z, q1.w, sel);
          }
        }
#pragma unroll 1
        for (int set = 0; set < sets; ++set, ++n) {
          const int un = n % PU;
          if (n >= PU) ok = ok && wait(x_empty(p, un), ((n / PU) & 1) ^ 1);
          if (!ok) break;
          uint8_t* dst = sm + L::oX + (p * PU + un) * kUnit + r * 128;
          if (SRC == kRead && ref.codes) {
            if (half == 0 && set == 0)
              *reinterpret_cast<uint2*>(sm + L::oRank + p * kRank + rank_offset(r, 4 * gr)) =
                  rank_key(fmaf(g.lm ? kLmMiddle : 1.0f, sz.x, sz.y) * down);
            const uint32_t s1 = half2_of(sz.x * down, sz.x * down);
            const float unit = sz.x * (down / 150.0f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[4], o[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t y = code_shift(w[c], q);
                v[c] = less_one_even(y);
                o[c] = less_one_odd(y);
                if (!g.lm) {
                  v[c] = hmul2(v[c], s1);
                  o[c] = hmul2(o[c], s1);
                } else {  // (level - middle) s in float32, split
                  v[c] = lm_part(lm_value(v[c]), unit, set);
                  o[c] = lm_part(lm_value(o[c]), unit, set);
                }
              }
              if (set && !g.lm) {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = o[c] = 0u;
              }
              *reinterpret_cast<uint4*>(dst + (((2 * q) ^ (r & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
              *reinterpret_cast<uint4*>(dst + (((2 * q + 1) ^ (r & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else if (SRC == kFinish) {
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              v[q] = merged ? reinterpret_cast<const uint4*>(merged + set * D + 64 * kb)[q] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(dst + ((q ^ (r & 7)) << 4)) = v[q];
          } else if (f32) {
#pragma unroll 1
            for (int q = 0; q < 8; q += 2) {
              float x[16];
              uint32_t hi[8], lo[8];
              fetch(64 * kb + 8 * q, x);
#pragma unroll
              for (int e = 0; e < 8; ++e) split_pair(x[2 * e] * down, x[2 * e + 1] * down, hi[e], lo[e]);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (set) hi[e] = lo[e];
              *reinterpret_cast<uint4*>(dst + ((q ^ (r & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(dst + (((q + 1) ^ (r & 7)) << 4)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
            }
          } else {
            const uint4* src = b16 && !set ? reinterpret_cast<const uint4*>(b16 + 64 * kb) : nullptr;
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = src ? __ldg(src + q) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(dst + ((q ^ (r & 7)) << 4)) =
                  make_uint4(scaled_half2(v[q].x, down), scaled_half2(v[q].y, down), scaled_half2(v[q].z, down), scaled_half2(v[q].w, down));
            if (SRC == kRead && half == 0 && set == 0)
              *reinterpret_cast<uint2*>(sm + L::oRank + p * kRank + rank_offset(r, 4 * gr)) = make_uint2(0, 0);
          }
          fence_async();
          __syncwarp();
          mbar_arrive_if(x_full(p, un), lane == 0);
        }
      }
    }
    if (!ok && lane == 0) fail();
  } else if (warp < kExpandWarps + kStoreWarps) {
    // ----------------------------- scale and store ----------------------------
    const int r = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; ok && j < mine; ++j) {
      const int acc = j % kAcc;
      const int64_t row = (int64_t(blockIdx.x) + int64_t(j) * gridDim.x) * 128 + r;
      bool keep;  // the row is stored
      if (SRC == kRead) {
        keep = row < rows;
        if (keep) {
          const uint32_t bt = fastdiv(uint32_t(row), a.div_hkv), b = fastdiv(bt, a.div_n);
          const int64_t pos = int64_t(a.r.start_pos[b]) + int(bt - b * uint32_t(a.r.n));
          keep = pos >= 0 && pos < min(a.r.seq_lens[b], g.cap);
        }
      } else {
        const int32_t* ql = SRC == kQuery ? a.q.q_lens : a.f.q_lens;
        keep = row_live(row, rows, ql, SRC == kQuery ? a.q.n : a.f.n, SRC == kQuery ? a.q.Hq : a.f.Hq);
      }
      ok = wait(f_full + 8 * acc, (j / kAcc) & 1);
      ok = ok && wait(acc_full + 8 * acc, (j / kAcc) & 1);
      if (!ok) break;
      fence_after();
      const float up = factor[acc * 128 + r];
#pragma unroll 1
      for (int c = 0; c < NC; c += 16) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + acc * kStep + c, v);
        tmem_wait16(v);
#pragma unroll
        for (int part = 1; part < kParts; ++part) {
          uint32_t w[16];
          tmem_ld16(tmem + lanes + acc * kStep + part * NC + c, w);
          tmem_wait16(w);
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(w[e]));
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * up);
        if (!keep) continue;
        if (out32) {
          float* dst = static_cast<float*>(out) + row * D + c0 + c;
          const uint32_t lo[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
          const uint32_t hi[8] = {v[8], v[9], v[10], v[11], v[12], v[13], v[14], v[15]};
          store32(dst, lo, aligned);
          store32(dst + 8, hi, aligned);
        } else {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            h[e] = pack_bf162(__float2bfloat16_rn(__uint_as_float(v[2 * e])), __float2bfloat16_rn(__uint_as_float(v[2 * e + 1])));
          store32(static_cast<__nv_bfloat16*>(out) + row * D + c0 + c, h, aligned);
        }
      }
      fence_before();
      __syncwarp();
      mbar_arrive_if(acc_empty + 8 * acc, lane == 0);
    }
    if (!ok && lane == 0) fail();
  } else {
    // ------------------------------ MMA issuer --------------------------------
    const uint32_t leader = elect_one();
    constexpr uint32_t id = idesc_of(NC, false, false);
    const uint32_t sX = base + L::oX, sB = base + L::oB, sRank = base + L::oRank;
    // D = 512: a tile has more units than a group's buffers hold, so the groups' tiles take turns unit by unit
    constexpr int kTogether = DG == 4 ? 2 : 1;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; ok && j < mine; j += kTogether) {
      const int count = min(kTogether, mine - j);
      if (j >= kAcc)
        for (int q = 0; q < count; ++q) ok = ok && wait(acc_empty + 8 * ((j + q) % kAcc), ((j / kAcc) & 1) ^ 1);
      int used = (j >> 1) * 2 * DG * sets;  // units of the group
#pragma unroll 1
      for (int kb = 0; ok && kb < 2 * DG; ++kb) {
        const uint32_t m = desc_of(sB + kb * (NC * 128), 16);
#pragma unroll 1
        for (int set = 0; ok && set < sets; ++set, ++used) {
          const int un = used % PU;
#pragma unroll 1
          for (int q = 0; q < count; ++q) {
            const int p = (j + q) & 1;
            ok = wait(x_full(p, un), (used / PU) & 1);
            if (!ok) break;
            fence_after();
            const uint32_t d = tmem + (j + q) % kAcc * kStep, large = kParts == 3 && kb >= DG ? d + NC : d,
                           small = d + (kParts - 1) * NC;
            const int done = kParts == 3 ? kb % DG : kb;  // units that the large accumulator has
            const uint32_t x = desc_of(sX + (p * PU + un) * kUnit, 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16_ss(set ? small : large, x + 2 * k, m + 2 * k, id, done | set | k, leader);
            if (RL && set == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_f16_ss(small, x + 2 * k, m + (L::kB >> 4) + 2 * k, id, kb | k, leader);
            }
            if (SRC == kRead && kb == 2 * DG - 2 && set == 0)  // the middles of all groups are there
              mma_f16_ss<kDescRank>(d, rank_desc(sRank + p * kRank), rank_desc(sRank + 2 * kRank), id, 1, leader);
            mma_commit(x_empty(p, un), leader);
          }
        }
      }
      for (int q = 0; ok && q < count; ++q) mma_commit(acc_full + 8 * ((j + q) % kAcc), leader);
    }
    if (!ok && lane == 0) fail();
    mma_commit(drained, leader);  // every product issued is complete before TMEM is freed
    mbar_wait(drained, 0);
    __syncwarp();
  }
  fence_before();
  __syncthreads();
  if (warp == kExpandWarps + kStoreWarps) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols) : "memory");
  }
}

template <int SRC, int DG, bool RL>
int launch(MmArgs& a, int64_t rows, int roles, cudaStream_t stream) {
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!sms[dev]) {
    int n = 0;
    if (cudaFuncSetAttribute(rows_mm_kernel<SRC, DG, RL>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<DG, RL>::kBytes) !=
            cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    sms[dev] = n;
  }
  a.tiles = (rows + 127) / 128;
  a.wait_turns = wait_turns();
  a.wait_poison = g_test_wait_poison;
  const int chunks = DG * 128 / Plan<DG, RL>::NC;
  const int per = int(std::min<int64_t>(a.tiles, std::max(1, sms[dev] / (chunks * roles))));
  return row_launch(SRC == kFinish, rows_mm_kernel<SRC, DG, RL>, dim3(per, chunks, roles), kThreads, Plan<DG, RL>::kBytes, stream, a);
}

template <int SRC, bool RL>
int launch_dim(MmArgs& a, int D, int64_t rows, int roles, cudaStream_t stream) {
  return D == 128 ? launch<SRC, 1, RL>(a, rows, roles, stream) : D == 256 ? launch<SRC, 2, RL>(a, rows, roles, stream)
                                                                          : launch<SRC, 4, RL>(a, rows, roles, stream);
}

}  // namespace

int launch_read_tc(const ReadArgs& r, cudaStream_t stream) {
  MmArgs a{};
  a.r = r;
  a.xl = r.out_fp32 && r.g.lm;
  a.div_hkv = fastdiv_make(uint32_t(r.g.Hkv));
  a.div_n = fastdiv_make(uint32_t(r.n));
  const int64_t rows = int64_t(r.g.B) * r.n * r.g.Hkv;
  const int roles = r.k_out && r.v_out ? 2 : 1;
  return r.out_fp32 ? launch_dim<kRead, true>(a, r.g.D, rows, roles, stream) : launch_dim<kRead, false>(a, r.g.D, rows, roles, stream);
}
int launch_qrot_rows_tc(const QrotRowsArgs& q, cudaStream_t stream) {
  MmArgs a{};
  a.q = q;
  a.xl = q.in_fp32;
  return launch_dim<kQuery, true>(a, q.D, q.rows, 1, stream);
}
int launch_finish_rows_tc(const FinishArgs& f, cudaStream_t stream) {
  MmArgs a{};
  a.f = f;
  a.xl = f.out_fp32;
  return f.out_fp32 ? launch_dim<kFinish, true>(a, f.D, f.rows, 1, stream) : launch_dim<kFinish, false>(a, f.D, f.rows, 1, stream);
}

}  // namespace oscar
