// Row products with a layer's rotation for few rows: kv_read (cached rows back
// into the model's basis), the query rotation and the merge + un-rotation of the
// row attention, float32 throughout.  X [rows x D] times R or R^T with a
// different way of producing X and storing the result; kv_rows_tc.cu has the
// form for many rows.  What bounds it: the latency of reading R (kv_read of one
// position: 8 us from launch to launch), with more rows the reads of R from the
// L2 cache by every CTA.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace oscar {
namespace {

// A CTA takes kFew rows and 128 output columns with four quarters of the sum
// over the row's channels side by side: 512 threads, thread (column, quarter).
// What counts at these sizes is the latency of reading the matrix, so every
// thread has its D / 4 loads in flight at once and there are as many CTAs as
// the rows give; the quarters meet in shared memory.
constexpr int kFew = 8;
constexpr int kFewThreads = 512;

// y[r] of this thread's column c0 + (tid & 127) for rows 0 .. kFew - 1 of X, returned in the threads of quarter 0.
template <int D, bool trans>
__device__ __forceinline__ void few_product(const float (*X)[D], float* red, const float* __restrict__ R, int c0, bool hadamard,
                                            float (&y)[kFew]) {
  const int c = threadIdx.x & 127, kq = threadIdx.x >> 7;
  constexpr int part = D / 4;
#pragma unroll
  for (int r = 0; r < kFew; ++r) y[r] = 0.f;
#pragma unroll 1
  for (int k0 = kq * part; k0 < (kq + 1) * part; k0 += 32) {
    float m[32];
    if (hadamard) {
#pragma unroll
      for (int k = 0; k < 32; ++k) m[k] = hadamard_at(k0 + k, c0 + c);
    } else if (trans) {
#pragma unroll
      for (int k = 0; k < 32; k += 4)
        *reinterpret_cast<float4*>(m + k) = __ldg(reinterpret_cast<const float4*>(R + int64_t(c0 + c) * D + k0 + k));
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) m[k] = __ldg(R + int64_t(k0 + k) * D + c0 + c);
    }
#pragma unroll
    for (int r = 0; r < kFew; ++r)
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&X[r][k0 + k]);
        y[r] = fmaf(x.x, m[k], fmaf(x.y, m[k + 1], fmaf(x.z, m[k + 2], fmaf(x.w, m[k + 3], y[r]))));
      }
  }
#pragma unroll
  for (int r = 0; r < kFew; ++r) red[(kq * kFew + r) * 128 + c] = y[r];
  __syncthreads();
  if (kq == 0) {
#pragma unroll
    for (int r = 0; r < kFew; ++r)
      y[r] = (red[r * 128 + c] + red[(kFew + r) * 128 + c]) + (red[(2 * kFew + r) * 128 + c] + red[(3 * kFew + r) * 128 + c]);
  }
}

__device__ __forceinline__ void store1(void* out, int64_t at, int fp32, float v) {
  if (fp32) static_cast<float*>(out)[at] = v;
  else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
}

template <int D>
__global__ void __launch_bounds__(kFewThreads) qrot_few_kernel(const QrotRowsArgs a) {
  __shared__ alignas(16) float X[kFew][D];
  __shared__ float red[4 * kFew * 128];
  const int64_t row0 = int64_t(blockIdx.x) * kFew;
  pdl_trigger();
  if (a.zero_word && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.zero_word = 0;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < kFew * D / kFewThreads; ++i) {
    const int at = threadIdx.x + i * kFewThreads, r = at / D, c = at % D;
    float v = 0.f;
    if (row_live(row0 + r, a.rows, a.q_lens, a.n, a.Hq)) {
      const int64_t src = (row0 + r) * D + c;
      v = a.in_fp32 ? static_cast<const float*>(a.q)[src] : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[src]);
      finite &= isfinite(v) != 0;
    }
    X[r][c] = v;
  }
  if (!finite) status_or(a.status, OSCAR_DEV_NONFINITE);
  __syncthreads();
  float y[kFew];
  few_product<D, false>(X, red, a.R_K, blockIdx.y * 128, a.hadamard != 0, y);
  if (threadIdx.x < 128)
#pragma unroll
    for (int r = 0; r < kFew; ++r)
      if (row0 + r < a.rows) a.qrot[(row0 + r) * D + blockIdx.y * 128 + threadIdx.x] = y[r] * a.qscale;
}

// kv_read: cached rows back into the model's basis.
template <int D>
__global__ void __launch_bounds__(kFewThreads) read_few_kernel(const ReadArgs a) {
  __shared__ alignas(16) float X[kFew][D];
  __shared__ float red[4 * kFew * 128];
  __shared__ int live[kFew];
  const Geom& g = a.g;
  const int role = blockIdx.z;
  void* out = role ? a.v_out : a.k_out;
  if (!out) return;
  const int64_t rows = int64_t(g.B) * a.n * g.Hkv, row0 = int64_t(blockIdx.x) * kFew;
  for (int i = threadIdx.x; i < kFew * (D / 16); i += kFewThreads) {
    const int r = i / (D / 16), w = i % (D / 16);
    const int64_t row = row0 + r;
    bool ok = row < rows;
    if (ok) {
      const int64_t bt = row / g.Hkv;
      const int b = int(bt / a.n);
      int T = a.seq_lens[b];
      if (T > g.cap) {
        status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
        T = g.cap;
      }
      const int64_t p = int64_t(a.start_pos[b]) + bt % a.n;
      ok = p >= 0 && p < T;
      if (ok) row_load16(g, row_ref(g, a.layer_base, role, int64_t(b) * g.Hkv + row % g.Hkv, T, int(p)), role, w, X[r]);
    }
    if (!ok)
      for (int e = 0; e < 16; ++e) X[r][16 * w + e] = 0.f;
    if (w == 0) live[r] = ok;  // other rows are left as they were
  }
  __syncthreads();
  const int c0 = blockIdx.y * 128;
  float y[kFew];
  if (role && a.absorb_v) {
    if (threadIdx.x < 128)
#pragma unroll
      for (int r = 0; r < kFew; ++r) y[r] = X[r][c0 + threadIdx.x];
  } else {
    few_product<D, true>(X, red, role ? a.R_V : a.R_K, c0, a.hadamard != 0, y);
  }
  if (threadIdx.x < 128)
#pragma unroll
    for (int r = 0; r < kFew; ++r)
      if (live[r]) store1(out, (row0 + r) * D + c0 + threadIdx.x, a.out_fp32, y[r]);
}

// Weights of a row's partial results over their sum, by a warp, a lane per partial result; the row's log-sum-exp.
__device__ __forceinline__ void row_weights(const FinishArgs& a, int64_t row, int lane, bool report, float* wgt) {
  const int all = a.ns + a.ns2;
        float m[4], l[4], top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int s = lane + 32 * j;
          float2 p = make_float2(-INFINITY, 0.f);
          if (s < a.ns) p = *reinterpret_cast<const float2*>(a.ml + (row * a.ns + s) * 2);
          else if (s < all) p = *reinterpret_cast<const float2*>(a.ml2 + (row * a.ns2 + s - a.ns) * 2);
          m[j] = p.x;
          l[j] = p.y;
          if (l[j] != 0.f) top = fmax_nan(top, m[j]);
        }
        const float ol = a.own_lse ? a.own_lse[row] * 1.4426950408889634f : -INFINITY;
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmax_nan(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmax_nan(top, ol);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m[j] = l[j] != 0.f ? exp2f(m[j] - top) : 0.f;
          sum += m[j] * l[j];
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        const float wo = ol != -INFINITY ? exp2f(ol - top) : 0.f;
        sum += wo;
        const float inv = sum != 0.f ? 1.0f / sum : 0.f;
        // a partial result without weight is not read, also where another one made the sum NaN
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (lane + 32 * j < all) wgt[lane + 32 * j] = m[j] != 0.f ? m[j] * inv : 0.f;
        if (lane == 0) {
          wgt[all] = wo != 0.f ? wo * inv : 0.f;
          if (report) {
            if (sum == 0.f) status_or(a.status, OSCAR_DEV_EMPTY);
            if (a.lse) a.lse[row] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
          }
        }
}
__device__ __forceinline__ void own_status(const FinishArgs& a) {
  // an empty cache of its own is not an error when the prefix has positions
  const int32_t st = a.own_status ? *a.own_status & ~OSCAR_DEV_EMPTY : 0;
  if (st) status_or(a.status, st);
}

// Merge of the partial results, V un-rotation and store.
template <int D>
__global__ void __launch_bounds__(kFewThreads) finish_few_kernel(const FinishArgs a) {
  __shared__ alignas(16) float X[kFew][D];
  __shared__ float red[4 * kFew * 128];
  __shared__ float wgt[kFew][2 * OSCAR_KV_MAX_SPLITS + 1];  // weight of each partial result over the sum
  __shared__ int live[kFew];
  const int64_t row0 = int64_t(blockIdx.x) * kFew;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = a.ns + a.ns2;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) own_status(a);
  if (warp < kFew) {  // a warp per row, a lane per partial result
    const int64_t row = row0 + warp;
    const bool ok = row_live(row, a.rows, a.q_lens, a.n, a.Hq);
    if (lane == 0) live[warp] = ok;
    if (ok) row_weights(a, row, lane, blockIdx.y == 0, wgt[warp]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kFew * (D / 4); i += kFewThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live[r]) {
      const int64_t row = row0 + r;
      auto add = [&](const float* src, float w) {
        if (w == 0.f) return;
        const float4 x = *reinterpret_cast<const float4*>(src + c);
        v.x = fmaf(w, x.x, v.x);
        v.y = fmaf(w, x.y, v.y);
        v.z = fmaf(w, x.z, v.z);
        v.w = fmaf(w, x.w, v.w);
      };
#pragma unroll 4
      for (int s = 0; s < a.ns; ++s) add(a.acc + (row * a.ns + s) * D, wgt[r][s]);
#pragma unroll 4
      for (int s = 0; s < a.ns2; ++s) add(a.acc2 + (row * a.ns2 + s) * D, wgt[r][a.ns + s]);
      if (a.own_o) add(a.own_o + row * D, wgt[r][all]);
    }
    *reinterpret_cast<float4*>(&X[r][c]) = v;
  }
  __syncthreads();
  const int c0 = blockIdx.y * 128;
  float y[kFew];
  if (a.absorb_v) {
    if (threadIdx.x < 128)
#pragma unroll
      for (int r = 0; r < kFew; ++r) y[r] = X[r][c0 + threadIdx.x];
  } else {
    few_product<D, true>(X, red, a.R_V, c0, a.hadamard != 0, y);
  }
  if (threadIdx.x < 128)
#pragma unroll
    for (int r = 0; r < kFew; ++r)
      if (live[r]) store1(a.out, (row0 + r) * D + c0 + threadIdx.x, a.out_fp32, y[r]);
}

// The merge alone, for the tensor-core un-rotation: a warp per row.  The merged row goes over the row's first partial
// result, scaled by a power of two to just below 2^7, as fp16 values and their rounding residues; the factor that undoes
// the scaling over its maximum.
constexpr int kMergeRows = 8;
template <int DG>
__global__ void __launch_bounds__(32 * kMergeRows) merge_kernel(const FinishArgs a) {
  constexpr int D = 128 * DG;
  __shared__ float weights[kMergeRows][2 * OSCAR_KV_MAX_SPLITS + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = a.ns + a.ns2;
  const int64_t row = int64_t(blockIdx.x) * kMergeRows + warp;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && threadIdx.x == 0) own_status(a);
  if (!row_live(row, a.rows, a.q_lens, a.n, a.Hq)) return;
  float* wgt = weights[warp];
  float* first = a.acc + row * a.ns * D;
  float4 v[DG];
#pragma unroll
  for (int j = 0; j < DG; ++j) v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float* src, float w) {
    if (w == 0.f) return;
#pragma unroll
    for (int j = 0; j < DG; ++j) {
      const float4 x = reinterpret_cast<const float4*>(src)[lane + 32 * j];
      v[j].x = fmaf(w, x.x, v[j].x);
      v[j].y = fmaf(w, x.y, v[j].y);
      v[j].z = fmaf(w, x.z, v[j].z);
      v[j].w = fmaf(w, x.w, v[j].w);
    }
  };
  if (all == 1 && !a.own_o) {  // one partial result: nothing to weigh, its loads go out at once
    const float2 p = *reinterpret_cast<const float2*>(a.ml + row * 2);
#pragma unroll
    for (int j = 0; j < DG; ++j) v[j] = reinterpret_cast<const float4*>(first)[lane + 32 * j];
    const float w = exp2f(p.x - p.x) / p.y;  // 1 / p.y, or NaN
#pragma unroll
    for (int j = 0; j < DG; ++j)
      v[j] = p.y != 0.f ? make_float4(v[j].x * w, v[j].y * w, v[j].z * w, v[j].w * w) : make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane == 0) {
      if (p.y == 0.f) status_or(a.status, OSCAR_DEV_EMPTY);
      if (a.lse) a.lse[row] = p.y != 0.f ? (p.x + log2f(p.y)) * 0.6931471805599453f : -INFINITY;
    }
  } else {
    row_weights(a, row, lane, true, wgt);
    __syncwarp();
#pragma unroll 4
    for (int s = 0; s < a.ns; ++s) add(first + int64_t(s) * D, wgt[s]);
#pragma unroll 4
    for (int s = 0; s < a.ns2; ++s) add(a.acc2 + (row * a.ns2 + s) * D, wgt[a.ns + s]);
    if (a.own_o) add(a.own_o + row * D, wgt[all]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < DG; ++j)
    m = max(max(max(max(m, __float_as_uint(fabsf(v[j].x))), __float_as_uint(fabsf(v[j].y))), __float_as_uint(fabsf(v[j].z))),
            __float_as_uint(fabsf(v[j].w)));
  m = __reduce_max_sync(0xffffffffu, m);  // also: every lane has read the first partial result
  const int e = max(-104, min(127, int(m >> 23) - 126)) - 7;
  const float down = pow2i(-e);
#pragma unroll
  for (int j = 0; j < DG; ++j) {
    const float x[4] = {v[j].x * down, v[j].y * down, v[j].z * down, v[j].w * down};
    __half hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      hi[q] = __float2half_rn(x[q]);
      lo[q] = __float2half_rn(x[q] - __half2float(hi[q]));
    }
    reinterpret_cast<uint2*>(first)[lane + 32 * j] = *reinterpret_cast<const uint2*>(hi);
    if (a.out_fp32) reinterpret_cast<uint2*>(first + D / 2)[lane + 32 * j] = *reinterpret_cast<const uint2*>(lo);
  }
  if (lane == 0) a.ml[row * a.ns * 2] = pow2i(e);
}

// Sizes from which the tensor-core kernels take over.  The others' time grows with rows x D^2, these have a fixed part of
// 9 / 20 / 20 us (kv_read at D = 128 / 256 / 512), 10 / 15 / 19 us (query rotation).  kv_read of 512 / 1024 / 2048 rows of
// D = 128: 6.2 / 9.4 / 17.3 us against 8.5 / 8.6 / 8.7 us; of 256 / 512 rows of D = 512: 30 / 59 us against 20 us.  Query
// rotation of 1024 / 4096 rows of D = 128: 4.3 / 9.6 us against 10.2 us, of 256 / 1024 rows of D = 512: 11 / 39 us against 19 us.
constexpr int64_t kTensorRead = int64_t(1) << 17;   // rows x D
constexpr int64_t kTensorQuery = int64_t(3) << 25;  // rows x D^2, also of the merge

int launched() { return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH; }

}  // namespace

int launch_read(const ReadArgs& a, cudaStream_t stream) {
  const int64_t rows = int64_t(a.g.B) * a.n * a.g.Hkv, tiles = (rows + kFew - 1) / kFew;
  if (rows == 0) return OSCAR_OK;
  if (rows * a.g.D >= kTensorRead && rows < (int64_t(1) << 31)) return launch_read_tc(a, stream);
  if (tiles >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  const dim3 grid(unsigned(tiles), a.g.Dg, 2);
  if (a.g.D == 128) read_few_kernel<128><<<grid, kFewThreads, 0, stream>>>(a);
  else if (a.g.D == 256) read_few_kernel<256><<<grid, kFewThreads, 0, stream>>>(a);
  else read_few_kernel<512><<<grid, kFewThreads, 0, stream>>>(a);
  return launched();
}

int launch_qrot_rows(const QrotRowsArgs& a, cudaStream_t stream) {
  if (a.rows * a.D * a.D >= kTensorQuery) return launch_qrot_rows_tc(a, stream);
  const dim3 grid(unsigned((a.rows + kFew - 1) / kFew), a.D / 128);
  if (a.D == 128) qrot_few_kernel<128><<<grid, kFewThreads, 0, stream>>>(a);
  else if (a.D == 256) qrot_few_kernel<256><<<grid, kFewThreads, 0, stream>>>(a);
  else qrot_few_kernel<512><<<grid, kFewThreads, 0, stream>>>(a);
  return launched();
}

int launch_finish_rows(const FinishArgs& a, cudaStream_t stream) {
  if (a.rows * a.D * a.D >= kTensorQuery) {
    const dim3 blocks(unsigned((a.rows + kMergeRows - 1) / kMergeRows));
    const auto kernel = a.D == 128 ? merge_kernel<1> : a.D == 256 ? merge_kernel<2> : merge_kernel<4>;
    const int rc = row_launch(a.dependent, kernel, blocks, 32 * kMergeRows, 0, stream, a);
    return rc == OSCAR_OK ? launch_finish_rows_tc(a, stream) : rc;
  }
  const dim3 grid(unsigned((a.rows + kFew - 1) / kFew), a.D / 128);
  const auto kernel = a.D == 128 ? finish_few_kernel<128> : a.D == 256 ? finish_few_kernel<256> : finish_few_kernel<512>;
  return row_launch(a.dependent, kernel, grid, kFewThreads, 0, stream, a);
}

}  // namespace oscar
