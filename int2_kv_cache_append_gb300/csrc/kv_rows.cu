// Row products with a layer's rotation: kv_read (cached rows back into the
// model's basis), the query rotation and the merge + un-rotation of the row
// attention.  All three are X [rows x D] times R or R^T with a different way of
// producing X and storing the result.
//
// A CTA holds 32 rows of X in shared memory (float32) and computes 128 output
// columns in 32-deep chunks of the matrix, 4 x 4 outputs per thread, float32
// FMA throughout.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kRows = 32;     // rows of X per CTA
constexpr int kCols = 128;    // output columns per CTA
constexpr int kDeep = 32;     // matrix rows staged at a time
constexpr int kThreads = 256;
constexpr int kPitch = kCols + 4;

// y[4][4] = X[4 rws + i][:] . M[:][c0 + 4 lane + j] with M = R (trans = false) or R^T.
__device__ __forceinline__ void rows_product(const float* X, int xpitch, const float* __restrict__ R, int D, int c0,
                                             bool trans, bool hadamard, float* Ms, float (&y)[4][4]) {
  const int lane = threadIdx.x & 31, rw = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[i][j] = 0.f;
  for (int k0 = 0; k0 < D; k0 += kDeep) {
    __syncthreads();  // the previous chunk (or X) is complete
    for (int i = threadIdx.x; i < kDeep * kCols; i += kThreads) {
      const int k = trans ? i % kDeep : i / kCols, c = trans ? i / kDeep : i % kCols;
      float v;
      if (hadamard) v = hadamard_at(k0 + k, c0 + c);
      else v = trans ? __ldg(R + int64_t(c0 + c) * D + k0 + k) : __ldg(R + int64_t(k0 + k) * D + c0 + c);
      Ms[k * kPitch + c] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kDeep; k += 4) {
      float x[4][4], m[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float4*>(x[i]) = *reinterpret_cast<const float4*>(X + (4 * rw + i) * xpitch + k0 + k);
        *reinterpret_cast<float4*>(m[i]) = *reinterpret_cast<const float4*>(Ms + (k + i) * kPitch + 4 * lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = fmaf(x[i][e], m[e][j], y[i][j]);
    }
  }
}

__device__ __forceinline__ void store4(void* out, int64_t at, int fp32, const float (&v)[4]) {
  if (fp32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(pack_bf162(__float2bfloat16_rn(v[0]), __float2bfloat16_rn(v[1])),
                   pack_bf162(__float2bfloat16_rn(v[2]), __float2bfloat16_rn(v[3])));
  }
}

// ------------------------------------------------------------------- kv_read
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
  extern __shared__ float sm[];
  const Geom& g = a.g;
  const int D = g.D, role = blockIdx.z, xp = D + 4;
  float* X = sm;
  float* Ms = sm + kRows * xp;
  void* out = role ? a.v_out : a.k_out;
  if (!out) return;
  const int64_t rows = int64_t(g.B) * a.n * g.Hkv, row0 = int64_t(blockIdx.x) * kRows;
  for (int i = threadIdx.x; i < kRows * (D / 16); i += kThreads) {
    const int r = i / (D / 16), w = i % (D / 16);
    const int64_t row = row0 + r;
    bool ok = row < rows;
    if (ok) {
      const int h = int(row % g.Hkv);
      const int64_t bt = row / g.Hkv;
      const int b = int(bt / a.n), t = int(bt % a.n);
      int T = a.seq_lens[b];
      if (T > g.cap) {
        status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
        T = g.cap;
      }
      const int64_t p = int64_t(a.start_pos[b]) + t;
      ok = p >= 0 && p < T;
      if (ok) row_load16(g, row_ref(g, a.layer_base, role, int64_t(b) * g.Hkv + h, T, int(p)), role, w, X + r * xp);
    }
    if (!ok)
      for (int e = 0; e < 16; ++e) X[r * xp + 16 * w + e] = 0.f;
  }
  const int c0 = blockIdx.y * kCols, lane = threadIdx.x & 31, rw = threadIdx.x >> 5;
  float y[4][4];
  if (role && a.absorb_v) {
    __syncthreads();
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) y[i][j] = X[(4 * rw + i) * xp + c0 + 4 * lane + j];
  } else {
    rows_product(X, xp, role ? a.R_V : a.R_K, D, c0, true, a.hadamard != 0, Ms, y);
  }
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * rw + i;
    if (row >= rows) break;
    const int64_t bt = row / g.Hkv;
    const int b = int(bt / a.n);
    const int64_t p = int64_t(a.start_pos[b]) + bt % a.n;
    if (p < 0 || p >= min(a.seq_lens[b], g.cap)) continue;  // left as it was
    store4(out, row * D + c0 + 4 * lane, a.out_fp32, y[i]);
  }
}

// ---------------------------------------------- query rotation and merge, few rows
//
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

// Merge of the partial results, V un-rotation and store.
template <int D>
__global__ void __launch_bounds__(kFewThreads) finish_few_kernel(const FinishArgs a) {
  __shared__ alignas(16) float X[kFew][D];
  __shared__ float red[4 * kFew * 128];
  __shared__ float wgt[kFew][2 * OSCAR_KV_MAX_SPLITS + 1];  // weight of each partial result over the sum
  __shared__ int live[kFew];
  const int64_t row0 = int64_t(blockIdx.x) * kFew;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = a.ns + a.ns2;
  if (a.own_status && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    // an empty cache of its own is not an error when the prefix has positions
    const int32_t st = *a.own_status & ~OSCAR_DEV_EMPTY;
    if (st) status_or(a.status, st);
  }
  if (warp < kFew) {  // a warp per row, a lane per partial result
    const int64_t row = row0 + warp;
    const bool ok = row_live(row, a.rows, a.q_lens, a.n, a.Hq);
    if (lane == 0) live[warp] = ok;
    if (ok) {
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
        if (lane + 32 * j < all) wgt[warp][lane + 32 * j] = m[j] != 0.f ? m[j] * inv : 0.f;
      if (lane == 0) {
        wgt[warp][all] = wo != 0.f ? wo * inv : 0.f;
        if (blockIdx.y == 0) {
          if (sum == 0.f) status_or(a.status, OSCAR_DEV_EMPTY);
          if (a.lse) a.lse[row] = sum != 0.f ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        }
      }
    }
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

// Rows from which the tensor-core kernels take over.
constexpr int64_t kTensorRows = 1024;       // kv_read
constexpr int64_t kTensorRowsQuery = 4096;  // query rotation, merge

size_t smem_of(int D) { return size_t(kRows * (D + 4) + kDeep * kPitch) * 4; }

// Raises the dynamic shared memory limit of kv_read, once per device.
bool ready() {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return false;
  if (done[dev]) return true;
  const int most = int(smem_of(512));
  if (cudaFuncSetAttribute(kv_read_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return false;
  done[dev] = true;
  return true;
}

int launched() { return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH; }

}  // namespace

int launch_read(const ReadArgs& a, cudaStream_t stream) {
  const int64_t tiles = (int64_t(a.g.B) * a.n * a.g.Hkv + kRows - 1) / kRows;
  if (tiles == 0) return OSCAR_OK;
  const int64_t rows = int64_t(a.g.B) * a.n * a.g.Hkv;
  if (rows >= kTensorRows && rows < (int64_t(1) << 31)) return launch_read_tc(a, stream);
  if (tiles >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  if (!ready()) return OSCAR_ERR_LAUNCH;
  kv_read_kernel<<<dim3(unsigned(tiles), a.g.Dg, 2), kThreads, smem_of(a.g.D), stream>>>(a);
  return launched();
}

int launch_qrot_rows(const QrotRowsArgs& a, cudaStream_t stream) {
  if (a.rows >= kTensorRowsQuery) return launch_qrot_rows_tc(a, stream);
  const dim3 grid(unsigned((a.rows + kFew - 1) / kFew), a.D / 128);
  if (a.D == 128) qrot_few_kernel<128><<<grid, kFewThreads, 0, stream>>>(a);
  else if (a.D == 256) qrot_few_kernel<256><<<grid, kFewThreads, 0, stream>>>(a);
  else qrot_few_kernel<512><<<grid, kFewThreads, 0, stream>>>(a);
  return launched();
}

int launch_finish_rows(const FinishArgs& a, cudaStream_t stream) {
  if (a.rows >= kTensorRowsQuery && a.ns <= 8 && a.ns2 <= 8) return launch_finish_rows_tc(a, stream);
  const dim3 grid(unsigned((a.rows + kFew - 1) / kFew), a.D / 128);
  if (a.D == 128) finish_few_kernel<128><<<grid, kFewThreads, 0, stream>>>(a);
  else if (a.D == 256) finish_few_kernel<256><<<grid, kFewThreads, 0, stream>>>(a);
  else finish_few_kernel<512><<<grid, kFewThreads, 0, stream>>>(a);
  return launched();
}

}  // namespace oscar
