// attn_prompt in float32: causal attention of packed prompts over their own K and
// V for float32 inputs or outputs (attn_prompt_tc.cu has bf16 ones).
//
// A block has 64 query rows of one KV head (row r of a sequence is query head
// h G + r mod G of token r / G) and walks the positions 64 at a time: S = Q K^T
// from shared memory, 4 x 4 scores per thread, the online softmax with its row
// statistics in registers, O += P V with 4 rows x D / 16 channels per thread.
// Rows lie in shared memory as in memory, so copies are asynchronous and V's are
// under way while the scores are formed; P takes K's place, so that two blocks of
// head_dim 128 share an SM and cover each other's waits.  The FMA pipes bound it:
// three prompts of up to 333 tokens, 24 heads, 88 us, of which the longest block's
// six tiles are the most (all products at the FMA rate: 24 us).
#include <algorithm>
#include <cfloat>

#include "prompt_items.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64, kTok = 64, kCh = 128;  // rows, positions, channels of a staged slice of K
constexpr int kLdP = kRows + 4;
constexpr int kLdK = kCh + 4;                    // rows 4 floats apart modulo the banks: 16-byte reads of 16 rows meet no bank twice

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf162(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y)),
                                            pack_bf162(__float2bfloat16_rn(v.z), __float2bfloat16_rn(v.w)));
}

// `rows` rows of `channels` (D apart in steps of `step` elements) to shared memory, zeros for those from `live` on; float32 by
// asynchronous copies.
template <int channels, int ld, typename T>
__device__ __forceinline__ void stage(float* to, const T* from, int64_t step, int rows, int live) {
  for (int i = threadIdx.x; i < rows * (channels / 4); i += kThreads) {
    const int r = i / (channels / 4), c = 4 * (i % (channels / 4));
    float* at = to + r * ld + c;
    if (r >= live) {
      *reinterpret_cast<float4*>(at) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else if constexpr (sizeof(T) == 4) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(at)), "l"(from + r * step + c) : "memory");
    } else {
      *reinterpret_cast<float4*>(at) = load4(from + r * step + c);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int groups>
__device__ __forceinline__ void staged() {
  asm volatile("cp.async.wait_group %0;" ::"n"(groups) : "memory");
}

template <typename T, typename U, int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 2 : 1) attn_prompt_kernel(const PromptArgs a) {
  constexpr int kLdQ = D + 4, kVTok = 8192 / D;  // positions of a staged slice of V
  extern __shared__ float sm[];
  float* qs = sm;                    // [kRows][kLdQ], scaled to log2 units
  float* ks = qs + kRows * kLdQ;     // [kTok][kLdK]; then P [kTok][kLdP]
  float* vs = ks + kTok * kLdK;      // [kVTok][D]
  float* ps = ks;
  __shared__ PromptItem shared_item;
  if (threadIdx.x < 32) {
    if (blockIdx.x == 0) prompt_check(a);
    int level = -1;
    const PromptItem it = prompt_item(a, blockIdx.x / a.Hkv, a.G, kRows, level);
    if (threadIdx.x == 0) shared_item = it;
  }
  __syncthreads();
  const PromptItem it = shared_item;
  if (it.b < 0) return;
  const int h = blockIdx.x % a.Hkv, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int row0 = it.tile * kRows, rows = it.len * a.G;
  const int64_t step = int64_t(a.Hkv) * D;
  const T* q = static_cast<const T*>(a.q);
  const T* k = static_cast<const T*>(a.k) + (int64_t(it.start) * a.Hkv + h) * D;
  const T* v = static_cast<const T*>(a.v) + (int64_t(it.start) * a.Hkv + h) * D;
  const int all = row0 / a.G;                                 // every row sees the positions up to this one
  const int end = min(it.len, (row0 + kRows - 1) / a.G + 1);  // and none sees this one
  stage<kCh, kLdK>(ks, k, step, kTok, end);
  auto head_row = [&](int r) { return int64_t(it.start + r / a.G) * a.Hq + h * a.G + r % a.G; };
  for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row0 + r < rows) x = load4(q + head_row(row0 + r) * D + c);
    *reinterpret_cast<float4*>(qs + r * kLdQ + c) = make_float4(x.x * a.qscale, x.y * a.qscale, x.z * a.qscale, x.w * a.qscale);
  }
  int last[4];  // the rows' last visible position
  float m[4], l[4], o[4][D / 16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    last[i] = row0 + 4 * ty + i < rows ? (row0 + 4 * ty + i) / a.G : -1;
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) o[i][j] = 0.f;
  }
  for (int p0 = 0; p0 < end; p0 += kTok) {
    stage<D, D>(vs, v + p0 * step, step, kVTok, end - p0);  // under way while the scores are formed
    float s[4][4] = {};                                     // position tx + 16 j
    for (int c0 = 0; c0 < D; c0 += kCh) {
      if (c0 > 0) {
        __syncthreads();
        stage<kCh, kLdK>(ks, k + p0 * step + c0, step, kTok, end - p0);
        staged<0>();
      } else {
        staged<1>();
      }
      __syncthreads();
      const float *qr = qs + 4 * ty * kLdQ + c0, *kr = ks + tx * kLdK;
#pragma unroll 4
      for (int c = 0; c < kCh; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = *reinterpret_cast<const float4*>(qr + i * kLdQ + c);
          y[i] = *reinterpret_cast<const float4*>(kr + 16 * i * kLdK + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            s[i][j] = fmaf(x[i].w, y[j].w, fmaf(x[i].z, y[j].z, fmaf(x[i].y, y[j].y, fmaf(x[i].x, y[j].x, s[i][j]))));
      }
    }
    const bool masked = p0 + kTok - 1 > all;
    __syncthreads();  // P goes where K was
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p0 + tx + 16 * j > last[i]) s[i][j] = -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float next = fmaxf(fmaxf(m[i], top), -FLT_MAX);  // finite also where nothing is visible
      const float f = exp2f(m[i] - next);
      m[i] = next;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = exp2f(s[i][j] - next);
        sum += s[i][j];
      }
#pragma unroll
      for (int x = 8; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[i] = l[i] * f + sum;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) o[i][j] *= f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4*>(ps + (tx + 16 * j) * kLdP + 4 * ty) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    for (int t0 = 0; t0 < kTok && p0 + t0 < end; t0 += kVTok) {
      if (t0 > 0) {
        __syncthreads();
        stage<D, D>(vs, v + (p0 + t0) * step, step, kVTok, end - p0 - t0);
      }
      staged<0>();
      __syncthreads();
#pragma unroll 2
      for (int t = 0; t < kVTok; ++t) {
        const float4 x = *reinterpret_cast<const float4*>(ps + (t0 + t) * kLdP + 4 * ty);
        const float xr[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(vs + t * D + 64 * c + 4 * tx);
          const float yr[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // a weight of zero does not take away what is not a number: a hidden value is left out
            if (masked && p0 + t0 + t > last[i]) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][4 * c + j] = fmaf(xr[i], yr[j], o[i][4 * c + j]);
          }
        }
      }
    }
    __syncthreads();
    if (p0 + kTok < end) stage<kCh, kLdK>(ks, k + (p0 + kTok) * step, step, kTok, end - p0 - kTok);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (last[i] < 0) continue;
    const int64_t r = head_row(row0 + 4 * ty + i);
    const float inv = 1.0f / l[i];
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(static_cast<U*>(a.out) + r * D + 64 * c + 4 * tx,
             make_float4(o[i][4 * c] * inv, o[i][4 * c + 1] * inv, o[i][4 * c + 2] * inv, o[i][4 * c + 3] * inv));
    if (a.lse && tx == 0) a.lse[r] = (m[i] + log2f(l[i])) * 0.6931471805599453f;
  }
}

template <typename T, typename U, int D>
int launch_d(const PromptArgs& a, cudaStream_t stream) {
  constexpr int smem = (kRows * (D + 4) + kTok * kLdK + 8192) * 4;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_prompt_kernel<T, U, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int64_t items = prompt_items(a, a.G, kRows) * a.Hkv;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_prompt_kernel<T, U, D><<<unsigned(items), kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}
template <typename T, typename U>
int launch_t(const PromptArgs& a, cudaStream_t stream) {
  switch (a.D) {
    case 128: return launch_d<T, U, 128>(a, stream);
    case 256: return launch_d<T, U, 256>(a, stream);
    default: return launch_d<T, U, 512>(a, stream);
  }
}

}  // namespace

int launch_attn_prompt(const PromptArgs& a, cudaStream_t stream) {
  if (a.in_fp32) return a.out_fp32 ? launch_t<float, float>(a, stream) : launch_t<float, __nv_bfloat16>(a, stream);
  return launch_t<__nv_bfloat16, float>(a, stream);
}

}  // namespace oscar
