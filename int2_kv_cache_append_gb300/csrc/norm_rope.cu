// qk_norm_rope: root-mean-square norm of every query and key head and the
// rotary position rotation, one pass over the rows.
//
//   y = x / sqrt(mean(x^2) + eps) * w,
//   (a, b) -> (a cos phi - b sin phi, b cos phi + a sin phi),  phi = position * inv_freq[i],
//
// for the pairs (i, i + rot / 2) or (2 i, 2 i + 1) of the first rot channels.
//
// Angles: position * inv_freq exceeds float32 after a few thousand positions (at
// 10^6 its last bit is 0.06), so an angle is counted in turns modulo one, in
// 64-bit fixed point: inv_freq / 2 pi mod 1 once per block in float64, then one
// 64-bit integer product per (token, frequency), exact modulo 2^64.  The tokens'
// sines and cosines lie in shared memory and serve all their heads.
//
// A row belongs to D / 16 lanes; each lane holds 8 channels of the first and 8 of
// the second half of the rotated channels (and likewise of the rest, if there is
// one), so every pair lies within a lane, and its loads and stores are 16 bytes.
// They are plain loads: a row may be written where it was read.
#include <algorithm>

#include "internal.h"

namespace oscar {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec8;  // 8 channels as float32
template <>
struct Vec8<__nv_bfloat16> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void to(float* v) const {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = pack_bf162(__float2bfloat16_rn(v[2 * i]), __float2bfloat16_rn(v[2 * i + 1]));
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <>
struct Vec8<float> {
  float4 x, y;
  __device__ __forceinline__ void load(const float* p) {
    x = *reinterpret_cast<const float4*>(p);
    y = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void to(float* v) const {
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *(reinterpret_cast<float4*>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;  // lanes of a row, rows of a warp
  extern __shared__ float2 turn[];             // [tb][rot / 2] (cos, sin), then the frequencies
  const int half = a.rot / 2, heads = a.Hq + a.Hkv;
  uint64_t* freq = reinterpret_cast<uint64_t*>(turn + a.tb * half);
  const int lane = threadIdx.x & 31, part = lane % LPR;
  // this lane's channels: first .. + 7 and second .. + 7
  const bool rotated = part < a.rot / 16;
  const int rest = part - a.rot / 16;
  const int first = rotated ? 8 * part : a.rot + 8 * rest;
  const int second = first + (rotated ? half : (D - a.rot) / 2);
  for (int i = threadIdx.x; i < half; i += kThreads) {
    double f = double(__ldg(a.inv_freq + i)) * 0.15915494309189533577;  // 1 / 2 pi: turns per position
    f -= floor(f);
    freq[i] = uint64_t(f * 18446744073709551616.0);
  }
  __syncthreads();
  const int groups = (a.n + a.tb - 1) / a.tb;
  for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int t0 = grp * a.tb, tokens = min(a.tb, a.n - t0);
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
      const int64_t pos = __ldg(a.positions + t0 + i / half);
      const uint64_t x = uint64_t(pos) * freq[i % half];
      float s, c;
      sincospif(float(int32_t(x >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns in [-1, 1)
      turn[i] = make_float2(c, s);
    }
    __syncthreads();
    const int rows = tokens * heads;
    for (int r0 = (threadIdx.x >> 5) * RPW; r0 < rows; r0 += kThreads / 32 * RPW) {
      const int r = r0 + lane / LPR;
      const bool live = r < rows;
      const int t = live ? r / heads : 0, hd = live ? r % heads : 0;
      const bool key = hd >= a.Hq;
      const int64_t tok = t0 + t;
      const T* src = key ? static_cast<const T*>(a.k) + tok * a.k_stride + (hd - a.Hq) * D
                         : static_cast<const T*>(a.q) + tok * a.q_stride + hd * D;
      T* dst = key ? static_cast<T*>(a.k_out) + (tok * a.Hkv + (hd - a.Hq)) * D
                   : static_cast<T*>(a.q_out) + (tok * a.Hq + hd) * D;
      Vec8<T> x0, x1;
      if (live) x0.load(src + first), x1.load(src + second);
      float u[8], v[8];
      x0.to(u), x1.to(v);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(u[i], u[i], fmaf(v[i], v[i], sum));
#pragma unroll
      for (int m = LPR / 2; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      const float f = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
      const float4* w = reinterpret_cast<const float4*>(key ? a.k_weight : a.q_weight);
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 wu = __ldg(w + (first + i) / 4), wv = __ldg(w + (second + i) / 4);
        u[i] *= f * wu.x, u[i + 1] *= f * wu.y, u[i + 2] *= f * wu.z, u[i + 3] *= f * wu.w;
        v[i] *= f * wv.x, v[i + 1] *= f * wv.y, v[i + 2] *= f * wv.z, v[i + 3] *= f * wv.w;
      }
      if (rotated) {
        const float2* cs = turn + t * half;
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 p = cs[(first + i) / 2], q = cs[(second + i) / 2];
            const float u0 = u[i], v0 = v[i];
            u[i] = u0 * p.x - u[i + 1] * p.y, u[i + 1] = u[i + 1] * p.x + u0 * p.y;
            v[i] = v0 * q.x - v[i + 1] * q.y, v[i + 1] = v[i + 1] * q.x + v0 * q.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 p = cs[first + i];
            const float u0 = u[i];
            u[i] = u0 * p.x - v[i] * p.y, v[i] = v[i] * p.x + u0 * p.y;
          }
        }
      }
      if (live) Vec8<T>::store(dst + first, u), Vec8<T>::store(dst + second, v);
    }
    __syncthreads();
  }
}

template <typename T>
int launch_t(const NormRopeArgs& a, int blocks, cudaStream_t stream) {
  const size_t smem = size_t(a.tb) * (a.rot / 2) * sizeof(float2) + size_t(a.rot / 2) * sizeof(uint64_t);
  switch (a.D) {
    case 128: norm_rope_kernel<T, 128><<<blocks, kThreads, smem, stream>>>(a); break;
    case 256: norm_rope_kernel<T, 256><<<blocks, kThreads, smem, stream>>>(a); break;
    default: norm_rope_kernel<T, 512><<<blocks, kThreads, smem, stream>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& args, cudaStream_t stream) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_LAUNCH;
  NormRopeArgs a = args;
  const int most = sms * 4;
  a.tb = std::min(4, std::max(1, a.n / most));
  const int blocks = std::min(most, (a.n + a.tb - 1) / a.tb);
  return a.fp32 ? launch_t<float>(a, blocks, stream) : launch_t<__nv_bfloat16>(a, blocks, stream);
}

}  // namespace oscar
