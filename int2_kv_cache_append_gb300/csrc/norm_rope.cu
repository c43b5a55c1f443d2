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
// 64-bit integer product per (token, frequency), exact modulo 2^64.  A warp has a
// token (or shares it with others, if there are few): its lanes' sines, cosines
// and weights stay in registers over all the token's heads.
//
// A row belongs to D / 16 lanes; each lane holds 8 channels of the first and 8 of
// the second half of the rotated channels (and likewise of the rest, if there is
// one), so every pair lies within a lane, and its loads and stores are 16 bytes.
// They are plain loads: a row may be written where it was read.
//
// What bounds it: DRAM (16,384 tokens of 72 heads in bf16, 604 MB: 108 us, 5.57 TB/s,
// 83 % of a copy's rate; float32 190 us, 95 %; the first 64 channels rotated 118 us;
// 36 heads of head_dim 256 110 us); one decode step takes 4 us.
#include <algorithm>

#include "internal.h"

namespace oscar {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

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

// Rows of a warp, each with D / 16 lanes.
template <int D>
constexpr int kRowsOfWarp = 32 / (D / 16);

// ALL: every channel is rotated.  With the question which lanes' are, the first call above takes 116 us instead of 106.5.
template <typename T, int D, bool ALL>
__global__ void __launch_bounds__(kThreads, 3) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 16, RPW = kRowsOfWarp<D>;
  __shared__ uint64_t freq[D / 2];
  __shared__ float2 turns[kWarps][D / 2];  // a warp's token: (cos, sin)
  const int half = a.rot / 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = lane % LPR, sub = lane / LPR;
  // this lane's channels: first .. + 7 and second .. + 7
  const bool rotated = ALL || part < a.rot / 16;
  const int rest = part - a.rot / 16;
  const int first = rotated ? 8 * part : a.rot + 8 * rest;
  const int second = first + (rotated ? half : (D - a.rot) / 2);
  for (int i = threadIdx.x; i < half; i += kThreads) {
    double f = double(__ldg(a.inv_freq + i)) * 0.15915494309189533577;  // 1 / 2 pi: turns per position
    f -= floor(f);
    freq[i] = uint64_t(f * 18446744073709551616.0);
  }
  __syncthreads();
  const int groups_q = (a.Hq + RPW - 1) / RPW, groups = groups_q + (a.Hkv + RPW - 1) / RPW;
  float2* turn = turns[warp];
  // `wpt` warps share a token's heads
  const int per_block = kWarps / a.wpt, share = warp % a.wpt;
  for (int64_t t = int64_t(blockIdx.x) * per_block + warp / a.wpt; t < a.n; t += int64_t(gridDim.x) * per_block) {
    if (half) {
      const int64_t pos = __ldg(a.positions + t);
      __syncwarp();
      for (int i = lane; i < half; i += 32) {
        const uint64_t x = uint64_t(pos) * freq[i];
        float s, c;
        sincospif(float(int32_t(x >> 32)) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns in [-1, 1)
        turn[i] = make_float2(c, s);
      }
      __syncwarp();
    }
    float2 cs[8];  // of the lane's pairs: half: i with first + i; interleaved: first's four, then second's
#pragma unroll
    for (int i = 0; i < 8; ++i)
      cs[i] = !rotated ? make_float2(1.f, 0.f) : a.interleaved ? turn[((i < 4 ? first : second) >> 1) + (i & 3)] : turn[first + i];
    int kind = -1;  // whose weights w holds: 0 queries, 1 keys
    float w[16];
    auto rows = [&](int gi, Vec8<T>& x, Vec8<T>& y) {  // loads; the row's head or -1
      const bool key = gi >= groups_q;
      const int hd = (key ? gi - groups_q : gi) * RPW + sub;
      if (gi >= groups || hd >= (key ? a.Hkv : a.Hq)) return -1;
      const T* src = (key ? static_cast<const T*>(a.k) + t * a.k_stride : static_cast<const T*>(a.q) + t * a.q_stride) + hd * D;
      x.load(src + first), y.load(src + second);
      return hd;
    };
    auto finish = [&](int gi, int hd, const Vec8<T>& x, const Vec8<T>& y) {
      if (gi >= groups) return;
      const int key = gi >= groups_q;
      if (key != kind) {
        kind = key;
        const float4* src = reinterpret_cast<const float4*>(key ? a.k_weight : a.q_weight);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 u = __ldg(src + (first + i) / 4), v = __ldg(src + (second + i) / 4);
          w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
          w[8 + i] = v.x, w[9 + i] = v.y, w[10 + i] = v.z, w[11 + i] = v.w;
        }
      }
      float u[8], v[8];
      x.to(u), y.to(v);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(u[i], u[i], fmaf(v[i], v[i], sum));
#pragma unroll
      for (int m = LPR / 2; m; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      const float f = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] *= f * w[i], v[i] *= f * w[8 + i];
      if (rotated) {  // also a turn by nothing joins what is not finite
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 p = cs[i / 2], q = cs[4 + i / 2];
            const float u0 = u[i], v0 = v[i];
            u[i] = u0 * p.x - u[i + 1] * p.y, u[i + 1] = u[i + 1] * p.x + u0 * p.y;
            v[i] = v0 * q.x - v[i + 1] * q.y, v[i + 1] = v[i + 1] * q.x + v0 * q.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float u0 = u[i];
            u[i] = u0 * cs[i].x - v[i] * cs[i].y, v[i] = v[i] * cs[i].x + u0 * cs[i].y;
          }
        }
      }
      if (hd < 0) return;
      T* dst = key ? static_cast<T*>(a.k_out) + (t * a.Hkv + hd) * D : static_cast<T*>(a.q_out) + (t * a.Hq + hd) * D;
      Vec8<T>::store(dst + first, u), Vec8<T>::store(dst + second, v);
    };
    // two groups' loads under way at a time
    for (int gi = share; gi < groups; gi += 2 * a.wpt) {
      Vec8<T> x0{}, y0{}, x1{}, y1{};
      const int h0 = rows(gi, x0, y0), h1 = rows(gi + a.wpt, x1, y1);
      finish(gi, h0, x0, y0);
      finish(gi + a.wpt, h1, x1, y1);
    }
  }
}

template <typename T, int D>
int launch_d(NormRopeArgs a, int sms, cudaStream_t stream) {
  const int groups = (a.Hq + kRowsOfWarp<D> - 1) / kRowsOfWarp<D> + (a.Hkv + kRowsOfWarp<D> - 1) / kRowsOfWarp<D>;
  // Warps of a token: all eight for few tokens, whose latency counts, one where there are enough to fill the GPU.  us a call with
  // 1 / 2 / 4 / 8 and 40 heads: 8 tokens 9.1 / 6.1 / 5.0 / 4.0, 256 9.1 / 6.4 / 5.0 / 5.0, 1024 9.4 / 7.8 / 10.3 / 11.9, 2048
  // 11.7 / 13.1 / 14.8 / 17.2, 16,384 67 / 76 / 92 / 113.
  a.wpt = 1;
  while (a.wpt < kWarps && int64_t(a.n) * a.wpt < 12 * sms && a.wpt < groups) a.wpt *= 2;
  const int64_t blocks = (int64_t(a.n) * a.wpt + kWarps - 1) / kWarps;
  const auto kernel = a.rot == D ? norm_rope_kernel<T, D, true> : norm_rope_kernel<T, D, false>;
  kernel<<<unsigned(std::min<int64_t>(blocks, 8 * sms)), kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}
template <typename T>
int launch_t(const NormRopeArgs& a, int sms, cudaStream_t stream) {
  return a.D == 128 ? launch_d<T, 128>(a, sms, stream) : a.D == 256 ? launch_d<T, 256>(a, sms, stream) : launch_d<T, 512>(a, sms, stream);
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_LAUNCH;
  return a.fp32 ? launch_t<float>(a, sms, stream) : launch_t<__nv_bfloat16>(a, sms, stream);
}

}  // namespace oscar
