// attn_mass: the attention weight that every cached position receives.
//
//   mass_out[p] = mass_in[p] + sum over query rows r that see p of exp(scale q_r . k_p - lse_r)
//
// for each (sequence, KV head), over the K role of the cache alone.  In the
// rotated basis and log2 units an INT2 key gives
//   s = scale_p (q' . c_p) + zero_p sum(q')   per group of 128 channels.
//
// A thread has one position; the rows' rotated queries lie in shared memory and
// are read by all threads at once.
#include <algorithm>

#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 128;
constexpr int kR = 8;  // query rows per pass over the keys

__global__ void __launch_bounds__(kThreads) attn_mass_kernel(const MassArgs a) {
  extern __shared__ float sm[];
  const Geom& g = a.g;
  float* qs = sm;                 // [D][kR]
  float* qsum = qs + g.D * kR;    // [Dg][kR]
  __shared__ float ref[kR];
  __shared__ int last[kR];
  const int unit = blockIdx.y, b = unit / g.Hkv, h = unit % g.Hkv;
  const int T = max(0, min(a.seq_lens[b], g.cap));
  if (a.seq_lens[b] > g.cap && threadIdx.x == 0 && blockIdx.x == 0) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
  const int p = blockIdx.x * kThreads + threadIdx.x;
  if (blockIdx.x * kThreads >= T) return;
  const int ql = max(0, a.q_lens ? min(a.q_lens[b], a.n) : a.n), rows = ql * g.G;
  const bool live = p < T;
  const RowRef ref_row = row_ref(g, a.layer_base, 0, unit, T, live ? p : 0);
  float mass = 0.f;
  for (int r0 = 0; r0 < rows; r0 += kR) {
    __syncthreads();
    const int n = min(kR, rows - r0);
    for (int i = threadIdx.x; i < g.D * kR; i += kThreads) {
      const int r = i % kR, c = i / kR, row = r0 + r;
      qs[i] = r < n ? a.qrot[(int64_t(b * a.n + row / g.G) * g.Hq + h * g.G + row % g.G) * g.D + c] : 0.f;
    }
    if (threadIdx.x < kR) {
      const int row = r0 + threadIdx.x;
      const bool on = threadIdx.x < n;
      const float x = on ? a.lse[int64_t(b * a.n + row / g.G) * g.Hq + h * g.G + row % g.G] : 0.f;
      ref[threadIdx.x] = x * 1.4426950408889634f;
      last[threadIdx.x] = on && x != -INFINITY ? T - ql + row / g.G : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.Dg * kR; i += kThreads) {
      float x = 0.f;
      for (int c = 0; c < kGroup; ++c) x += qs[((i / kR) * kGroup + c) * kR + i % kR];
      qsum[i] = x;
    }
    __syncthreads();
    float s[kR] = {};
    if (live) {
      if (ref_row.wide) {
        for (int c = 0; c < g.D; c += 2) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(ref_row.wide + c);
          const float k0 = __uint_as_float(x << 16), k1 = __uint_as_float(x & 0xFFFF0000u);
#pragma unroll
          for (int r = 0; r < kR; ++r) s[r] = fmaf(k0, qs[c * kR + r], fmaf(k1, qs[(c + 1) * kR + r], s[r]));
        }
      } else {
        for (int d = 0; d < g.Dg; ++d) {
          const float2 sz = __half22float2(ref_row.sz[d]);
          float dot[kR] = {};
          for (int j = 0; j < 8; ++j) {
            const uint32_t x = ref_row.codes[8 * d + j];
            const float* base = qs + (kGroup * d + 64 * (j & 1) + (j & ~1)) * kR;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = int(x >> (2 * i)) & 3;
              const float level = g.lm ? kLmRho * float(c) + (1.0f - kLmRho) * float(c >> 1) : float(c);
#pragma unroll
              for (int r = 0; r < kR; ++r) dot[r] = fmaf(level, base[(8 * (i & 7) + (i >> 3)) * kR + r], dot[r]);
            }
          }
#pragma unroll
          for (int r = 0; r < kR; ++r) s[r] += fmaf(sz.x, dot[r], sz.y * qsum[d * kR + r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kR; ++r)
      if (p <= last[r]) mass += exp2f(s[r] - ref[r]);
  }
  if (live) {
    const int64_t at = int64_t(unit) * g.cap + p;
    a.mass_out[at] = mass + (a.mass_in ? a.mass_in[at] : 0.f);
  }
}

}  // namespace

int launch_attn_mass(const MassArgs& a, cudaStream_t stream) {
  const int smem = (a.g.D + a.g.Dg) * kR * 4;
  const int64_t units = int64_t(a.g.B) * a.g.Hkv;
  if (units > 65535) return OSCAR_ERR_UNSUPPORTED;
  attn_mass_kernel<<<dim3(unsigned((int64_t(a.g.cap) + kThreads - 1) / kThreads), unsigned(units)), kThreads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace oscar
