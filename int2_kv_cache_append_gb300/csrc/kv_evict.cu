// kv_evict: the cached positions of largest mass, and the windows, into another
// cache.
//
// With T the length, S the sink and W the window, the body [S, max(S, T - W)) of
// a (sequence, KV head) keeps its min(keep, body) rows of largest mass, the lower
// position first among equal ones, in order of position; sink and window stay.
// Two kernels:
//
//   select  one block per (sequence, KV head): the smallest kept key by four
//           8-bit histogram passes over the masses (as integers that order as the
//           numbers do), then the list of the kept positions by block-wide sums;
//   gather  the rows of every new position: a position of the new cache is a sink
//           row, a listed one, or one of the window moved down by what is gone.
#include <algorithm>

#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kGatherThreads = 256;
constexpr int kChunk = 64;  // new positions per gather block

// Integers in the order of the numbers; -0 as 0, what is not a number below all.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (!(x == x)) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Span {
  int T, body, held, gone;  // length, body positions, those kept, those dropped
};
__device__ __forceinline__ Span span_of(const EvictArgs& a, int T) {
  Span s;
  s.T = T;
  s.body = T > a.g.S ? max(0, T - a.g.W - a.g.S) : 0;
  s.held = min(s.body, a.keep);
  s.gone = s.body - s.held;
  return s;
}

__device__ __forceinline__ int block_exclusive(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return sum - x + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[256], sums[32];
  __shared__ uint32_t pick;
  __shared__ int left;
  const int unit = blockIdx.x, b = unit / a.g.Hkv;
  const int given = a.seq_lens[b], T = max(0, min(given, a.g.cap));
  if (unit % a.g.Hkv == 0 && threadIdx.x == 0) {
    if (given > a.g.cap) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
    a.lens[b] = T;
  }
  const Span s = span_of(a, T);
  int32_t* list = a.list + int64_t(unit) * a.list_cap;
  int32_t* kept = a.kept ? a.kept + int64_t(unit) * a.keep : nullptr;
  if (kept)
    for (int i = s.held + threadIdx.x; i < a.keep; i += kSelThreads) kept[i] = -1;
  if (s.held == 0) return;
  const float* mass = a.mass + int64_t(unit) * a.g.cap + a.g.S;
  if (s.gone == 0) {
    for (int i = threadIdx.x; i < s.held; i += kSelThreads) {
      list[i] = a.g.S + i;
      if (kept) kept[i] = a.g.S + i;
    }
    return;
  }
  uint32_t prefix = 0, mask = 0;
  int need = s.held;  // kept ones among the keys with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < s.body; i += kSelThreads) {
      const uint32_t key = mass_key(mass[i]);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int n = need, d = 255;
      while (n > hist[d]) n -= hist[d--];
      pick = uint32_t(d);
      left = n;
    }
    __syncthreads();
    prefix |= pick << shift;
    mask |= 255u << shift;
    need = left;
    __syncthreads();
  }
  // keys above the prefix, and the first `need` equal to it
  int at = 0, equal = 0;
  for (int i0 = 0; i0 < s.body; i0 += kSelThreads) {
    const int i = i0 + threadIdx.x;
    const uint32_t key = i < s.body ? mass_key(mass[i]) : 0u;
    const bool above = i < s.body && key > prefix, same = i < s.body && key == prefix;
    int total;
    const int before = block_exclusive(int(same), sums, total);
    const bool take = above || (same && equal + before < need);
    equal += total;
    const int slot = block_exclusive(int(take), sums, total);
    if (take) {
      list[at + slot] = a.g.S + i;
      if (kept) kept[at + slot] = a.g.S + i;
    }
    at += total;
  }
}

__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  __shared__ int old_of[kChunk];
  const Geom &g = a.g, &og = a.og;
  const int unit = blockIdx.y, b = unit / g.Hkv;
  const Span s = span_of(a, a.lens[b]);
  const int T = s.T - s.gone;  // the new length
  if (unit % g.Hkv == 0 && blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[b] = T;
  const int p0 = blockIdx.x * kChunk;
  const int32_t* list = a.list + int64_t(unit) * a.list_cap;
  const int n = min(kChunk, T - p0);
  if (threadIdx.x < kChunk) {
    const int p = p0 + threadIdx.x;
    const int old = p < g.S || p >= T ? p : p < g.S + s.held ? list[p - g.S] : p + s.gone;
    old_of[threadIdx.x] = old;
    if (a.out_mass && p < og.cap)
      a.out_mass[int64_t(unit) * og.cap + p] = p < T ? a.mass[int64_t(unit) * g.cap + old] : 0.f;
  }
  if (n <= 0) return;
  __syncthreads();
  const int row16 = g.D / 8, code16 = g.D / 64;  // 16-byte pieces of a BF16 and of a code row
  for (int role = 0; role < 2; ++role) {
    const uint8_t* src = a.base + (role ? g.role_bytes : 0);
    uint8_t* dst = a.out_base + (role ? og.role_bytes : 0);
    if (role && g.vb) {
      const uint4* in = reinterpret_cast<const uint4*>(src) + int64_t(unit) * g.cap * row16;
      uint4* out = reinterpret_cast<uint4*>(dst) + (int64_t(unit) * og.cap + p0) * row16;
      for (int i = threadIdx.x; i < n * row16; i += kGatherThreads)
        out[i] = __ldg(in + int64_t(old_of[i / row16]) * row16 + i % row16);
      continue;
    }
    for (int i = threadIdx.x; i < n * row16; i += kGatherThreads) {  // the windows
      const int j = i / row16, p = p0 + j, c = i % row16;
      if (p < g.S) {
        const int64_t at = (int64_t(unit) * g.S + p) * row16 + c;
        reinterpret_cast<uint4*>(dst)[at] = __ldg(reinterpret_cast<const uint4*>(src) + at);
      } else if (p >= T - g.W) {
        const int64_t from = (int64_t(unit) * g.W + old_of[j] % g.W) * row16 + c, to = (int64_t(unit) * g.W + p % g.W) * row16 + c;
        reinterpret_cast<uint4*>(dst + og.sink_bytes)[to] = __ldg(reinterpret_cast<const uint4*>(src + g.sink_bytes) + from);
      }
    }
    const uint8_t* in = src + g.sink_bytes + g.ring_bytes;
    uint8_t* out = dst + og.sink_bytes + og.ring_bytes;
    for (int i = threadIdx.x; i < n * code16; i += kGatherThreads) {
      const int j = i / code16, p = p0 + j, c = i % code16;
      if (p < g.S) continue;
      reinterpret_cast<uint4*>(out)[(int64_t(unit) * og.ncap + p - g.S) * code16 + c] =
          __ldg(reinterpret_cast<const uint4*>(in) + (int64_t(unit) * g.ncap + old_of[j] - g.S) * code16 + c);
    }
    for (int i = threadIdx.x; i < n * g.Dg; i += kGatherThreads) {
      const int j = i / g.Dg, p = p0 + j, c = i % g.Dg;
      if (p < g.S) continue;
      reinterpret_cast<uint32_t*>(out + og.codes_bytes)[(int64_t(unit) * og.ncap + p - g.S) * g.Dg + c] =
          __ldg(reinterpret_cast<const uint32_t*>(in + g.codes_bytes) + (int64_t(unit) * g.ncap + old_of[j] - g.S) * g.Dg + c);
    }
  }
}

}  // namespace

int launch_kv_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t units = int64_t(a.g.B) * a.g.Hkv;
  if (units > 65535) return OSCAR_ERR_UNSUPPORTED;
  evict_select_kernel<<<unsigned(units), kSelThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return OSCAR_ERR_LAUNCH;
  evict_gather_kernel<<<dim3(unsigned((a.og.cap + kChunk - 1) / kChunk), unsigned(units)), kGatherThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace oscar
