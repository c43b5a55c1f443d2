// kv_evict: the cached positions of largest mass, and the windows, into another
// cache.
//
// With T the length, S the sink and W the window, the body [S, max(S, T - W)) of
// a (sequence, KV head) keeps its min(keep, body) rows of largest mass, the lower
// position first among equal ones, in order of position; sink and window stay.
// Two kernels:
//
//   select  one cluster of blocks per (sequence, KV head): the smallest kept key by
//           three histogram passes over the masses (as integers that order as the
//           numbers do; 11, 11 and 10 bits), which stay in shared memory after the
//           first, the blocks' bins added through
//           distributed shared memory; then every warp counts and lists the kept
//           ones of a contiguous piece;
//   gather  the rows of every new position: a position of the new cache is a sink
//           row, a listed one, or one of the window moved down by what is gone.
//           (32 ragged sequences of 32K to 4096 positions, 8 KV heads: selection 45 us,
//           most of it instructions; gather 60 us, 5.8 TB/s; 8 heads of 65,536 positions at
//           head_dim 512 30 and 45 us).
//           Blocks of 128 positions issue all their loads before the first store;
//           the windows' BF16 rows have blocks of their own.
#include <cooperative_groups.h>

#include <algorithm>

#include "rows.cuh"

namespace cg = cooperative_groups;

namespace oscar {
namespace {

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;        // 11 bits of a key
constexpr int kLoads = 4;          // masses of a thread under way
constexpr int kHeld = 24 * 1024;   // keys of a block that stay in shared memory, read once; two blocks to an SM
constexpr int kMostCluster = 4;
constexpr int kGatherThreads = 256;
constexpr int kBody = 128;         // new positions of a gather block
constexpr int kWide = 32;          // window rows of one

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

// x summed over the threads before this one
__device__ __forceinline__ int block_exclusive(int x, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
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
  return sum - x + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const EvictArgs a) {
  __shared__ int hist[kBins], sums[kSelWarps], above_of[kSelWarps], same_of[kSelWarps];
  __shared__ int pick, left, totals[2];
  extern __shared__ uint32_t held[];
  const cg::cluster_group cluster = cg::this_cluster();
  const int size = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int unit = blockIdx.x / size, b = unit / a.g.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int given = a.seq_lens[b], T = max(0, min(given, a.g.cap));
  if (rank == 0 && unit % a.g.Hkv == 0 && threadIdx.x == 0) {
    if (given > a.g.cap) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
    a.lens[b] = T;
  }
  const Span s = span_of(a, T);
  int32_t* list = a.list + int64_t(unit) * a.list_cap;
  int32_t* kept = a.kept ? a.kept + int64_t(unit) * a.keep : nullptr;
  const int first = rank * kSelThreads + threadIdx.x, step = size * kSelThreads;
  if (kept)
    for (int64_t i = int64_t(s.held) + first; i < a.keep; i += step) kept[i] = -1;
  if (s.held == 0) return;
  if (s.gone == 0) {
    for (int i = first; i < s.held; i += step) {
      list[i] = a.g.S + i;
      if (kept) kept[i] = a.g.S + i;
    }
    return;
  }
  const float* mass = a.mass + int64_t(unit) * a.g.cap + a.g.S;
  const int part = (s.body + size - 1) / size, lo = min(s.body, rank * part), hi = min(s.body, lo + part);
  auto key_at = [&](int i) { return i - lo < kHeld ? held[i - lo] : mass_key(__ldg(mass + i)); };
  uint32_t prefix = 0, mask = 0;
  int need = s.held;  // kept ones among the keys with this prefix
#pragma unroll 1
  for (int round = 0; round < 3; ++round) {
    const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += kLoads * kSelThreads) {
      uint32_t key[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int at = i + u * kSelThreads;
        key[u] = at >= hi ? 0u : round ? key_at(at) : mass_key(__ldg(mass + at));
      }
      if (round == 0) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const int at = i + u * kSelThreads;
          if (at < hi && at - lo < kHeld) held[at - lo] = key[u];
        }
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        if (i + u * kSelThreads < hi && (key[u] & mask) == prefix) atomicAdd(&hist[(key[u] >> shift) & ((1u << bits) - 1)], 1);
    }
    cluster.sync();
    // bins from the largest keys down: which one has the last that is kept
    int n[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 2; ++e)
      for (int c = 0; c < size; ++c) n[e] += cluster.map_shared_rank(hist, c)[kBins - 1 - (2 * int(threadIdx.x) + e)];
    int before = block_exclusive(n[0] + n[1], sums);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < need && need <= before + n[e]) {
        pick = kBins - 1 - (2 * int(threadIdx.x) + e);
        left = need - before;
      }
      before += n[e];
    }
    cluster.sync();  // also: nobody reads these bins any more
    prefix |= uint32_t(pick) << shift;
    mask |= ((1u << bits) - 1) << shift;
    need = left;
  }
  // keys above the prefix, and the first `need` equal to it: counted warp by warp, then listed
  const int piece = (hi - lo + kSelWarps - 1) / kSelWarps, w0 = min(hi, lo + warp * piece), w1 = min(hi, w0 + piece);
  int above = 0, same = 0;
  for (int i = w0 + lane; i < w1; i += kLoads * 32) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const uint32_t key = i + 32 * u < w1 ? key_at(i + 32 * u) : 0u;
      above += i + 32 * u < w1 && key > prefix;
      same += i + 32 * u < w1 && key == prefix;
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  same = __reduce_add_sync(0xffffffffu, same);
  if (lane == 0) above_of[warp] = above, same_of[warp] = same;
  __syncthreads();
  if (warp == 0) {
    const int x = __reduce_add_sync(0xffffffffu, above_of[lane]), y = __reduce_add_sync(0xffffffffu, same_of[lane]);
    if (lane == 0) totals[0] = x, totals[1] = y;
  }
  cluster.sync();
  above = same = 0;
  for (int c = 0; c < rank; ++c) above += cluster.map_shared_rank(totals, c)[0], same += cluster.map_shared_rank(totals, c)[1];
  for (int w = 0; w < warp; ++w) above += above_of[w], same += same_of[w];
  const unsigned before = (1u << lane) - 1;
#pragma unroll 1
  for (int i0 = w0; i0 < w1; i0 += kLoads * 32) {
    uint32_t key[kLoads];
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = i0 + 32 * u + lane;
      key[u] = i < w1 ? key_at(i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      const int i = i0 + 32 * u + lane;
      const unsigned is_above = __ballot_sync(0xffffffffu, i < w1 && key[u] > prefix);
      const unsigned is_same = __ballot_sync(0xffffffffu, i < w1 && key[u] == prefix);
      const int x = above + __popc(is_above & before), y = same + __popc(is_same & before);
      const bool mine = (is_above >> lane & 1) || ((is_same >> lane & 1) && y < need);
      if (mine) {
        const int slot = x + min(y, need);
        list[slot] = a.g.S + i;
        if (kept) kept[slot] = a.g.S + i;
      }
      above += __popc(is_above), same += __popc(is_same);
    }
  }
  cluster.sync();  // no block leaves while another reads its totals
}

template <int D>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const EvictArgs a) {
  constexpr int kRow16 = D / 8, kCode16 = D / 64, Dg = D / kGroup;  // 16-byte pieces of a BF16 and of a code row
  __shared__ int old_of[kBody];
  const Geom &g = a.g, &og = a.og;
  const int unit = blockIdx.y, b = unit / g.Hkv;
  pdl_wait();  // the lists
  const Span s = span_of(a, a.lens[b]);
  const int T = s.T - s.gone;  // the new length
  if (unit % g.Hkv == 0 && blockIdx.x == 0 && threadIdx.x == 0) a.new_lens[b] = T;
  const int roles = g.vb ? 1 : 2;  // of the INT2 layout
  if (int(blockIdx.x) >= a.body_blocks) {
    // ------------------------------ window rows ---------------------------------
    const int r0 = (int(blockIdx.x) - a.body_blocks) * kWide, wide = max(g.S, T - g.W);
    constexpr int kPieces = kWide * kRow16 / kGatherThreads;
#pragma unroll 1
    for (int role = 0; role < roles; ++role) {
      const uint8_t* src = a.base + role * g.role_bytes;
      uint8_t* dst = a.out_base + role * og.role_bytes;
      uint4 x[kPieces], *to[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = threadIdx.x + i * kGatherThreads, r = r0 + at / kRow16, c = at % kRow16;
        const int p = wide + r - g.S;  // rows of the sink, then of the ring by position
        to[i] = nullptr;
        if (r < min(g.S, T)) {
          const int64_t n = (int64_t(unit) * g.S + r) * kRow16 + c;
          x[i] = __ldg(reinterpret_cast<const uint4*>(src) + n);
          to[i] = reinterpret_cast<uint4*>(dst) + n;
        } else if (r >= g.S && p < T) {
          x[i] = __ldg(reinterpret_cast<const uint4*>(src + g.sink_bytes) + (int64_t(unit) * g.W + (p + s.gone) % g.W) * kRow16 + c);
          to[i] = reinterpret_cast<uint4*>(dst + og.sink_bytes) + (int64_t(unit) * g.W + p % g.W) * kRow16 + c;
        }
      }
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (to[i]) *to[i] = x[i];
    }
    return;
  }
  const int p0 = blockIdx.x * kBody, n = min(kBody, T - p0);
  const int32_t* list = a.list + int64_t(unit) * a.list_cap;
  if (threadIdx.x < kBody) {
    const int p = p0 + threadIdx.x;
    const int old = p < g.S || p >= T ? p : p < g.S + s.held ? list[p - g.S] : p + s.gone;
    old_of[threadIdx.x] = old;
    if (a.out_mass && p < og.cap)
      a.out_mass[int64_t(unit) * og.cap + p] = p < T ? a.mass[int64_t(unit) * g.cap + old] : 0.f;
  }
  if (n <= 0) return;
  __syncthreads();
  const int skip = max(0, g.S - p0);  // sink positions have no INT2 row
  {
    // all loads of a block first: codes and scales of both roles
    constexpr int kPieces = kBody * kCode16 / kGatherThreads, kPairs = 2 * kBody * Dg / kGatherThreads;
    uint4 x[2][kPieces];
    uint32_t z[kPairs];
    const uint8_t* src = a.base + g.sink_bytes + g.ring_bytes;
    uint8_t* dst = a.out_base + og.sink_bytes + og.ring_bytes;
    const int64_t from = int64_t(unit) * g.ncap - g.S, to = int64_t(unit) * og.ncap - g.S + p0;
#pragma unroll
    for (int role = 0; role < 2; ++role)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = threadIdx.x + i * kGatherThreads, j = at / kCode16, c = at % kCode16;
        if (role < roles && j >= skip && j < n)
          x[role][i] = __ldg(reinterpret_cast<const uint4*>(src + role * g.role_bytes) + (from + old_of[j]) * kCode16 + c);
      }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int at = threadIdx.x + i * kGatherThreads, role = at / (kBody * Dg), j = at / Dg % kBody, c = at % Dg;
      if (role < roles && j >= skip && j < n)
        z[i] = __ldg(reinterpret_cast<const uint32_t*>(src + role * g.role_bytes + g.codes_bytes) + (from + old_of[j]) * Dg + c);
    }
#pragma unroll
    for (int role = 0; role < 2; ++role)
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int at = threadIdx.x + i * kGatherThreads, j = at / kCode16, c = at % kCode16;
        if (role < roles && j >= skip && j < n) reinterpret_cast<uint4*>(dst + role * og.role_bytes)[(to + j) * kCode16 + c] = x[role][i];
      }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int at = threadIdx.x + i * kGatherThreads, role = at / (kBody * Dg), j = at / Dg % kBody, c = at % Dg;
      if (role < roles && j >= skip && j < n)
        reinterpret_cast<uint32_t*>(dst + role * og.role_bytes + og.codes_bytes)[(to + j) * Dg + c] = z[i];
    }
  }
  if (g.vb) {  // V rows are BF16 at every position
    const uint4* in = reinterpret_cast<const uint4*>(a.base + g.role_bytes) + int64_t(unit) * g.cap * kRow16;
    uint4* out = reinterpret_cast<uint4*>(a.out_base + og.role_bytes) + (int64_t(unit) * og.cap + p0) * kRow16;
#pragma unroll 8
    for (int i = threadIdx.x; i < n * kRow16; i += kGatherThreads)
      out[i] = __ldg(in + int64_t(old_of[i / kRow16]) * kRow16 + i % kRow16);
  }
}

template <int D>
int launch_gather(const EvictArgs& a, dim3 grid, cudaStream_t stream) {
  return row_launch(true, evict_gather_kernel<D>, grid, kGatherThreads, 0, stream, a);
}

}  // namespace

int launch_kv_evict(const EvictArgs& args, cudaStream_t stream) {
  EvictArgs a = args;
  const int64_t units = int64_t(a.g.B) * a.g.Hkv;
  int dev = 0, sms = 0;
  if (units > 65535 || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return OSCAR_ERR_LAUNCH;
  static bool done[64] = {false};
  if (dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  // Blocks of a unit: as many as fill the GPU (two on an SM), none with less than 4096 positions, four at most.  us a call with
  // 1 / 2 / 4 / 8: 8 units of 65,536 positions 91 / 50 / 30 / 30, 32 of 32,768 51 / 30 / 26 / 51, 128 of 32,768 90 / 76 / 98 /
  // 204, 256 of 32,768 142 / 147 / 181 / 381, 8 of 8192 18 / 16 / 18 / 24.
  int size = 1;
  while (size < kMostCluster && 2 * size * units <= 2 * sms && a.g.cap / (2 * size) >= 4096) size *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(size);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * size));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kHeld * 4;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a) != cudaSuccess) return OSCAR_ERR_LAUNCH;
  a.body_blocks = (a.og.cap + kBody - 1) / kBody;
  const int64_t wide = (int64_t(a.g.S) + a.g.W + kWide - 1) / kWide;
  if (a.body_blocks + wide >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  const dim3 grid(unsigned(a.body_blocks + wide), unsigned(units));
  return a.g.D == 128 ? launch_gather<128>(a, grid, stream) : a.g.D == 256 ? launch_gather<256>(a, grid, stream)
                                                                            : launch_gather<512>(a, grid, stream);
}

}  // namespace oscar
