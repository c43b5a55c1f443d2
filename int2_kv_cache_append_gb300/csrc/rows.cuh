// Cache rows addressed by position, for the kernels that work on blocks of
// positions or of query rows (kv_read, attn_extend, attn_decode_prefix).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace oscar {

constexpr int kSplitUnit = 128;  // positions: the shares of a split cache start at multiples of it

// Launch after the kernel before it in the stream; dependent: it may start once every block of that one has called
// pdl_trigger or ended, and waits (pdl_wait) before it reads what that one or an earlier one wrote.  Every block of a
// kernel that is launched so waits before it ends, so that "complete" holds for everything before it, too.  What an earlier
// kernel of the same call writes (rotated queries, partial results, merged rows) is read by plain loads: __ldg promises
// memory that nobody writes while the kernel runs, and its loads may be moved above pdl_wait.
template <class... P>
int row_launch(bool dependent, void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, P... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

// A row attention's wait for the kernels before it (RowsArgs::ready).
__device__ __forceinline__ void rows_wait(const RowsArgs& a) {
  pdl_wait();
  if (a.ready && !a.beside && blockIdx.x == 0 && threadIdx.x == 0)
    asm volatile("st.release.gpu.global.s32 [%0], 1;" ::"l"(a.ready) : "memory");
}
// One thread's bounded wait for *ready, a barrier before the others read the queries: the store has been made, or will be by
// a block that is running, when a kernel starts beside.
__device__ __forceinline__ bool ready_wait(const int32_t* ready, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    int32_t x;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(x) : "l"(ready) : "memory");
    if (x) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// Length of sequence b in the cache that is read, clamped to the capacity;
// `report`: this thread flags a length above it.
__device__ __forceinline__ int row_seq_len(const RowsArgs& a, int b, bool report) {
  int T = a.seq_lens[b];
  if (T > a.g.cap) {
    if (report) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);
    T = a.g.cap;
  }
  return max(T, 0);
}
// Query tokens of sequence b.
__device__ __forceinline__ int row_q_len(const RowsArgs& a, int b) {
  return a.q_lens ? min(a.q_lens[b], a.n) : a.n;
}

// Row (b n + t) Hq + head of a query block is one of the sequence's tokens.
__device__ __forceinline__ bool row_live(int64_t row, int64_t rows, const int32_t* q_lens, int n, int Hq) {
  if (row >= rows) return false;
  if (!q_lens) return true;
  const uint32_t bt = uint32_t(row) / uint32_t(Hq);  // rows < 2^31
  return int(bt % uint32_t(n)) < q_lens[bt / uint32_t(n)];
}

// Where one cached row of a role lives: BF16 (a window, or K-only INT2's V
// rows) or INT2 (codes and scale / zero pairs).
struct RowRef {
  const __nv_bfloat16* wide;  // D values, or NULL
  const uint32_t* codes;      // D / 16 words
  const __half2* sz;          // D / 128 (scale, zero) pairs
};

// Row of position p (0 <= p < T) of unit = b * Hkv + h in a sequence of length
// T: sink below S, ring for the last W positions, INT2 between.
__device__ __forceinline__ RowRef row_ref(const Geom& g, const uint8_t* layer_base, int role, int64_t unit, int T,
                                          int p) {
  RowRef r{nullptr, nullptr, nullptr};
  const uint8_t* base = layer_base + (role ? g.role_bytes : 0);
  if (role && g.vb) {
    r.wide = reinterpret_cast<const __nv_bfloat16*>(base) + (unit * g.cap + p) * g.D;
  } else if (p < g.S) {
    r.wide = reinterpret_cast<const __nv_bfloat16*>(base) + (unit * g.S + p) * g.D;
  } else if (p >= T - g.W) {
    r.wide = reinterpret_cast<const __nv_bfloat16*>(base + g.sink_bytes) + (unit * g.W + p % g.W) * g.D;
  } else {
    const int64_t row = unit * g.ncap + (p - g.S);
    const uint8_t* codes = base + g.sink_bytes + g.ring_bytes;
    r.codes = reinterpret_cast<const uint32_t*>(codes) + row * (g.D / 16);
    r.sz = reinterpret_cast<const __half2*>(codes + g.codes_bytes) + row * g.Dg;
  }
  return r;
}

// Sixteen channels of a row as float32: code word w of an INT2 row (the
// channels the header's layout gives that word), channels 16 w .. 16 w + 15 of
// a BF16 row.
__device__ __forceinline__ void row_load16(const Geom& g, const RowRef& r, int role, int w, float* dst) {
  if (r.wide) {
    const uint4* src = reinterpret_cast<const uint4*>(r.wide + 16 * w);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 x = src[q];
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dst[16 * w + 8 * q + 2 * e] = __uint_as_float(v[e] << 16);
        dst[16 * w + 8 * q + 2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
      }
    }
    return;
  }
  const uint32_t x = r.codes[w];
  const float2 sz = __half22float2(r.sz[w >> 3]);
  const int j = w & 7;
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    const int c = int(x >> (2 * n)) & 3;
    const float level = g.lm ? kLmRho * float(c) + (1.0f - kLmRho) * float(c >> 1) : float(c);
    // K: word 2c + i, bit 2p + 16 hi -> channel 64 i + 8 p + 2 c + hi; V: word g, bit 2n -> channel 8 n + g
    const int ch = role == 0 ? 64 * (j & 1) + 8 * (n & 7) + (j & ~1) + (n >> 3) : 8 * n + j;
    dst[128 * (w >> 3) + ch] = fmaf(sz.x, level, sz.y);
  }
}

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

// Element [i][k] of the in-quant Hadamard: block-diagonal, order 128.
__device__ __forceinline__ float hadamard_at(int i, int k) {
  if ((i ^ k) >> 7) return 0.f;
  return (__popc(i & k & 127) & 1) ? -kInvSqrt128 : kInvSqrt128;
}

}  // namespace oscar
