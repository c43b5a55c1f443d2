// Attention of blocks of query rows over one cache, in float32 throughout: the
// kernel behind attn_extend and attn_decode_prefix when the output is float32.
//
// One pass with a running maximum and sum: a CTA holds 32 rotated query rows
// of one (sequence, KV head), walks its share of the positions 32 at a time
// (rows of any region expanded to float32 in shared memory), and keeps the
// rows' maxima, sums and outputs in registers.  Eight threads share a row: each
// takes every eighth position of the scores and D / 8 channels of the output.
// What bounds it: shared-memory reads (one 16-byte read per four FMAs in
// P V, five per sixteen in Q K^T).  No size of it has been made fast: it is
// there for its precision.  A chunk of 2048 tokens x 64 heads over 16,384
// positions takes 62 ms, 64 sequences x 64 heads on a prefix of 131,072 40 ms:
// both longer than the formula in elementary float32 tensor operations (40 and
// 23 ms) and 45 to 90 times the bf16 output's kernels.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "rows.cuh"

namespace oscar {
namespace {

constexpr int kRowTile = 32;
constexpr int kTokTile = 32;
constexpr int kThreads = 256;
constexpr int kPitchS = kTokTile + 4;
constexpr float kNone = -1e30f;  // running maximum before the first visible position

template <int D>
__global__ void __launch_bounds__(kThreads) attn_rows_kernel(const RowsArgs a) {
  extern __shared__ float sm[];
  constexpr int xp = D + 4;
  const Geom& g = a.g;
  float* Qs = sm;
  float* Ks = Qs + kRowTile * xp;
  float* Vs = Ks + kTokTile * xp;
  float* Ss = Vs + kTokTile * xp;
  // item: split s of row tile rt (last tiles first: with a causal mask they are the longest) of unit u
  pdl_wait();
  if (a.early) pdl_trigger();
  const int units = g.B * g.Hkv, rows = a.n * g.G, tiles = (rows + kRowTile - 1) / kRowTile;
  const int s = int(blockIdx.x % unsigned(a.ns));
  const int64_t it = blockIdx.x / unsigned(a.ns);
  const int u = int(it % units), rt = tiles - 1 - int(it / units);
  const int b = u / g.Hkv, h = u % g.Hkv;
  const int T = row_seq_len(a, b, threadIdx.x == 0 && blockIdx.x < unsigned(a.ns) * units);
  const int ql = row_q_len(a, b);
  const int r = threadIdx.x >> 3, tq = threadIdx.x & 7;
  const int row = rt * kRowTile + r, t = row / g.G;
  const bool live = row < rows && t < ql;
  const int lim = live ? (a.causal ? T - ql + t : T - 1) : -1;  // last visible position
  const int t_last = min((rt * kRowTile + kRowTile - 1) / g.G, ql - 1);
  if (rt * kRowTile / g.G >= ql) return;  // only padding
  const int vis = max(0, a.causal ? min(T, T - ql + t_last + 1) : T);
  const int blocks = (vis + kSplitUnit - 1) / kSplitUnit;
  const int p0 = int(int64_t(blocks) * s / a.ns) * kSplitUnit;
  const int p1 = min(vis, int(int64_t(blocks) * (s + 1) / a.ns) * kSplitUnit);
  const int64_t out_row = (int64_t(b) * a.n + t) * g.Hq + h * g.G + row % g.G;

  for (int i = threadIdx.x; i < kRowTile * (D / 4); i += kThreads) {
    const int rr = i / (D / 4), c = (i % (D / 4)) * 4;
    const int qr = rt * kRowTile + rr;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (qr < rows && qr / g.G < ql)
      v = *reinterpret_cast<const float4*>(
          a.qrot + ((int64_t(b) * a.n + qr / g.G) * g.Hq + h * g.G + qr % g.G) * D + c);
    *reinterpret_cast<float4*>(Qs + rr * xp + c) = v;
  }
  float m = kNone, l = 0.f;
  float4 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);

  for (int p = p0; p < p1; p += kTokTile) {
    __syncthreads();  // the previous tile has been used (and Q is complete)
    for (int i = threadIdx.x; i < 2 * kTokTile * (D / 16); i += kThreads) {
      const int role = i / (kTokTile * (D / 16)), k = i % (kTokTile * (D / 16));
      const int tok = k / (D / 16), w = k % (D / 16);
      float* dst = (role ? Vs : Ks) + tok * xp;
      if (p + tok < p1) {
        row_load16(g, row_ref(g, a.layer_base, role, u, T, p + tok), role, w, dst);
      } else {
        for (int e = 0; e < 16; ++e) dst[16 * w + e] = 0.f;
      }
    }
    __syncthreads();
    float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      const float4 q = *reinterpret_cast<const float4*>(Qs + r * xp + c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(Ks + (tq + 8 * j) * xp + c);
        sc[j] = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, fmaf(q.w, k.w, sc[j]))));
      }
    }
    float mx = m;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int pos = p + tq + 8 * j;
      if (pos > lim || pos >= p1) sc[j] = -INFINITY;
      mx = fmaxf(mx, sc[j]);
    }
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float f = exp2f(m - mx);
    m = mx;
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sc[j] = exp2f(sc[j] - m);
      sum += sc[j];
      Ss[r * kPitchS + tq + 8 * j] = sc[j];
    }
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = fmaf(l, f, sum);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      o[i].x *= f;
      o[i].y *= f;
      o[i].z *= f;
      o[i].w *= f;
    }
    __syncwarp();
    for (int k = 0; k < kTokTile; ++k) {
      const float w = Ss[r * kPitchS + k];
      if (w == 0.f) continue;  // a hidden position: whatever its value row holds stays out
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(Vs + k * xp + 4 * tq + 32 * i);
        o[i].x = fmaf(w, v.x, o[i].x);
        o[i].y = fmaf(w, v.y, o[i].y);
        o[i].z = fmaf(w, v.z, o[i].z);
        o[i].w = fmaf(w, v.w, o[i].w);
      }
    }
    __syncwarp();
  }
  if (!live) return;
  const int64_t slot = out_row * a.ns + s;
  if (tq == 0) *reinterpret_cast<float2*>(a.ml + slot * 2) = make_float2(m, l);
  if (l == 0.f) return;  // nothing visible in this share: the merge does not read the sums
#pragma unroll
  for (int i = 0; i < D / 32; ++i) *reinterpret_cast<float4*>(a.acc + slot * D + 4 * tq + 32 * i) = o[i];
}

template <int D>
int launch(const RowsArgs& a, cudaStream_t stream) {
  constexpr int smem = ((kRowTile + 2 * kTokTile) * (D + 4) + kRowTile * kPitchS) * 4;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int64_t tiles = (int64_t(a.n) * a.g.G + kRowTile - 1) / kRowTile;
  const int64_t items = tiles * a.g.B * a.g.Hkv * a.ns;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  return row_launch(true, attn_rows_kernel<D>, dim3(unsigned(items)), kThreads, smem, stream, a);
}

}  // namespace

int rows_splits(const Geom& g, int64_t rows, int seq_len_hint) {
  // two CTAs on each of 152 SMs, whichever device there is (as rows_splits_tc)
  const int64_t items = (rows + kRowTile - 1) / kRowTile * g.B * g.Hkv;
  const int64_t blocks = (int64_t(seq_len_hint) + kSplitUnit - 1) / kSplitUnit;
  return int(std::max<int64_t>(1, std::min<int64_t>({OSCAR_KV_MAX_SPLITS, 304 / items, blocks})));
}

int launch_attn_rows(const RowsArgs& a, cudaStream_t stream) {
  if (a.g.D == 128) return launch<128>(a, stream);
  if (a.g.D == 256) return launch<256>(a, stream);
  return launch<512>(a, stream);
}

}  // namespace oscar
