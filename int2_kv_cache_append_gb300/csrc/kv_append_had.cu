// kv_append of many rows with the in-quant Hadamard.
//
// The rotation reads no matrix, so the rows' bytes are the bound if the codec's
// instructions are few: a row of 128 channels has four lanes, 32 channels each
// (channel = 128 j + 32 m + 8 q + i for lane q of group j), so five of the seven
// butterfly stages and most of the extrema are within a lane, in packed float32
// pairs, and eight rows of head_dim 128 share a warp.  Stages and codec are those
// of the row-parallel kernel in its order (bits 5, 6, then 0 .. 4; every step one
// float32 rounding), so the bytes are the same.
//
// What bounds it: instructions, 850 for eight rows (four ragged prompts of 8192 tokens, 8
// KV heads: 55 us, 2.1 TB/s; the row-parallel kernel 185 us).
//
// The lane's codes of a word lie in two bit pairs per half (K) or four (V); two
// exchanges add the four lanes' parts up and leave each with two whole words.
#include "rows_tc.cuh"

namespace oscar {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 both(uint64_t x) {
  float2 d;
  unpack2(x, d.x, d.y);
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void butterfly(uint64_t& a, uint64_t& b) {
  const uint64_t s = add2(a, b), d = sub2(a, b);
  a = s, b = d;
}
// the pair of the lane `mask` away plus (lower lane) or minus (upper) this one
__device__ __forceinline__ uint64_t across(uint64_t x, int mask, uint64_t sign) {
  const float2 v = both(x);
  return fma2(x, sign, pack2(__shfl_xor_sync(0xffffffffu, v.x, mask), __shfl_xor_sync(0xffffffffu, v.y, mask)));
}
// word 2 L + .. of the eight partial words of four lanes, to lane L
__device__ __forceinline__ uint2 gather_words(const uint32_t (&w)[8], int q) {
  uint32_t u[4];
  const bool up = q & 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t give = up ? w[i] : w[4 + i];
    u[i] = (up ? w[4 + i] : w[i]) | __shfl_xor_sync(0xffffffffu, give, 2);
  }
  const bool odd = q & 1;
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t give = odd ? u[i] : u[2 + i];
    r[i] = (odd ? u[2 + i] : u[i]) | __shfl_xor_sync(0xffffffffu, give, 1);
  }
  return make_uint2(r[0], r[1]);
}

template <int D, bool FP32, bool LM>
__global__ void __launch_bounds__(kThreads, 3) kv_append_had_kernel(const AppendArgs a) {
  constexpr int LPR = D / 32, RPW = 32 / LPR;  // lanes of a row, rows of a warp
  const Geom& g = a.g;
  const int lane = threadIdx.x & 31, q = lane & 3, j = (lane % LPR) / 4, role = blockIdx.y;
  const uint32_t row = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * RPW + lane / LPR;  // below 2^31 + a block's
  const bool valid = row < a.rows;
  const int c0 = kGroup * j + 8 * q;  // the lane's first channel
  uint64_t x[4][4];                   // channels c0 + 32 m + 2 k, + 1
  {
    const int64_t at = int64_t(valid ? row : 0) * D + c0;
    if (FP32) {
      const float* src = static_cast<const float*>(role ? a.v_new : a.k_new) + at;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(src + 32 * m)), v = __ldg(reinterpret_cast<const float4*>(src + 32 * m) + 1);
        x[m][0] = pack2(u.x, u.y), x[m][1] = pack2(u.z, u.w), x[m][2] = pack2(v.x, v.y), x[m][3] = pack2(v.z, v.w);
      }
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(role ? a.v_new : a.k_new) + at;
      uint4 u[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] = __ldg(reinterpret_cast<const uint4*>(src + 32 * m));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t w[4] = {u[m].x, u[m].y, u[m].z, u[m].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[m][k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
      }
    }
  }
  // whose row it is, while the loads are under way
  int b = 0, h = 0, p = -1, newlen = 0;
  bool mine = valid;
  if (valid) {
    const uint32_t bt = fastdiv(row, a.div_hkv);
    h = int(row - bt * uint32_t(g.Hkv));
    int t, count = a.n_new;
    if (a.cu) {
      const NewToken tok = packed_token(a.cu, g.B, bt);
      mine = tok.b >= 0;
      b = max(tok.b, 0), t = tok.t, count = tok.count;
    } else {
      b = int(fastdiv(bt, a.div_n_new));
      t = int(bt - uint32_t(b) * uint32_t(a.n_new));
    }
    p = a.start_pos[b] + t;
    newlen = a.start_pos[b] + count;
  }

  // x H: bits 5 and 6, 0, 1 and 2 within the lane, 3 and 4 across
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    butterfly(x[0][k], x[1][k]);
    butterfly(x[2][k], x[3][k]);
    butterfly(x[0][k], x[2][k]);
    butterfly(x[1][k], x[3][k]);
  }
  const uint64_t sign3 = splat_x2(q & 1 ? -1.f : 1.f), sign4 = splat_x2(q & 2 ? -1.f : 1.f), unit = splat_x2(kInvSqrt128);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = both(x[m][k]);
      x[m][k] = pack2(v.x + v.y, v.x - v.y);
    }
    butterfly(x[m][0], x[m][1]);
    butterfly(x[m][2], x[m][3]);
    butterfly(x[m][0], x[m][2]);
    butterfly(x[m][1], x[m][3]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[m][k] = across(x[m][k], 1, sign3);
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) x[m][k] = mul2(across(x[m][k], 2, sign4), unit);

  if (a.debug_rot && valid) {
    uint64_t* dst = reinterpret_cast<uint64_t*>(a.debug_rot + (int64_t(row) * 2 + role) * D + c0);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[16 * m + k] = x[m][k];
  }
  const bool inside = mine && p >= 0 && p < g.cap;
  if (mine && !inside && lane % LPR == 0) status_or(a.status, OSCAR_DEV_OVER_CAPACITY);

  uint8_t* role_base = a.layer_base + role * g.role_bytes;
  const int64_t bh = int64_t(b) * g.Hkv + h;
  const bool whole = role == 1 && g.vb;  // K-only INT2: the V row is kept BF16 at its position
  const bool to_sink = inside && !whole && p < g.S, to_ring = inside && !whole && g.W > 0 && p >= newlen - g.W;
  if (to_sink || to_ring || (inside && whole)) {
    uint4* d0 = reinterpret_cast<uint4*>(role_base + (whole ? bh * g.cap + p : bh * g.S + p) * (2 * D) + 2 * c0);
    uint4* d1 = to_ring ? reinterpret_cast<uint4*>(role_base + g.sink_bytes + (bh * g.W + p % g.W) * (2 * D) + 2 * c0) : nullptr;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = both(x[m][k]);
        u[k] = pack_bf162(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y));
      }
      const uint4 w = make_uint4(u[0], u[1], u[2], u[3]);
      if (to_sink || whole) d0[4 * m] = w;
      if (to_ring) d1[4 * m] = w;
    }
  }

  float amax = 0.f;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = both(x[m][k]);
      amax = fmax3_nan(amax, fabsf(v.x), fabsf(v.y));
    }
  const bool finite = isfinite(amax);
  if (!finite) {  // the largest of those that are numbers
    amax = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = both(x[m][k]);
        amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (inside && !finite) status_or(a.status, OSCAR_DEV_NONFINITE);
  if (whole) return;  // all of the block

  const float tclip = __fmul_rn(role ? a.v_clip : a.k_clip, amax);
  float mn = INFINITY, mx = -INFINITY;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 v = both(x[m][k]);
      v.x = fminf(fmaxf(v.x, -tclip), tclip);
      v.y = fminf(fmaxf(v.y, -tclip), tclip);
      mn = fminf(mn, fminf(v.x, v.y));
      mx = fmaxf(mx, fmaxf(v.x, v.y));
      x[m][k] = pack2(v.x, v.y);
    }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const float s32 = __fdiv_rn(__fsub_rn(mx, mn), LM ? kLmSpan : 3.0f);
  const __half sh = __float2half_rn(s32), zh = __float2half_rn(mn);
  const float sf = __half2float(sh), zf = __half2float(zh);
  const bool rng_ok = isfinite(sf) && isfinite(zf);
  const bool body = inside && p >= g.S;
  if (body && !rng_ok && q == 0) status_or(a.status, OSCAR_DEV_FP16_RANGE);
  const bool ok = rng_ok && sf != 0.f;
  const uint64_t zz = splat_x2(zf), ii = splat_x2(ok ? __frcp_rn(sf) : 0.f);
  uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 y = both(mul2(sub2(x[m][k], zz), ii));
      const uint32_t u = LM ? lm_code(y.x) : min(__float2uint_rn(y.x), 3u);  // the conversion saturates below 0
      const uint32_t v = LM ? lm_code(y.y) : min(__float2uint_rn(y.y), 3u);
      if (role == 0) {  // word 2 k + (m >> 1), code 2 (q >> 1) + 4 (m & 1) + (q & 1) of its low (even channel) and high half
        w[2 * k + (m >> 1)] |= (u | v << 16) << (8 * (m & 1));
      } else {          // word 2 k (+ 1), code q + 4 m
        w[2 * k] |= u << (8 * m);
        w[2 * k + 1] |= v << (8 * m);
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = ok ? w[i] << (2 * q) : 0u;
  const uint2 words = gather_words(w, q);
  if (!body) return;
  const int64_t irow = bh * g.ncap + (p - g.S);
  uint8_t* codes = role_base + g.sink_bytes + g.ring_bytes;
  reinterpret_cast<uint2*>(codes + irow * (D / 4) + 32 * j)[q] = words;
  if (q == 0) reinterpret_cast<uint32_t*>(codes + g.codes_bytes)[irow * (D / kGroup) + j] = pack_half2(sh, zh);
}

template <int D>
int launch_d(const AppendArgs& args, cudaStream_t stream) {
  if (args.rows >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  AppendArgs a = args;
  a.div_hkv = fastdiv_make(uint32_t(a.g.Hkv));
  a.div_n_new = fastdiv_make(uint32_t(a.n_new > 0 ? a.n_new : 1));
  const int64_t per = int64_t(kThreads / 32) * (32 / (D / 32)), blocks = (a.rows + per - 1) / per;
  const dim3 grid(unsigned(blocks), 2);
  const auto kernel = a.in_fp32 ? (a.g.lm ? kv_append_had_kernel<D, true, true> : kv_append_had_kernel<D, true, false>)
                                : (a.g.lm ? kv_append_had_kernel<D, false, true> : kv_append_had_kernel<D, false, false>);
  kernel<<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace

int launch_append_had(const AppendArgs& a, cudaStream_t stream) {
  return a.g.D == 128 ? launch_d<128>(a, stream) : a.g.D == 256 ? launch_d<256>(a, stream) : launch_d<512>(a, stream);
}

}  // namespace oscar
