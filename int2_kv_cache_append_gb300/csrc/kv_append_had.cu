// kv_append of many rows with the in-quant Hadamard.
//
// The rotation reads no matrix, so the rows' bytes are the bound if the codec's
// instructions are few: a row of 128 channels has four lanes with 32 consecutive
// channels each (channel = 128 j + 32 q + i for lane q of group j), so five of the
// seven butterfly stages and most of the extrema are within a lane, in packed
// float32 pairs, and eight rows of head_dim 128 share a warp.  Stages and codec are
// those of the row-parallel kernel in its order (bits 5, 6, then 0 .. 4; every step
// one float32 rounding), so the bytes are the same.
//
// Codes of channels 8 apart are next to each other in a word, of K and of V: a lane
// packs byte g of its channels g, g + 8, g + 16, g + 24 with saturating conversions,
// and one (K) or two (V) exchanges put the four lanes' bytes together.
//
// What bounds it: instructions and their latency, 690 for eight rows (four ragged prompts of
// 8192 tokens, 8 KV heads: 46.5 us, 2.5 TB/s; three blocks an SM instead of four 53 us; the
// row-parallel kernel 185 us).
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
// bits << 4 and two codes, each the nearest of 0 .. 3
__device__ __forceinline__ uint32_t pack_codes(int second, int first, uint32_t bits) {
  uint32_t d;
  asm("cvt.pack.sat.u2.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(second), "r"(first), "r"(bits));
  return d;
}

template <int D, bool FP32, bool LM, bool PACKED>
__global__ void __launch_bounds__(kThreads, 4) kv_append_had_kernel(const AppendArgs a) {
  constexpr int LPR = D / 32, RPW = 32 / LPR;  // lanes of a row, rows of a warp
  // Launched like the row-parallel kernel, for decode steps of large batches: a layer of 160 sequences and 8 heads takes 82.1 us,
  // launched plainly 85.2 (row-parallel 84.0).  What is read is read by plain loads (row_launch).
  pdl_wait();
  pdl_trigger();
  const Geom& g = a.g;
  append_check<PACKED>(a);
  const int lane = threadIdx.x & 31, q = lane & 3, j = (lane % LPR) / 4, role = blockIdx.y;
  const uint32_t row = (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * RPW + lane / LPR;  // below 2^31 + a block's
  const bool valid = row < a.rows;
  const int c0 = kGroup * j + 32 * q;  // the lane's first channel
  uint64_t x[16];                      // channels c0 + 2 k, + 1
  {
    const int64_t at = int64_t(valid ? row : 0) * D + c0;
    if (FP32) {
      const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(role ? a.v_new : a.k_new) + at);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        const float4 u = src[m];
        x[2 * m] = pack2(u.x, u.y), x[2 * m + 1] = pack2(u.z, u.w);
      }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(role ? a.v_new : a.k_new) + at);
      uint4 u[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) u[m] = src[m];
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const uint32_t w[4] = {u[m].x, u[m].y, u[m].z, u[m].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) x[4 * m + k] = pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
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
    if (PACKED) {
      const NewToken tok = packed_token(a.cu, g.B, a.n_rows, bt);
      mine = tok.b >= 0;
      b = max(tok.b, 0), t = tok.t, count = tok.count;
    } else {
      b = int(fastdiv(bt, a.div_n_new));
      t = int(bt - uint32_t(b) * uint32_t(a.n_new));
    }
    p = a.start_pos[b] + t;
    newlen = a.start_pos[b] + count;
  }

  // x H: bits 5 and 6 across lanes, 0 within a pair, 1 .. 4 within the lane
  const uint64_t sign5 = splat_x2(q & 1 ? -1.f : 1.f), sign6 = splat_x2(q & 2 ? -1.f : 1.f), unit = splat_x2(kInvSqrt128);
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = across(x[k], 1, sign5);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 v = both(across(x[k], 2, sign6));
    x[k] = pack2(v.x + v.y, v.x - v.y);
  }
#pragma unroll
  for (int bit = 1; bit < 16; bit <<= 1)
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (!(k & bit)) butterfly(x[k], x[k | bit]);
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = mul2(x[k], unit);

  if (a.debug_rot && valid) {
    uint64_t* dst = reinterpret_cast<uint64_t*>(a.debug_rot + (int64_t(row) * 2 + role) * D + c0);
#pragma unroll
    for (int k = 0; k < 16; ++k) dst[k] = x[k];
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
        const float2 v = both(x[4 * m + k]);
        u[k] = pack_bf162(__float2bfloat16_rn(v.x), __float2bfloat16_rn(v.y));
      }
      const uint4 w = make_uint4(u[0], u[1], u[2], u[3]);
      if (to_sink || whole) d0[m] = w;
      if (to_ring) d1[m] = w;
    }
  }

  float rmn = INFINITY, rmx = -INFINITY;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 v = both(x[k]);
    rmn = fmin3_nan(rmn, v.x, v.y);
    rmx = fmax3_nan(rmx, v.x, v.y);
  }
  const bool finite = isfinite(rmn) && isfinite(rmx);
  float amax = fmaxf(fabsf(rmn), fabsf(rmx));
  const bool strange = __any_sync(0xffffffffu, !finite);
  if (strange) {  // the largest of those that are numbers
    amax = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 v = both(x[k]);
      amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
    }
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (inside && !finite) status_or(a.status, OSCAR_DEV_NONFINITE);
  if (whole) return;  // all of the block

  const float tclip = __fmul_rn(role ? a.v_clip : a.k_clip, amax);
  auto clip = [&]() {
    rmn = INFINITY, rmx = -INFINITY;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float2 v = both(x[k]);
      v.x = fminf(fmaxf(v.x, -tclip), tclip);
      v.y = fminf(fmaxf(v.y, -tclip), tclip);
      rmn = fminf(rmn, fminf(v.x, v.y));
      rmx = fmaxf(rmx, fmaxf(v.x, v.y));
      x[k] = pack2(v.x, v.y);
    }
  };
  if (strange) clip();
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    rmn = fminf(rmn, __shfl_xor_sync(0xffffffffu, rmn, o));
    rmx = fmaxf(rmx, __shfl_xor_sync(0xffffffffu, rmx, o));
  }
  const float mn = fminf(fmaxf(rmn, -tclip), tclip), mx = fminf(fmaxf(rmx, -tclip), tclip);  // of the clipped values
  const float s32 = __fdiv_rn(__fsub_rn(mx, mn), LM ? kLmSpan : 3.0f);
  const __half sh = __float2half_rn(s32), zh = __float2half_rn(mn);
  const float sf = __half2float(sh), zf = __half2float(zh);
  const bool rng_ok = isfinite(sf) && isfinite(zf);
  const bool body = inside && p >= g.S;
  if (body && !rng_ok && q == 0) status_or(a.status, OSCAR_DEV_FP16_RANGE);
  const bool ok = rng_ok && sf != 0.f;
  const float inv = ok ? __frcp_rn(sf) : 0.f;
  auto code = [&](float y) { return LM ? lm_code(y) : __float2int_rn(y); };
  // Values that the clip would change have the codes 0 and 3 without it where the clipped ones have (each step is
  // monotone); a scale that is small beside the zero's rounding may make others of them.
  const int top = code(__fmul_rn(__fsub_rn(mx, zf), inv)), bottom = code(__fmul_rn(__fsub_rn(mn, zf), inv));
  if (__any_sync(0xffffffffu, ok && ((rmx > tclip && top < 3) || (rmn < -tclip && bottom > 0)))) clip();
  const uint64_t zz = splat_x2(zf), ii = splat_x2(inv);
  uint32_t w[2] = {0, 0};  // byte g: the codes of channels g + 8 k
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int e = 2; e >= 0; e -= 2) {  // channels g and g + 1, g = 4 r + e
      int lo[4], hi[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 y = both(mul2(sub2(x[4 * k + 2 * r + e / 2], zz), ii));
        lo[k] = code(y.x), hi[k] = code(y.y);
      }
      w[r] = pack_codes(hi[1], hi[0], pack_codes(hi[3], hi[2], w[r]));
      w[r] = pack_codes(lo[1], lo[0], pack_codes(lo[3], lo[2], w[r]));
    }
  if (!ok) w[0] = w[1] = 0;
  uint32_t words[2];
  if (role == 0) {
    // word 2 c + (q >> 1): bytes of c's channel pair, of the lanes q and q ^ 1 in turn; the even lane has c = 0, 1
    const bool odd = q & 1;
    const uint32_t keep = odd ? w[1] : w[0], got = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
    const uint32_t u = odd ? got : keep, v = odd ? keep : got;
    words[0] = prmt(u, v, 0x5140), words[1] = prmt(u, v, 0x7362);
  } else {
    // word g: byte g of the lanes in turn; lane q has words 2 q and 2 q + 1
    const bool up = q & 2, odd = q & 1;
    const uint32_t keep = up ? w[1] : w[0], got = __shfl_xor_sync(0xffffffffu, up ? w[0] : w[1], 2);  // of q, of q ^ 2
    const uint32_t mine2 = prmt(keep, got, odd ? 0x7632 : 0x5410);
    const uint32_t theirs = __shfl_xor_sync(0xffffffffu, prmt(keep, got, odd ? 0x5410 : 0x7632), 1);  // of q ^ 1, of q ^ 3
    const uint32_t order = q == 0 ? 0x6240u : q == 1 ? 0x2604u : q == 2 ? 0x4062u : 0x0426u;
    words[0] = prmt(mine2, theirs, order), words[1] = prmt(mine2, theirs, order + 0x1111u);
  }
  if (!body) return;
  const int64_t irow = bh * g.ncap + (p - g.S);
  uint8_t* codes = role_base + g.sink_bytes + g.ring_bytes;
  uint32_t* to = reinterpret_cast<uint32_t*>(codes + irow * (D / 4) + 32 * j);
  if (role == 0) to[4 * (q & 1) + (q >> 1)] = words[0], to[4 * (q & 1) + (q >> 1) + 2] = words[1];
  else reinterpret_cast<uint2*>(to)[q] = make_uint2(words[0], words[1]);
  if (q == 0) reinterpret_cast<uint32_t*>(codes + g.codes_bytes)[irow * (D / kGroup) + j] = pack_half2(sh, zh);
}

template <int D, bool PACKED>
int launch_d(const AppendArgs& args, cudaStream_t stream) {
  if (args.rows >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  AppendArgs a = args;
  a.div_hkv = fastdiv_make(uint32_t(a.g.Hkv));
  a.div_n_new = fastdiv_make(uint32_t(a.n_new > 0 ? a.n_new : 1));
  const int64_t per = int64_t(kThreads / 32) * (32 / (D / 32)), blocks = (a.rows + per - 1) / per;
  const dim3 grid(unsigned(blocks), 2);
  const auto kernel = a.in_fp32 ? (a.g.lm ? kv_append_had_kernel<D, true, true, PACKED> : kv_append_had_kernel<D, true, false, PACKED>)
                                : (a.g.lm ? kv_append_had_kernel<D, false, true, PACKED> : kv_append_had_kernel<D, false, false, PACKED>);
  return row_launch(true, kernel, grid, kThreads, 0, stream, a);
}

template <bool PACKED>
int launch_p(const AppendArgs& a, cudaStream_t stream) {
  return a.g.D == 128 ? launch_d<128, PACKED>(a, stream) : a.g.D == 256 ? launch_d<256, PACKED>(a, stream) : launch_d<512, PACKED>(a, stream);
}

}  // namespace

int launch_append_had(const AppendArgs& a, cudaStream_t stream) { return a.cu ? launch_p<true>(a, stream) : launch_p<false>(a, stream); }

}  // namespace oscar
