// attn_prompt on the 5th-generation tensor cores: bf16 inputs and outputs,
// head_dim 128.
//
// A block has two tiles of up to 128 query rows of one KV head: floor(128 / G)
// tokens with all their G query heads each, so that K and V are read once for the
// group and the causal mask cuts through few tokens.  It walks the positions 128
// at a time:
//
//   S_w [128 rows x 128 positions] = Q_w K^T,   O_w [128 rows x 128 channels] += P_w V
//
// S_w, O_w and P_w (bf16, over the scores that it was made from) lie in TMEM, 128
// columns each of the 512; Q, and K and V tiles in turn in a ring of five, come by
// TMA.  One warp issues all products, the two tiles' in turn: while one tile's
// softmax runs, the tensor cores work on the other's.  Products of one thread
// execute in the order of issue, so S_w of the next positions may follow P_w V
// over the same columns, and a finished S_w says that O_w is complete.
//
// Softmax: a thread has a row; its reference M follows the row's maximum only when
// that has grown by 2^8, and then the warp rescales its rows of O.  P is rounded to
// bf16, V's type; row sums are taken before the rounding, in float32.
//
// Positions that some of the block's rows do not see: their scores are set to
// -inf, which makes P zero, and a warp pair looks through those V rows first: where
// a value is infinite or not a number, zero times it would reach every row.  It is
// replaced by zero there, and added to the rows that see it at the end.
#include <algorithm>

#include "prompt_tc.cuh"

namespace oscar {
namespace {

constexpr int D = 128, N = 128;        // channels; query rows of a tile
constexpr int kSoftWarps = 8;
constexpr int kThreads = 12 * 32;      // softmax, products, loads, two warps that look through V
constexpr int kMma = 8, kLoad = 9, kCheck = 10;
constexpr int kTile = kTok * D * 2;    // bytes of a Q, K or V tile: two blocks of 64 channels
constexpr int kStages = 5;
constexpr int kChecked = 2;            // position tiles with tokens that some rows do not see
constexpr float kNone = -1e30f;
constexpr float kTop = 8.f;            // log2 of the largest P
constexpr int oQ = 0, oKV = 2 * kTile, oOdd = oKV + kStages * kTile, oBar = oOdd + 3 * D * 4;
constexpr int kBars = 2 * kStages + 2 + 2 + 2 + 2 + 2 * kChecked + 1;
constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;  // + alignment slack
static_assert(oBar % 8 == 0 && kBytes <= 232448 - 64, "shared memory");
constexpr uint32_t cS = 0, cO = 256;   // TMEM columns, 128 per tile
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "registers of a launch with 168 a thread");

__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  __shared__ PromptItem item;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = N / a.G;  // tokens of a tile

  const uint32_t bar = base + oBar;
  const uint32_t full = bar, empty = full + 8 * kStages, q_full = empty + 8 * kStages, s_full = q_full + 16,
                 p_full = s_full + 16, o_full = p_full + 16, values = o_full + 16, checked = values + 8 * kChecked,
                 drained = checked + 8 * kChecked;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + oBar + kBars * 8);
  int* odd = reinterpret_cast<int*>(sm + oOdd);
  int* any_odd = reinterpret_cast<int*>(tmem_slot + 1);
  if (warp == 0) {
    if (blockIdx.x == 0) prompt_check(a);
    const PromptItem it = prompt_item(a, blockIdx.x / a.Hkv, 1, 2 * tt);
    if (lane == 0) item = it;
  }
  if (threadIdx.x == kLoad * 32) {
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
      mbar_init(p_full + 8 * i, 4);
      mbar_init(o_full + 8 * i, 1);
    }
    for (int i = 0; i < kChecked; ++i) mbar_init(values + 8 * i, 1), mbar_init(checked + 8 * i, 2);
    mbar_init(drained, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == kCheck * 32) *any_odd = 0;
  if (warp >= kCheck)
    for (int i = threadIdx.x - kCheck * 32; i < 3 * D; i += 64) odd[i] = 0x7fffffff;
  __syncthreads();
  const PromptItem it = item;
  if (it.b < 0) return;
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  const int h = blockIdx.x % a.Hkv, t0 = it.tile * 2 * tt;
  auto tiles_of = [&](int w) {  // position tiles of query tile w
    const int first = t0 + w * tt;
    return first < it.len ? (min(first + tt, it.len) + kTok - 1) / kTok : 0;
  };
  const int nA = tiles_of(0), nB = tiles_of(1), nt = max(nA, nB);
  const int check0 = (t0 + 1) / kTok;  // the first tile with a token behind t0
  auto fail = [&]() { status_or(a.status, OSCAR_DEV_TIMEOUT); };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int w = warp >> 2, row = threadIdx.x & 127, n = w ? nB : nA;
    const int first = t0 + w * tt, tok = first + row / a.G;
    const bool live = row < tt * a.G && tok < it.len;
    const int lim = live ? tok : -1, least = first + (row & ~31) / a.G;  // the warp's first token
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t S = tmem + lanes + cS + 128 * w, O = tmem + lanes + cO + 128 * w;
    const uint64_t scale2 = splat_x2(a.qscale);
    float M = kNone;
    uint64_t l2 = 0;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      ok = wait_warp(s_full + 8 * w, j & 1, a.wait_turns);
      if (!ok) break;
      fence_after();
      uint32_t r[64], u[64];
      tmem_ld64(S, r);
      tmem_ld64(S + 64, u);
      if (j * kTok + kTok - 1 > least) {
        const int see = lim - j * kTok;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          r[c] = c <= see ? r[c] : 0xFF800000u;
          u[c] = c + 64 <= see ? u[c] : 0xFF800000u;
        }
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        top[0] = max3(top[0], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        top[1] = max3(top[1], __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
        top[2] = max3(top[2], __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
        top[3] = max3(top[3], __uint_as_float(u[c + 2]), __uint_as_float(u[c + 3]));
      }
      const float t = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.qscale;
      const bool grow = t > M + kTop;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2f(M - t) : 1.f;
        if (grow) M = t;
        l2 = mul2(l2, splat_x2(f));
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(O + c, o);
            tmem_wait16(o);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(O + c, o);
          }
        }
      }
      const uint64_t m2 = splat_x2(-M);
      uint64_t sum = 0, sum1 = 0;
      auto half = [&](const uint32_t (&x)[64], uint32_t to) {
#pragma unroll
        for (int c = 0; c < 64; c += 32) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float y, z;
            unpack2(fma2(pack2(__uint_as_float(x[c + 2 * i]), __uint_as_float(x[c + 2 * i + 1])), scale2, m2), y, z);
            y = ex2z(y);
            z = ex2z(z);
            p[i] = bf162_of(y, z);
            if (i & 1) sum = add2(sum, pack2(y, z));
            else sum1 = add2(sum1, pack2(y, z));
          }
          tmem_st16(to + c / 2, p);
        }
      };
      half(r, S);
      half(u, S + 32);
      l2 = add2(l2, add2(sum, sum1));
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      mbar_arrive_if(p_full + 8 * w, lane == 0);
    }
    if (n > 0 && ok) ok = wait_warp(o_full + 8 * w, 0, a.wait_turns);
    for (int i = 0; i < min(kChecked, nt - check0) && ok; ++i) ok = wait_warp(checked + 8 * i, 0, a.wait_turns);
    if (ok && n > 0) {
      fence_after();
      float l, l1;
      unpack2(l2, l, l1);
      l += l1;
      const float inv = 1.0f / l;
      const bool strange = *any_odd != 0;
      const int64_t at = int64_t(it.start + tok) * a.Hq + h * a.G + row % a.G;
      if (live && a.lse) a.lse[at] = (M + log2f(l)) * 0.6931471805599453f;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D);
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tmem_ld16(O + c, o);
        tmem_wait16(o);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(o[i]) * inv;
        if (strange) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (odd[c + i] <= tok) x[i] = __int_as_float(0x7FC00000);
            if (odd[D + c + i] <= tok) x[i] += INFINITY;
            if (odd[2 * D + c + i] <= tok) x[i] -= INFINITY;
          }
        }
        if (live) {
          uint32_t q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = bf162_of(x[2 * i], x[2 * i + 1]);
          dst[c / 8] = make_uint4(q[0], q[1], q[2], q[3]);
          dst[c / 8 + 1] = make_uint4(q[4], q[5], q[6], q[7]);
        }
      }
    }
    if (!ok && lane == 0) fail();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoad) {
      // ------------------------------- loads -----------------------------------
      if (lane == 0) {
        // the V tiles that are looked through have a barrier of their own, which that pair waits for: it would be behind in
        // the phases of `full`, which here completes at once
        auto tile = [&](int s, const CUtensorMap* map, int token) {
          const uint32_t to = base + oKV + (s % kStages) * kTile;
          uint32_t br = full + 8 * (s % kStages);
          if ((s & 1) && s / 2 >= check0) {
            mbar_arrive(br);
            br = values + 8 * (s / 2 - check0);
          }
          mbar_arrive_expect_tx(br, kTile);
          tma_load_2d(to, map, h * D, it.start + token, br);
          tma_load_2d(to + kTile / 2, map, h * D + 64, it.start + token, br);
        };
        auto queries = [&](int w) {
          mbar_arrive_expect_tx(q_full + 8 * w, 2 * tt * a.G * 128);
          for (int c = 0; c < 2; ++c)
            tma_load_3d(base + oQ + w * kTile + c * (kTile / 2), &mq, 64 * c, h * a.G, it.start + t0 + w * tt, q_full + 8 * w);
        };
        queries(0);
        bool ok = true;
        int s = 0;
        for (; s < 2 * nt && ok; ++s) {
          if (s >= kStages) ok = mbar_wait(empty + 8 * (s % kStages), (s / kStages - 1) & 1, a.wait_turns * 1000ull);
          if (!ok) break;
          tile(s, s & 1 ? &mv : &mk, (s / 2) * kTok);
          if (s == 0 && nB > 0) queries(1);
        }
        if (!ok) fail();
        // what was issued lands before the block ends, also where a wait ran out
        mbar_wait(q_full, 0);
        if (nB > 0) mbar_wait(q_full + 8, 0);
        for (int i = max(0, s - kStages); i < s; ++i) {
          if ((i & 1) && i / 2 >= check0) mbar_wait(values + 8 * (i / 2 - check0), 0);
          else mbar_wait(full + 8 * (i % kStages), (i / kStages) & 1);
        }
      }
    } else if (warp == kMma) {
      // ------------------------------ products ---------------------------------
      const uint32_t leader = elect_one();
      constexpr uint32_t id_qk = idesc_of(kTok, false, false) | kBf16, id_pv = idesc_of(D, false, true) | kBf16;
      const uint32_t dQ = desc_of(base + oQ, 16), dK = desc_of(base + oKV, 16), dV = desc_of(base + oKV, kTile / 2);
      Waits waits{a.wait_turns};
      Ring<kStages> kr, vr;  // stages of the next K and V tile: 0, 2, 4, .. and 1, 3, 5, ..
      vr.next();
      auto product_qk = [&](int w) {
        const uint32_t k = dK + kr.at * (kTile >> 4), q = dQ + w * (kTile >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_f16_ss(cS + 128 * w, q + (j >> 2) * (kTile >> 5) + 2 * (j & 3), k + (j >> 2) * (kTile >> 5) + 2 * (j & 3), id_qk, j > 0, leader);
        mma_commit(s_full + 8 * w, leader);
      };
      auto product_pv = [&](int w, uint32_t acc) {
        const uint32_t v = dV + vr.at * (kTile >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma_f16_ts(cO + 128 * w, cS + 128 * w + 8 * j, v + 128 * j, id_pv, j ? 1 : acc, leader);
      };
      waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
      waits.on(q_full, 0);
      waits.on(full + 8 * kr.at, kr.phase);
      fence_after();
      if (waits.ok) product_qk(0);
      if (nB > 0) {
        waits.on(q_full + 8, 0);
        fence_after();
        if (waits.ok) product_qk(1);
      }
      if (waits.ok) mma_commit(empty + 8 * kr.at, leader);
      kr.next(), kr.next();
#pragma unroll 1
      for (int j = 0; j < nt; ++j) {
        waits.on(full + 8 * vr.at, vr.phase);
        if (j >= check0) waits.on(checked + 8 * (j - check0), 0);
        const bool more = j + 1 < nt;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const int n = w ? nB : nA;
          if (j < n) {
            waits.on(p_full + 8 * w, j & 1);
            fence_after();
            if (!__all_sync(0xffffffffu, waits.ok)) break;
            product_pv(w, j > 0);
            if (j + 1 == n) mma_commit(o_full + 8 * w, leader);
          }
          if (w == 1) mma_commit(empty + 8 * vr.at, leader);
          if (j + 1 < n) {
            waits.on(full + 8 * kr.at, kr.phase);
            fence_after();
            if (!__all_sync(0xffffffffu, waits.ok)) break;
            product_qk(w);
          }
          if (w == 1 && more) mma_commit(empty + 8 * kr.at, leader);
        }
        if (!__all_sync(0xffffffffu, waits.ok)) break;
        kr.next(), kr.next();
        vr.next(), vr.next();
      }
      if (!__all_sync(0xffffffffu, waits.ok) && lane == 0) fail();
      mma_commit(drained, leader);  // every product issued is complete before TMEM is freed
      mbar_wait(drained, 0);
      __syncwarp();
    } else {
      // --------------------------- a look through V -----------------------------
      bool ok = true;
#pragma unroll 1
      for (int j = check0; j < nt && ok; ++j) {
        const int s = 2 * j + 1;
        ok = wait_warp(values + 8 * (j - check0), 0, a.wait_turns);
        if (ok) check_values<kTok, D>(sm + oKV + (s % kStages) * kTile, odd, j * kTok, t0, it.len, threadIdx.x - kCheck * 32);
        __syncwarp();
        for (int c = lane; c < 3 * D; c += 32)
          if (odd[c] != 0x7fffffff) *any_odd = 1;
        fence_async();
        __syncwarp();
        mbar_arrive_if(checked + 8 * (j - check0), lane == 0);
      }
      if (!ok && lane == 0) fail();
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace

int launch_attn_prompt_tc(const PromptArgs& a, cudaStream_t stream) {
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_prompt_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int tt = N / a.G;
  CUtensorMap mq, mk, mv;
  if (!encode_heads_bf16(&mq, a.q, uint64_t(a.n), a.Hq, D, uint32_t(a.G), uint32_t(tt)) ||
      !encode_rows_bf16(&mk, a.k, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok) ||
      !encode_rows_bf16(&mv, a.v, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok))
    return OSCAR_ERR_LAUNCH;
  const int64_t items = prompt_items(a, 1, 2 * tt) * a.Hkv;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_prompt_tc_kernel<<<unsigned(items), kThreads, kBytes, stream>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace oscar
