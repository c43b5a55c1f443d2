// attn_prompt on the 5th-generation tensor cores: bf16 inputs and outputs,
// head_dim 256 and 512.
//
// A block has one tile of up to 128 query rows (floor(128 / G) tokens with the G
// heads of one KV head) and 256 channels of the output: at head_dim 512 two blocks
// share the query tile, since scores and output of 512 channels do not fit the 512
// TMEM columns together; each forms the scores of its own.  Two score tiles
// alternate, so the products of one run under the softmax of the other; O has the
// other 256 columns.  K comes in units of 64 channels of 128 positions, V in units
// of 64 positions of 128 channels, 16 KB each, in one ring in the order in which
// they are used.
//
// Softmax: eight warps; the two threads of a row have 64 positions each and
// exchange their maxima once per tile.  Arithmetic, masks and the look through V
// are those of head_dim 128 (attn_prompt_tc.cu).
#include <algorithm>

#include "prompt_tc.cuh"

namespace oscar {
namespace {

constexpr int N = 128, kOut = 256;     // query rows; output channels of a block
constexpr int kSoftWarps = 8;
constexpr int kThreads = 12 * 32;
constexpr int kMma = 8, kLoad = 9, kCheck = 10;
constexpr int kChecked = 2;            // position tiles with tokens that some rows do not see
constexpr int kValueUnits = 4;         // V units of a position tile
constexpr float kNone = -1e30f;
constexpr float kTop = 8.f, kAbove = 12.f;
constexpr uint32_t cS = 0, cO = 256;   // TMEM columns: two score tiles, O

template <int D>
struct Wide {
  static constexpr int kKeyUnits = D / 64;
  static constexpr int kUnits = D == 256 ? 9 : 5;
  static constexpr int oRing = D * N * 2;
  static constexpr int oOdd = oRing + kUnits * kUnit;
  static constexpr int oSwap = oOdd + 3 * kOut * 4;
  static constexpr int oBar = oSwap + 4 * N * 4;
  static constexpr int kBars = 2 * kUnits + 1 + 2 + 1 + 1 + 2 * kChecked * kValueUnits + 1;
  static constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;
  static_assert(oBar % 8 == 0 && kBytes <= 232448 - 64, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_wide_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                            const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
  using C = Wide<D>;
  constexpr int kParts = D / kOut, kUnits = C::kUnits;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  __shared__ PromptItem item;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = N / a.G;

  const uint32_t bar = base + C::oBar;
  const uint32_t full = bar, empty = full + 8 * kUnits, q_full = empty + 8 * kUnits, s_full = q_full + 8, p_full = s_full + 16,
                 p_done = p_full + 8, values = p_done + 8, checked = values + 8 * kChecked * kValueUnits,
                 drained = checked + 8 * kChecked * kValueUnits;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::oBar + C::kBars * 8);
  int* any_odd = reinterpret_cast<int*>(tmem_slot + 1);
  int* odd = reinterpret_cast<int*>(sm + C::oOdd);
  float* swap = reinterpret_cast<float*>(sm + C::oSwap);  // [2][2][N]
  if (warp == 0) {
    if (blockIdx.x == 0) prompt_check(a);
    int level = -1;
    const PromptItem it = prompt_item(a, blockIdx.x / (a.Hkv * kParts), 1, tt, level);
    if (lane == 0) item = it;
  }
  if (threadIdx.x == kLoad * 32) {
    for (int i = 0; i < kUnits; ++i) mbar_init(full + 8 * i, 1), mbar_init(empty + 8 * i, 1);
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) mbar_init(s_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
    mbar_init(p_full, kSoftWarps);
    mbar_init(p_done, 1);
    for (int i = 0; i < kChecked * kValueUnits; ++i) mbar_init(values + 8 * i, 1), mbar_init(checked + 8 * i, 2);
    mbar_init(drained, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == kCheck * 32) *any_odd = 0;
  if (warp >= kCheck)
    for (int i = threadIdx.x - kCheck * 32; i < 3 * kOut; i += 64) odd[i] = 0x7fffffff;
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
  const int part = blockIdx.x % kParts, h = blockIdx.x / kParts % a.Hkv, t0 = it.tile * tt;
  const int nt = (min(t0 + tt, it.len) + kTok - 1) / kTok;
  const int check0 = (t0 + 1) / kTok;  // the first tile with a token behind t0
  auto fail = [&]() { status_or(a.status, OSCAR_DEV_TIMEOUT); };
  auto wait = [&](uint32_t br, uint32_t parity) { return wait_warp(br, parity, a.wait_turns); };

  if (warp < kSoftWarps) {
    const int half = warp >> 2, row = threadIdx.x & 127;
    const int tok = t0 + row / a.G;
    const bool live = row < tt * a.G && tok < it.len;
    const int lim = live ? tok : -1, least = t0 + (row & ~31) / a.G;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t O = tmem + lanes + cO + 128 * half;
    const uint64_t scale2 = splat_x2(a.qscale);
    float M = kNone;
    uint64_t l2 = 0;
    bool ok = true;
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      const uint32_t S = tmem + lanes + cS + 128 * (j & 1) + 64 * half;
      ok = ok && wait(s_full + 8 * (j & 1), (j >> 1) & 1);
      fence_after();
      uint32_t r[64];
      tmem_ld64(S, r);
      if (j * kTok + kTok - 1 > least) {
        const int see = lim - j * kTok - 64 * half;
#pragma unroll
        for (int c = 0; c < 64; ++c) r[c] = c <= see ? r[c] : 0xFF800000u;
      }
      float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 64; c += 4) {
        top = max3(top, __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        top1 = max3(top1, __uint_as_float(r[c + 2]), __uint_as_float(r[c + 3]));
      }
      float* mine = swap + (j & 1) * 2 * N;
      mine[half * N + row] = fmaxf(top, top1);
      if (any256(3, !ok)) {
        ok = false;
        break;
      }
      const float t = fmaxf(mine[row], mine[N + row]) * a.qscale;
      const bool grow = t > M + kTop;
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2f(M - (t + kAbove)) : 1.f;
        if (grow) M = t + kAbove;
        l2 = mul2(l2, splat_x2(f));
        if (j > 0) {
          ok = wait(p_done, (j - 1) & 1);  // O is not in use
          fence_after();
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
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
#pragma unroll
      for (int c = 0; c < 64; c += 32) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float y, z;
          unpack2(fma2(pack2(__uint_as_float(r[c + 2 * i]), __uint_as_float(r[c + 2 * i + 1])), scale2, m2), y, z);
          y = ex2z(y);
          z = ex2z(z);
          p[i] = bf162_of(y, z);
          if (i & 1) sum = add2(sum, pack2(y, z));
          else sum1 = add2(sum1, pack2(y, z));
        }
        tmem_st16(S + c / 2, p);  // the thread's 64 positions in 32 columns
      }
      l2 = add2(l2, add2(sum, sum1));
      // every warp sees every phase of p_done: the next one cannot complete before this warp's arrival below
      if (j > 0) ok = ok && wait(p_done, (j - 1) & 1);
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      fence_before();
      __syncwarp();
      mbar_arrive_if(p_full, lane == 0);
    }
    ok = ok && wait(p_done, (nt - 1) & 1);
    for (int i = 0; i < min(kChecked, nt - check0) * kValueUnits && ok; ++i) ok = wait(checked + 8 * i, 0);
    float l, l1;
    unpack2(l2, l, l1);
    l += l1;
    float* sums = swap + (nt & 1) * 2 * N;  // not the last tile's maxima, which may still be read
    sums[half * N + row] = l;
    if (!any256(3, !ok)) {
      fence_after();
      l = sums[row] + sums[N + row];
      const float inv = 1.0f / l;
      const bool strange = *any_odd != 0;
      const int64_t at = int64_t(it.start + tok) * a.Hq + h * a.G + row % a.G;
      if (live && a.lse && half == 0 && part == 0) a.lse[at] = (M + log2f(l)) * 0.6931471805599453f;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at * D + part * kOut + 128 * half);
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        uint32_t o[16];
        tmem_ld16(O + c, o);
        tmem_wait16(o);
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(o[i]) * inv;
        if (strange) {
          const int* at_c = odd + 128 * half + c;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (at_c[i] <= tok) x[i] = __int_as_float(0x7FC00000);
            if (at_c[kOut + i] <= tok) x[i] += INFINITY;
            if (at_c[2 * kOut + i] <= tok) x[i] -= INFINITY;
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
    } else if (lane == 0) {
      fail();
    }
  } else if (warp == kLoad) {
    // -------------------------------- loads ------------------------------------
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, C::kKeyUnits * tt * a.G * 128);
      for (int c = 0; c < C::kKeyUnits; ++c)
        tma_load_3d(base + c * kUnit, &mq, 64 * c, h * a.G, it.start + t0, q_full);
      Ring<kUnits> at;
      int issued = 0, looked = 0;
      bool ok = true;
      auto room = [&]() {
        if (ok && issued >= kUnits) ok = mbar_wait(empty + 8 * at.at, at.phase ^ 1, a.wait_turns * 1000ull);
        return ok;
      };
      auto keys = [&](int j) {
        for (int c = 0; c < C::kKeyUnits && room(); ++c) {
          mbar_arrive_expect_tx(full + 8 * at.at, kUnit);
          tma_load_2d(base + C::oRing + at.at * kUnit, &mk, h * D + 64 * c, it.start + j * kTok, full + 8 * at.at);
          at.next(), ++issued;
        }
      };
      // units that are looked through have a barrier of their own, which that pair waits for: it would be behind in the
      // phases of `full`, which here completes at once
      auto rows = [&](int j) {
        for (int i = 0; i < kValueUnits && room(); ++i) {
          uint32_t br = full + 8 * at.at;
          if (j >= check0) {
            mbar_arrive(br);
            br = values + 8 * looked++;
          }
          const uint32_t to = base + C::oRing + at.at * kUnit;
          const int x = h * D + part * kOut + 128 * (i & 1), y = it.start + j * kTok + 64 * (i >> 1);
          mbar_arrive_expect_tx(br, kUnit);
          tma_load_2d(to, &mv, x, y, br);
          tma_load_2d(to + kUnit / 2, &mv, x + 64, y, br);
          at.next(), ++issued;
        }
      };
      keys(0);
      for (int j = 0; j < nt && ok; ++j) {
        if (j + 1 < nt) keys(j + 1);
        rows(j);
      }
      if (!ok) fail();
      // what was issued lands before the block ends, also where a wait ran out
      mbar_wait(q_full, 0);
      for (int i = max(0, issued - kUnits); i < issued; ++i) mbar_wait(full + 8 * (i % kUnits), (i / kUnits) & 1);
      for (int i = 0; i < looked; ++i) mbar_wait(values + 8 * i, 0);
    }
  } else if (warp == kMma) {
    // ------------------------------- products ----------------------------------
    const uint32_t leader = elect_one();
    constexpr uint32_t id_qk = idesc_of(kTok, false, false) | kBf16, id_pv = idesc_of(128, false, true) | kBf16;
    const uint32_t dQ = desc_of(base, 16), dK = desc_of(base + C::oRing, 16), dV = desc_of(base + C::oRing, kUnit / 2);
    Waits waits{a.wait_turns};
    Ring<kUnits> at;
    auto product_qk = [&](uint32_t odd_tile) {
#pragma unroll 1
      for (int c = 0; c < C::kKeyUnits; ++c) {
        waits.on(full + 8 * at.at, at.phase);
        fence_after();
        const uint32_t q = dQ + c * (kUnit >> 4), k = dK + at.at * (kUnit >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16_ss(cS + 128 * odd_tile, q + 2 * j, k + 2 * j, id_qk, c | j, leader);
        mma_commit(empty + 8 * at.at, leader);
        at.next();
      }
      mma_commit(s_full + 8 * odd_tile, leader);
    };
    auto product_pv = [&](int j) {
      waits.on(p_full, j & 1);
#pragma unroll 1
      for (int i = 0; i < kValueUnits; ++i) {
        waits.on(full + 8 * at.at, at.phase);
        if (j >= check0) waits.on(checked + 8 * ((j - check0) * kValueUnits + i), 0);
        fence_after();
        const uint32_t v = dV + at.at * (kUnit >> 4), p = cS + 128 * (j & 1) + 64 * (i >> 1);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16_ts(cO + 128 * (i & 1), p + 8 * k, v + 128 * k, id_pv, j > 0 || i > 1 || k > 0, leader);
        mma_commit(empty + 8 * at.at, leader);
        at.next();
      }
      mma_commit(p_done, leader);
    };
    waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
    waits.on(q_full, 0);
    fence_after();
    if (__all_sync(0xffffffffu, waits.ok)) product_qk(0);
#pragma unroll 1
    for (int j = 0; j < nt; ++j) {
      if (!__all_sync(0xffffffffu, waits.ok)) break;
      // scores of tile j + 1 go where P of tile j - 1 was, whose products were issued before
      if (j + 1 < nt) product_qk((j + 1) & 1);
      if (!__all_sync(0xffffffffu, waits.ok)) break;
      product_pv(j);
    }
    if (!__all_sync(0xffffffffu, waits.ok) && lane == 0) fail();
    mma_commit(drained, leader);  // every product issued is complete before TMEM is freed
    mbar_wait(drained, 0);
    __syncwarp();
  } else {
    // ---------------------------- a look through V ------------------------------
    bool ok = true;
    // units behind those of tile j: the keys of tiles 0 .. j + 1 and the values of tiles 0 .. j - 1
#pragma unroll 1
    for (int j = check0; j < nt && ok; ++j)
#pragma unroll 1
      for (int i = 0; i < kValueUnits && ok; ++i) {
        const int unit = min(j + 2, nt) * C::kKeyUnits + j * kValueUnits + i, n = (j - check0) * kValueUnits + i;
        ok = wait(values + 8 * n, 0);
        int* to = odd + 128 * (i & 1);
        if (ok)
          check_values<64, kOut>(sm + C::oRing + (unit % kUnits) * kUnit, to, j * kTok + 64 * (i >> 1), t0, it.len,
                                 threadIdx.x - kCheck * 32);
        __syncwarp();
        for (int c = lane; c < 3 * kOut; c += 32)
          if (odd[c] != 0x7fffffff) *any_odd = 1;
        fence_async();
        __syncwarp();
        mbar_arrive_if(checked + 8 * n, lane == 0);
      }
    if (!ok && lane == 0) fail();
  }
  fence_before();
  __syncthreads();
  if (warp == kMma) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int D>
int launch_d(const PromptArgs& a, cudaStream_t stream) {
  using C = Wide<D>;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!done[dev]) {
    if (cudaFuncSetAttribute(attn_prompt_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    done[dev] = true;
  }
  const int tt = N / a.G;
  CUtensorMap mq, mk, mv;
  if (!encode_heads_bf16(&mq, a.q, uint64_t(a.n), a.Hq, D, uint32_t(a.G), uint32_t(tt)) ||
      !encode_rows_bf16(&mk, a.k, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok) ||
      !encode_rows_bf16(&mv, a.v, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, 64))
    return OSCAR_ERR_LAUNCH;
  const int64_t items = prompt_items(a, 1, tt) * a.Hkv * (D / kOut);
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_prompt_wide_kernel<D><<<unsigned(items), kThreads, C::kBytes, stream>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace

int launch_attn_prompt_wide(const PromptArgs& a, cudaStream_t stream) {
  return a.D == 256 ? launch_d<256>(a, stream) : launch_d<512>(a, stream);
}

}  // namespace oscar
