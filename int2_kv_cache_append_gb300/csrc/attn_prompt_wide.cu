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
// exchange their maxima once per tile.  What bounds it at head_dim 256 is what
// bounds head_dim 128 (8192 tokens, 16 heads: 356 us, 1.54 PFLOP/s); at 512 a third
// of the products are the second half's scores, and 80 KB of units under way do not
// cover the way from L2 (8192 tokens 1.06 ms, 1.04 PFLOP/s without those; four
// ragged prompts of 2048 329 us, 0.48).  Arithmetic, masks, the look through V and
// the order of the items are those of head_dim 128 (attn_prompt_tc.cu).
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
constexpr int kItems = 3;              // items found ahead
constexpr uint32_t cS = 0, cO = 256;   // TMEM columns: two score tiles, O

template <int D>
struct Wide {
  static constexpr int kKeyUnits = D / 64;
  static constexpr int kUnits = D == 256 ? 9 : 5;
  static constexpr int oRing = D * N * 2;
  static constexpr int oOdd = oRing + kUnits * kUnit;
  static constexpr int oSwap = oOdd + 3 * kOut * 4;  // maxima [2][2][N], both sums [2][N]
  static constexpr int oBar = oSwap + 8 * N * 4;
  static constexpr int kBars = 2 * kUnits + 2 + 2 + 1 + 1 + 2 * kChecked * kValueUnits + 1 + 1 + 2 * kItems + 1;
  static constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;
  static_assert(oBar % 8 == 0 && kBytes <= 232448 - 64, "shared memory");
};

// Barriers, by their order in shared memory.
template <int kUnits>
struct WideBars {
  uint32_t full, empty, q_full, q_empty, s_full, p_full, p_done, values, checked, looked, odd_free, item_full, item_empty, drained;
  __device__ __forceinline__ explicit WideBars(uint32_t at) {
    full = at, empty = full + 8 * kUnits, q_full = empty + 8 * kUnits, q_empty = q_full + 8, s_full = q_empty + 8,
    p_full = s_full + 16, p_done = p_full + 8, values = p_done + 8, checked = values + 8 * kChecked * kValueUnits,
    looked = checked + 8 * kChecked * kValueUnits, odd_free = looked + 8, item_full = odd_free + 8,
    item_empty = item_full + 8 * kItems, drained = item_empty + 8 * kItems;
  }
};

// An item as all roles see it: its sequence, head and half of the channels, first token, tiles of positions.
struct WideWork {
  int start, len, h, part, t0, nt, check0;
  __device__ __forceinline__ WideWork(const PromptItem& it, int head, int parts, int tt)
      : start(it.start), len(it.len), h(head / parts), part(head % parts), t0(it.tile * tt) {
    nt = (min(t0 + tt, len) + kTok - 1) / kTok;
    check0 = (t0 + 1) / kTok;  // the first tile with a token behind t0
  }
  __device__ __forceinline__ int checks() const { return max(0, min(kChecked, nt - check0)); }
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
  __shared__ PromptItem items[kItems];
  __shared__ int heads[kItems];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = N / a.G;
  const WideBars<kUnits> bar(base + C::oBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::oBar + C::kBars * 8);
  int* any_odd = reinterpret_cast<int*>(tmem_slot + 1);
  int* odd = reinterpret_cast<int*>(sm + C::oOdd);
  float* swap = reinterpret_cast<float*>(sm + C::oSwap);
  if (threadIdx.x == kLoad * 32) {
    for (int i = 0; i < kUnits; ++i) mbar_init(bar.full + 8 * i, 1), mbar_init(bar.empty + 8 * i, 1);
    mbar_init(bar.q_full, 1), mbar_init(bar.q_empty, 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar.s_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
    mbar_init(bar.p_full, kSoftWarps);
    mbar_init(bar.p_done, 1);
    for (int i = 0; i < kChecked * kValueUnits; ++i) mbar_init(bar.values + 8 * i, 1), mbar_init(bar.checked + 8 * i, 2);
    mbar_init(bar.looked, 2);
    mbar_init(bar.odd_free, kSoftWarps);
    for (int i = 0; i < kItems; ++i) mbar_init(bar.item_full + 8 * i, 1), mbar_init(bar.item_empty + 8 * i, kSoftWarps + 3);
    mbar_init(bar.drained, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == kCheck * 32) *any_odd = 0;
  if (warp >= kCheck)
    for (int i = threadIdx.x - kCheck * 32; i < 3 * kOut; i += 64) odd[i] = 0x7fffffff;
  if (warp == kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;
  auto fail = [&]() { status_or(a.status, OSCAR_DEV_TIMEOUT); };
  auto wait = [&](uint32_t br, uint32_t parity) { return wait_warp(br, parity, a.wait_turns); };
  // The next item, by every warp but the loads': false at the end (or where a wait ran out: ok).
  auto next = [&](Ring<kItems>& at, bool& ok, PromptItem& it, int& head) {
    ok = wait(bar.item_full + 8 * at.at, at.phase);
    if (!ok) return false;
    it = items[at.at], head = heads[at.at];
    __syncwarp();
    mbar_arrive_if(bar.item_empty + 8 * at.at, lane == 0);
    at.next();
    return it.b >= 0;
  };
  Ring<kItems> at_item;
  PromptItem it;
  int head;

  if (warp < kSoftWarps) {
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t O = tmem + lanes + cO + 128 * half;
    float2* shared_sums = reinterpret_cast<float2*>(swap + 4 * N);
    uint32_t tile = 0, p_phase = 0, l_phase = 0;  // tile: of all items, s_full and the maxima alternate by it
    bool ok = true;
#pragma unroll 1
    while (next(at_item, ok, it, head)) {
      const WideWork x(it, head, kParts, tt);
      const int tok = x.t0 + row / a.G;
      const bool live = row < tt * a.G && tok < x.len;
      const int lim = live ? tok : -1, least = x.t0 + (row & ~31) / a.G;
      Reference ref;
      RowSums sums;
#pragma unroll 1
      for (int j = 0; j < x.nt; ++j, ++tile) {
        const uint32_t S = tmem + lanes + cS + 128 * (tile & 1) + 64 * half;
        ok = ok && wait(bar.s_full + 8 * (tile & 1), tile >> 1 & 1);
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
        float* mine = swap + (tile & 1) * 2 * N;
        mine[half * N + row] = fmaxf(top, top1);
        if (any256(3, !ok)) {
          ok = false;
          break;
        }
        const float most = fmaxf(mine[row], mine[N + row]);
        const bool grow = most * ref.scale > ref.M + kTop;
        bool done = j == 0;  // the products of the tile before
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ref.follow(most, a.qscale) : 1.f;
          sums.scale(f);
          if (j > 0) {
            ok = wait(bar.p_done, p_phase);  // O is not in use
            p_phase ^= 1;
            done = true;
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
        const uint64_t scale2 = splat_x2(ref.scale), m2 = splat_x2(-ref.M);
        TileSums part;
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
            part.add(i & 1, y, z, p[i]);
          }
          tmem_st16(S + c / 2, p);  // the thread's 64 positions in 32 columns
        }
        part.into(sums);
        // every warp sees every phase of p_done: the next one cannot complete before this warp's arrival below
        if (!done) {
          ok = ok && wait(bar.p_done, p_phase);
          p_phase ^= 1;
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        mbar_arrive_if(bar.p_full, lane == 0);
      }
      ok = ok && wait(bar.p_done, p_phase);
      p_phase ^= 1;
      ok = ok && wait(bar.looked, l_phase);
      l_phase ^= 1;
      shared_sums[half * N + row] = sums.total();
      if (any256(3, !ok)) {
        ok = false;
        break;
      }
      fence_after();
      const float l = shared_sums[row].x + shared_sums[N + row].x;
      const float inv = 1.0f / (shared_sums[row].y + shared_sums[N + row].y);
      const bool strange = *any_odd != 0;
      const int64_t at = int64_t(x.start + tok) * a.Hq + x.h * a.G + row % a.G;
      if (live && a.lse && half == 0 && x.part == 0) a.lse[at] = ref.lse(l, a.qscale);
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at * D + x.part * kOut + 128 * half;
      const bool aligned32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        uint32_t o[16];
        tmem_ld16(O + c, o);
        tmem_wait16(o);
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * inv;
        if (strange) {
          const int* at_c = odd + 128 * half + c;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (at_c[i] <= tok) y[i] = __int_as_float(0x7FC00000);
            if (at_c[kOut + i] <= tok) y[i] += INFINITY;
            if (at_c[2 * kOut + i] <= tok) y[i] -= INFINITY;
          }
        }
        if (live) store16(dst + c, y, aligned32);
      }
      fence_before();  // O has been read when the next item's first P arrives
      __syncwarp();
      mbar_arrive_if(bar.odd_free, lane == 0);
    }
    if (!ok && lane == 0) fail();
  } else if (warp == kLoad) {
    // -------------------------------- loads ------------------------------------
    // It also finds the items, in the order of prompt_item, dealt to the blocks forth and back, so that those with the
    // longest of one round have the shortest of the next.
    const int64_t each = int64_t(a.Hkv) * kParts, total = prompt_items(a, 1, tt) * each;
    if (blockIdx.x == 0) prompt_check(a);
    const uint64_t limit = a.wait_turns * 1000ull;
    Ring<kUnits> at;
    uint32_t v_phase = 0, v_used = 0;  // bits of `values`
    int64_t round = 0;
    int level = -1, published = 0, issued = 0;
    bool ok = true;
#pragma unroll 1
    for (;;) {
      it = PromptItem{-1, 0, 0, 0};
      head = 0;
      while (round * gridDim.x < total) {
        const int64_t i = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        ++round;
        if (i >= total) continue;
        it = prompt_item(a, int(i / each), 1, tt, level);
        head = int(i % each);
        break;
      }
      const WideWork x(it, head, kParts, tt);
      // `looked` of the item before, waited for once it is needed: before values are loaded that are looked through.  An item
      // without such values (its only token ends a position tile) has its own `looked` as soon as the rows of the item before
      // are written; a wait for that one's phase would then be a phase late and never end.  So it comes first.
      bool told = published == 0;
      if (!told && it.b >= 0 && x.checks() == 0) ok = wait(bar.looked, (published - 1) & 1), told = true;
      if (ok && published >= kItems) ok = wait(bar.item_empty + 8 * at_item.at, at_item.phase ^ 1);
      if (!ok) break;
      if (lane == 0) {
        items[at_item.at] = it, heads[at_item.at] = head;
        mbar_arrive(bar.item_full + 8 * at_item.at);
      }
      at_item.next();
      if (it.b < 0) break;
      if (lane == 0) {
        auto room = [&]() {
          if (ok && issued >= kUnits) ok = mbar_wait(bar.empty + 8 * at.at, at.phase ^ 1, limit);
          return ok;
        };
        auto keys = [&](int j) {
          for (int c = 0; c < C::kKeyUnits && room(); ++c) {
            mbar_arrive_expect_tx(bar.full + 8 * at.at, kUnit);
            tma_load_2d(base + C::oRing + at.at * kUnit, &mk, x.h * D + 64 * c, x.start + j * kTok, bar.full + 8 * at.at);
            at.next(), ++issued;
          }
        };
        auto before = [&]() {  // the item before has been looked through
          if (!told && ok) ok = mbar_wait(bar.looked, (published - 1) & 1, limit);
          told = true;
        };
        // units that are looked through have a barrier of their own, which that pair waits for: it would be behind in the
        // phases of `full`, which here completes at once
        auto rows = [&](int j) {
          if (j >= x.check0) before();
          for (int i = 0; i < kValueUnits && room(); ++i) {
            uint32_t br = bar.full + 8 * at.at;
            if (j >= x.check0) {
              mbar_arrive(br);
              const int n = (j - x.check0) * kValueUnits + i;
              br = bar.values + 8 * n;
              v_used |= 1u << n, v_phase ^= 1u << n;
            }
            const uint32_t to = base + C::oRing + at.at * kUnit;
            const int c = x.h * D + x.part * kOut + 128 * (i & 1), y = x.start + j * kTok + 64 * (i >> 1);
            mbar_arrive_expect_tx(br, kUnit);
            tma_load_2d(to, &mv, c, y, br);
            tma_load_2d(to + kUnit / 2, &mv, c + 64, y, br);
            at.next(), ++issued;
          }
        };
        // once the products of the item before have read its queries
        if (published > 0) ok = mbar_wait(bar.q_empty, (published - 1) & 1, limit);
        if (ok) {
          mbar_arrive_expect_tx(bar.q_full, C::kKeyUnits * tt * a.G * 128);
          for (int c = 0; c < C::kKeyUnits; ++c)
            tma_load_3d(base + c * kUnit, &mq, 64 * c, x.h * a.G, x.start + x.t0, bar.q_full);
          keys(0);
        }
        for (int j = 0; j < x.nt && ok; ++j) {
          if (j + 1 < x.nt) keys(j + 1);
          rows(j);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++published;
      if (!ok) break;
    }
    if (lane == 0) {
      if (!ok) fail();
      // what was issued lands before the block ends, also where a wait ran out (an item's queries come before its keys)
      for (int i = max(0, issued - kUnits); i < issued; ++i) mbar_wait(bar.full + 8 * (i % kUnits), (i / kUnits) & 1);
      for (int i = 0; i < kChecked * kValueUnits; ++i)
        if (v_used >> i & 1) mbar_wait(bar.values + 8 * i, (v_phase >> i & 1) ^ 1);
    }
  } else if (warp == kMma) {
    // ------------------------------- products ----------------------------------
    const uint32_t leader = elect_one();
    constexpr uint32_t id_qk = idesc_of(kTok, false, false) | kBf16, id_pv = idesc_of(128, false, true) | kBf16;
    const uint32_t dQ = desc_of(base, 16), dK = desc_of(base + C::oRing, 16), dV = desc_of(base + C::oRing, kUnit / 2);
    Waits waits{a.wait_turns};
    Ring<kUnits> at;
    uint32_t tile = 0, p_phase = 0, q_phase = 0, c_phase = 0;  // c_phase: bits of `checked`
    bool ok = true;
    auto product_qk = [&](uint32_t odd_tile) {
#pragma unroll 1
      for (int c = 0; c < C::kKeyUnits; ++c) {
        waits.on(bar.full + 8 * at.at, at.phase);
        fence_after();
        const uint32_t q = dQ + c * (kUnit >> 4), k = dK + at.at * (kUnit >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma_f16_ss(cS + 128 * odd_tile, q + 2 * j, k + 2 * j, id_qk, c | j, leader);
        mma_commit(bar.empty + 8 * at.at, leader);
        at.next();
      }
      mma_commit(bar.s_full + 8 * odd_tile, leader);
    };
    waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
#pragma unroll 1
    while (__all_sync(0xffffffffu, waits.ok) && next(at_item, ok, it, head)) {
      const WideWork x(it, head, kParts, tt);
      waits.on(bar.q_full, q_phase);
      q_phase ^= 1;
      fence_after();
      if (!__all_sync(0xffffffffu, waits.ok)) break;
      product_qk(tile & 1);
      if (x.nt == 1) mma_commit(bar.q_empty, leader);
#pragma unroll 1
      for (int j = 0; j < x.nt; ++j, ++tile) {
        if (!__all_sync(0xffffffffu, waits.ok)) break;
        // scores of tile j + 1 go where P of tile j - 1 was, whose products were issued before
        if (j + 1 < x.nt) {
          product_qk((tile + 1) & 1);
          if (j + 2 == x.nt) mma_commit(bar.q_empty, leader);
        }
        waits.on(bar.p_full, p_phase);
        p_phase ^= 1;
        if (!__all_sync(0xffffffffu, waits.ok)) break;
#pragma unroll 1
        for (int i = 0; i < kValueUnits; ++i) {
          waits.on(bar.full + 8 * at.at, at.phase);
          if (j >= x.check0) {
            const int n = (j - x.check0) * kValueUnits + i;
            waits.on(bar.checked + 8 * n, c_phase >> n & 1);
            c_phase ^= 1u << n;
          }
          fence_after();
          const uint32_t v = dV + at.at * (kUnit >> 4), p = cS + 128 * (tile & 1) + 64 * (i >> 1);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ts(cO + 128 * (i & 1), p + 8 * k, v + 128 * k, id_pv, j > 0 || i > 1 || k > 0, leader);
          mma_commit(bar.empty + 8 * at.at, leader);
          at.next();
        }
        mma_commit(bar.p_done, leader);
      }
    }
    if (!__all_sync(0xffffffffu, waits.ok && ok) && lane == 0) fail();
    mma_commit(bar.drained, leader);  // every product issued is complete before TMEM is freed
    mbar_wait(bar.drained, 0);
    __syncwarp();
  } else {
    // ---------------------------- a look through V ------------------------------
    const int me = threadIdx.x - kCheck * 32;
    uint32_t v_phase = 0, free_phase = 1;
    int first = 0;  // the item's first unit, modulo the ring
    bool ok = true;
#pragma unroll 1
    while (next(at_item, ok, it, head)) {
      const WideWork x(it, head, kParts, tt);
      // the rows of the item before have been written (of the first: at once)
      ok = wait(bar.odd_free, free_phase);
      if (!ok) break;
      free_phase ^= 1;
      asm volatile("bar.sync 4, 64;" ::: "memory");
      const bool reset = *any_odd != 0;
      asm volatile("bar.sync 4, 64;" ::: "memory");
      if (reset) {
        for (int i = me; i < 3 * kOut; i += 64) odd[i] = 0x7fffffff;
        if (me == 0) *any_odd = 0;
        asm volatile("bar.sync 4, 64;" ::: "memory");
      }
#pragma unroll 1
      for (int n = 0; n < x.checks() * kValueUnits; ++n) {
        const int j = x.check0 + n / kValueUnits, i = n % kValueUnits;
        ok = wait(bar.values + 8 * n, v_phase >> n & 1);
        if (!ok) break;
        v_phase ^= 1u << n;
        // units of the item before this one: the keys of tiles 0 .. j + 1 and the values of tiles 0 .. j - 1
        const int unit = (first + min(j + 2, x.nt) * C::kKeyUnits + j * kValueUnits + i) % kUnits;
        check_values<64, kOut>(sm + C::oRing + unit * kUnit, odd + 128 * (i & 1), j * kTok + 64 * (i >> 1), x.t0, x.len, me);
        __syncwarp();
        for (int c = lane; c < 3 * kOut; c += 32)
          if (odd[c] != 0x7fffffff) *any_odd = 1;
        fence_async();
        __syncwarp();
        mbar_arrive_if(bar.checked + 8 * n, lane == 0);
      }
      if (!ok) break;
      __syncwarp();
      mbar_arrive_if(bar.looked, lane == 0);
      first = (first + x.nt * (C::kKeyUnits + kValueUnits)) % kUnits;
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
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!sms[dev]) {
    int n = 0;
    if (cudaFuncSetAttribute(attn_prompt_wide_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    sms[dev] = n;
  }
  const int tt = N / a.G;
  CUtensorMap mq, mk, mv;
  if (!encode_heads_bf16(&mq, a.q, uint64_t(a.n), a.Hq, D, uint32_t(a.G), uint32_t(tt)) ||
      !encode_rows_bf16(&mk, a.k, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok) ||
      !encode_rows_bf16(&mv, a.v, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, 64))
    return OSCAR_ERR_LAUNCH;
  const int64_t items = prompt_items(a, 1, tt) * a.Hkv * (D / kOut);
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_prompt_wide_kernel<D><<<unsigned(std::min<int64_t>(items, sms[dev])), kThreads, C::kBytes, stream>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace

int launch_attn_prompt_wide(const PromptArgs& a, cudaStream_t stream) {
  return a.D == 256 ? launch_d<256>(a, stream) : launch_d<512>(a, stream);
}

}  // namespace oscar
