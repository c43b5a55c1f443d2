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
// A block stays for many items: the loads, which also find the items, run ahead into
// the next one's tiles, and its first products run under the last one's softmax and
// output.
//
// Softmax: a thread has a row; its reference M lies 2^12 above the row's maximum when
// it is chosen and follows it only when that has grown by 2^20, which makes the
// warp rescale its rows of O: P and O are floating point, so they lose nothing by
// it, and 2^20 is hardly ever reached (M at the maximum, followed from 2^8 on: 522 us
// instead of 450 for eight ragged prompts of activations with outliers).  P is
// rounded to bf16, V's type.  With M at the maximum the largest weight would be 1,
// without a rounding; anywhere else it has one like the others, so O is divided by the
// sum of the rounded weights (RowSums), in float32; lse has the sum before the rounding.
//
// Positions that some of the block's rows do not see: their scores are set to
// -inf, which makes P zero, and a warp pair looks through those V rows first: where
// a value is infinite or not a number, zero times it would reach every row.  It is
// replaced by zero there, and added to the rows that see it at the end.
//
// What bounds it: over long sequences the tensor cores (16,384 tokens, 32 heads:
// 1.43 ms, 1.54 PFLOP/s of the products that a causal mask leaves, 82 % of cuBLAS's
// rate); over short ones the hand-over from item to item, where the output is read,
// scaled and stored while the next scores wait (eight ragged prompts of up to 4096
// tokens 463 us, 64 %; 64 of 512 217 us, 34 %).
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
constexpr int oQ = 0, oKV = 2 * kTile, oOdd = oKV + kStages * kTile, oBar = oOdd + 3 * D * 4;
constexpr int kItems = 3;              // items found ahead
constexpr int kBars = 2 * kStages + 5 * 2 + 2 * kChecked + 1 + 2 * kItems + 1;
constexpr int kBytes = oBar + kBars * 8 + 32 + 1024;  // + alignment slack
static_assert(oBar % 8 == 0 && kBytes <= 232448 - 64, "shared memory");
constexpr uint32_t cS = 0, cO = 256;   // TMEM columns, 128 per tile
constexpr int kSoftRegs = 216, kOtherRegs = 72;
static_assert(2 * kSoftRegs + kOtherRegs <= 3 * 168, "registers of a launch with 168 a thread");

// Barriers, by their order in shared memory.
struct Bars {
  uint32_t full, empty, q_full, q_empty, s_full, p_full, o_full, values, checked, odd_free, item_full, item_empty, drained;
  __device__ __forceinline__ explicit Bars(uint32_t at) {
    full = at, empty = full + 8 * kStages, q_full = empty + 8 * kStages, q_empty = q_full + 16, s_full = q_empty + 16,
    p_full = s_full + 16, o_full = p_full + 16, values = o_full + 16, checked = values + 8 * kChecked,
    odd_free = checked + 8 * kChecked, item_full = odd_free + 8, item_empty = item_full + 8 * kItems,
    drained = item_empty + 8 * kItems;
  }
};

// An item as all roles see it: its sequence and head, first token, tiles of positions of both query tiles.
struct Work {
  int start, len, h, t0, nA, nB, nt, check0;
  __device__ __forceinline__ Work(const PromptItem& it, int head, int tt) : start(it.start), len(it.len), h(head), t0(it.tile * 2 * tt) {
    auto tiles = [&](int first) { return first < len ? (min(first + tt, len) + kTok - 1) / kTok : 0; };
    nA = tiles(t0), nB = tiles(t0 + tt), nt = max(nA, nB);
    check0 = (t0 + 1) / kTok;  // the first tile with a token behind t0
  }
  __device__ __forceinline__ int checks() const { return max(0, min(kChecked, nt - check0)); }
};

__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const PromptArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base - raw);
  __shared__ PromptItem items[kItems];
  __shared__ int heads[kItems];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tt = N / a.G;  // tokens of a tile
  const Bars bar(base + oBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + oBar + kBars * 8);
  int* odd = reinterpret_cast<int*>(sm + oOdd);
  int* any_odd = reinterpret_cast<int*>(tmem_slot + 1);
  if (threadIdx.x == kLoad * 32) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar.full + 8 * i, 1), mbar_init(bar.empty + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.q_full + 8 * i, 1), mbar_init(bar.q_empty + 8 * i, 1);
      mbar_init(bar.s_full + 8 * i, 1 + (i == 0 && a.wait_poison > 0));
      mbar_init(bar.p_full + 8 * i, 4);
      mbar_init(bar.o_full + 8 * i, 1);
    }
    for (int i = 0; i < kChecked; ++i) mbar_init(bar.values + 8 * i, 1), mbar_init(bar.checked + 8 * i, 2);
    mbar_init(bar.odd_free, kSoftWarps);
    for (int i = 0; i < kItems; ++i) mbar_init(bar.item_full + 8 * i, 1), mbar_init(bar.item_empty + 8 * i, kSoftWarps + 3);
    mbar_init(bar.drained, 1);
    mbar_fence_init();
  }
  if (threadIdx.x == kCheck * 32) *any_odd = 0;
  if (warp >= kCheck)
    for (int i = threadIdx.x - kCheck * 32; i < 3 * D; i += 64) odd[i] = 0x7fffffff;
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
  auto next = [&](Ring<kItems>& at, bool& ok, PromptItem& it, int& h) {
    ok = wait(bar.item_full + 8 * at.at, at.phase);
    if (!ok) return false;
    it = items[at.at], h = heads[at.at];
    __syncwarp();
    mbar_arrive_if(bar.item_empty + 8 * at.at, lane == 0);
    at.next();
    return it.b >= 0;
  };

  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
    const uint32_t S = tmem + lanes + cS + 128 * w, O = tmem + lanes + cO + 128 * w;
    uint32_t s_phase = 0, o_phase = 0, c_phase = 0;
    Ring<kItems> at_item;
    bool ok = true;
    PromptItem it;
    int h;
#pragma unroll 1
    while (next(at_item, ok, it, h)) {
      const Work x(it, h, tt);
      const int n = w ? x.nB : x.nA, first = x.t0 + w * tt, tok = first + row / a.G;
      const bool live = row < tt * a.G && tok < x.len;
      const int lim = live ? tok : -1, least = first + (row & ~31) / a.G;  // the warp's first token
      Reference ref;
      RowSums sums;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        ok = wait(bar.s_full + 8 * w, s_phase);
        if (!ok) break;
        s_phase ^= 1;
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
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const bool grow = most * ref.scale > ref.M + kTop;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ref.follow(most, a.qscale) : 1.f;
          sums.scale(f);
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
        const uint64_t scale2 = splat_x2(ref.scale), m2 = splat_x2(-ref.M);
        TileSums part;
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
              part.add(i & 1, y, z, p[i]);
            }
            tmem_st16(to + c / 2, p);
          }
        };
        half(r, S);
        half(u, S + 32);
        part.into(sums);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        mbar_arrive_if(bar.p_full + 8 * w, lane == 0);
      }
      if (ok && n > 0) {
        ok = wait(bar.o_full + 8 * w, o_phase);
        o_phase ^= 1;
      }
      for (int i = 0; i < kChecked; ++i) ok = ok && wait(bar.checked + 8 * i, c_phase);
      c_phase ^= 1;
      if (!ok) break;
      if (n > 0) {
        fence_after();
        const float2 l = sums.total();
        const float inv = 1.0f / l.y;
        const bool strange = *any_odd != 0;
        const int64_t at = int64_t(x.start + tok) * a.Hq + x.h * a.G + row % a.G;
        if (live && a.lse) a.lse[at] = ref.lse(l.x, a.qscale);
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + at * D;
        const bool aligned32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[2][16];
          tmem_ld16(O + c, o[0]);
          tmem_ld16(O + c + 16, o[1]);
          tmem_wait16(o[0]);
          tmem_wait16(o[1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[e][i]) * inv;
            if (strange) {
              const int* at_c = odd + c + 16 * e;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (at_c[i] <= tok) y[i] = __int_as_float(0x7FC00000);
                if (at_c[D + i] <= tok) y[i] += INFINITY;
                if (at_c[2 * D + i] <= tok) y[i] -= INFINITY;
              }
            }
            if (live) store16(dst + c + 16 * e, y, aligned32);
          }
        }
        fence_before();  // O has been read when the next item's first P arrives
      }
      __syncwarp();
      mbar_arrive_if(bar.odd_free, lane == 0);
    }
    if (!ok && lane == 0) fail();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoad) {
      // ------------------------------- loads -----------------------------------
      // It also finds the items, in the order of prompt_item, dealt to the blocks forth and back, so that those with the
      // longest of one round have the shortest of the next.
      const int64_t total = prompt_items(a, 1, 2 * tt) * a.Hkv;
      if (blockIdx.x == 0) prompt_check(a);
      const uint64_t limit = a.wait_turns * 1000ull;
      Ring<kItems> at_item;
      Ring<kStages> at;
      uint32_t q_phase = 0, q_used = 0, v_phase = 0, v_used = 0, c_phase = 0;  // bits of the barriers of a kind
      int64_t round = 0;
      int level = -1;
      int published = 0, issued = 0;
      bool ok = true;
#pragma unroll 1
      for (;;) {
        PromptItem it{-1, 0, 0, 0};
        int h = 0;
        while (round * gridDim.x < total) {
          const int64_t i = round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
          ++round;
          if (i >= total) continue;
          it = prompt_item(a, int(i / a.Hkv), 1, 2 * tt, level);
          h = int(i % a.Hkv);
          break;
        }
        if (published >= kItems) ok = wait(bar.item_empty + 8 * at_item.at, at_item.phase ^ 1);
        if (!ok) break;
        if (lane == 0) {
          items[at_item.at] = it, heads[at_item.at] = h;
          mbar_arrive(bar.item_full + 8 * at_item.at);
        }
        at_item.next();
        if (it.b < 0) break;
        if (lane == 0) {
          const Work x(it, h, tt);
          auto room = [&]() {
            if (ok && issued >= kStages) ok = mbar_wait(bar.empty + 8 * at.at, at.phase ^ 1, limit);
            return ok;
          };
          auto tile = [&](const CUtensorMap* map, int token, uint32_t br) {
            const uint32_t to = base + oKV + at.at * kTile;
            mbar_arrive_expect_tx(br, kTile);
            tma_load_2d(to, map, x.h * D, x.start + token, br);
            tma_load_2d(to + kTile / 2, map, x.h * D + 64, x.start + token, br);
            at.next(), ++issued;
          };
          auto queries = [&](int w) {  // once the products of the item before that has the tile have read it
            if (ok && (q_used >> w & 1)) ok = mbar_wait(bar.q_empty + 8 * w, (q_phase >> w & 1) ^ 1, limit);
            if (!ok) return;
            mbar_arrive_expect_tx(bar.q_full + 8 * w, 2 * tt * a.G * 128);
            for (int c = 0; c < 2; ++c)
              tma_load_3d(base + oQ + w * kTile + c * (kTile / 2), &mq, 64 * c, x.h * a.G, x.start + x.t0 + w * tt, bar.q_full + 8 * w);
            q_used |= 1u << w, q_phase ^= 1u << w;
          };
          bool told = published == 0;
          auto before = [&]() {  // the item before has been looked through
            for (int i = 0; i < kChecked && !told && ok; ++i) ok = mbar_wait(bar.checked + 8 * i, c_phase, limit);
            if (!told) c_phase ^= 1;
            told = true;
          };
          for (int j = 0; j < x.nt && ok; ++j) {
            if (room()) tile(&mk, j * kTok, bar.full + 8 * at.at);
            if (j == 0) {
              queries(0);
              if (x.nB > 0) queries(1);
            }
            // V tiles that are looked through have a barrier of their own, which that pair of warps waits for: it would be
            // behind in the phases of `full`, which here completes at once
            if (j >= x.check0) before();
            if (!room()) break;
            uint32_t br = bar.full + 8 * at.at;
            if (j >= x.check0) {
              mbar_arrive(br);
              const int i = j - x.check0;
              br = bar.values + 8 * i;
              v_used |= 1u << i, v_phase ^= 1u << i;
            }
            tile(&mv, j * kTok, br);
          }
          if (ok) before();
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++published;
        if (!ok) break;
      }
      if (lane == 0) {
        if (!ok) fail();
        // what was issued lands before the block ends, also where a wait ran out
        for (int i = 0; i < 2; ++i) {
          if (q_used >> i & 1) mbar_wait(bar.q_full + 8 * i, (q_phase >> i & 1) ^ 1);
          if (v_used >> i & 1) mbar_wait(bar.values + 8 * i, (v_phase >> i & 1) ^ 1);
        }
        for (int i = max(0, issued - kStages); i < issued; ++i) mbar_wait(bar.full + 8 * (i % kStages), (i / kStages) & 1);
      }
    } else if (warp == kMma) {
      // ------------------------------ products ---------------------------------
      const uint32_t leader = elect_one();
      constexpr uint32_t id_qk = idesc_of(kTok, false, false) | kBf16, id_pv = idesc_of(D, false, true) | kBf16;
      const uint32_t dQ = desc_of(base + oQ, 16), dK = desc_of(base + oKV, 16), dV = desc_of(base + oKV, kTile / 2);
      Waits waits{a.wait_turns};
      Ring<kStages> kr, vr;  // stages of the next K and V tile, which alternate
      vr.next();
      auto product_qk = [&](int w) {
        const uint32_t k = dK + kr.at * (kTile >> 4), q = dQ + w * (kTile >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          mma_f16_ss(cS + 128 * w, q + (j >> 2) * (kTile >> 5) + 2 * (j & 3), k + (j >> 2) * (kTile >> 5) + 2 * (j & 3), id_qk, j > 0, leader);
        mma_commit(bar.s_full + 8 * w, leader);
      };
      auto product_pv = [&](int w, uint32_t acc) {
        const uint32_t v = dV + vr.at * (kTile >> 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) mma_f16_ts(cO + 128 * w, cS + 128 * w + 8 * j, v + 128 * j, id_pv, j ? 1 : acc, leader);
      };
      waits.ok &= tmem == 0;  // all of TMEM: column addresses are constants
      uint32_t q_phase[2] = {0, 0}, p_phase[2] = {0, 0}, c_phase = 0;
      Ring<kItems> at_item;
      bool ok = true;
      PromptItem it;
      int h;
#pragma unroll 1
      while (__all_sync(0xffffffffu, waits.ok) && next(at_item, ok, it, h)) {
        const Work x(it, h, tt);
        const int n[2] = {x.nA, x.nB};
        waits.on(bar.full + 8 * kr.at, kr.phase);
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (n[w] > 0) {
            waits.on(bar.q_full + 8 * w, q_phase[w]);
            q_phase[w] ^= 1;
            fence_after();
            if (!__all_sync(0xffffffffu, waits.ok)) break;
            product_qk(w);
            if (n[w] == 1) mma_commit(bar.q_empty + 8 * w, leader);
          }
        if (!__all_sync(0xffffffffu, waits.ok)) break;
        mma_commit(bar.empty + 8 * kr.at, leader);
        kr.next(), kr.next();
#pragma unroll 1
        for (int j = 0; j < x.nt; ++j) {
          waits.on(bar.full + 8 * vr.at, vr.phase);
          if (j >= x.check0) waits.on(bar.checked + 8 * (j - x.check0), c_phase);
          const bool more = j + 1 < x.nt;
          // The phases of tiles that the item does not have: before its last product, without which no row is written and so
          // nothing of the next item looked through.
          if (!more) {
            for (int i = x.checks(); i < kChecked; ++i) waits.on(bar.checked + 8 * i, c_phase);
            c_phase ^= 1;
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (j < n[w]) {
              waits.on(bar.p_full + 8 * w, p_phase[w]);
              p_phase[w] ^= 1;
              fence_after();
              if (!__all_sync(0xffffffffu, waits.ok)) break;
              product_pv(w, j > 0);
              if (j + 1 == n[w]) mma_commit(bar.o_full + 8 * w, leader);
            }
            if (w == 1) mma_commit(bar.empty + 8 * vr.at, leader);
            if (j + 1 < n[w]) {
              waits.on(bar.full + 8 * kr.at, kr.phase);
              fence_after();
              if (!__all_sync(0xffffffffu, waits.ok)) break;
              product_qk(w);
              if (j + 2 == n[w]) mma_commit(bar.q_empty + 8 * w, leader);
            }
          }
          if (!__all_sync(0xffffffffu, waits.ok)) break;
          if (more) {
            mma_commit(bar.empty + 8 * kr.at, leader);
            kr.next(), kr.next();
          }
          vr.next(), vr.next();
        }
      }
      if (!__all_sync(0xffffffffu, waits.ok && ok) && lane == 0) fail();
      mma_commit(bar.drained, leader);  // every product issued is complete before TMEM is freed
      mbar_wait(bar.drained, 0);
      __syncwarp();
    } else {
      // --------------------------- a look through V -----------------------------
      const int me = threadIdx.x - kCheck * 32;
      Ring<kItems> at_item;
      uint32_t v_phase = 0, free_phase = 1;
      int first_stage = 0;  // the item's
      bool ok = true;
      PromptItem it;
      int h;
#pragma unroll 1
      while (next(at_item, ok, it, h)) {
        const Work x(it, h, tt);
        // the rows of the item before have been written (of the first: at once)
        ok = wait(bar.odd_free, free_phase);
        if (!ok) break;
        free_phase ^= 1;
        asm volatile("bar.sync 4, 64;" ::: "memory");
        const bool reset = *any_odd != 0;
        asm volatile("bar.sync 4, 64;" ::: "memory");
        if (reset) {
          for (int i = me; i < 3 * D; i += 64) odd[i] = 0x7fffffff;
          if (me == 0) *any_odd = 0;
          asm volatile("bar.sync 4, 64;" ::: "memory");
        }
        for (int i = 0; i < kChecked; ++i) {
          if (i < x.checks()) {
            ok = wait(bar.values + 8 * i, v_phase >> i & 1);
            if (!ok) break;
            v_phase ^= 1u << i;
            const int j = x.check0 + i, stage = (first_stage + 2 * j + 1) % kStages;
            check_values<kTok, D>(sm + oKV + stage * kTile, odd, j * kTok, x.t0, x.len, me);
            __syncwarp();
            for (int c = lane; c < 3 * D; c += 32)
              if (odd[c] != 0x7fffffff) *any_odd = 1;
            fence_async();
          }
          __syncwarp();
          mbar_arrive_if(bar.checked + 8 * i, lane == 0);
        }
        if (!ok) break;
        first_stage = (first_stage + 2 * x.nt) % kStages;
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
  static int sms[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return OSCAR_ERR_LAUNCH;
  if (!sms[dev]) {
    int n = 0;
    if (cudaFuncSetAttribute(attn_prompt_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return OSCAR_ERR_LAUNCH;
    sms[dev] = n;
  }
  const int tt = N / a.G;
  CUtensorMap mq, mk, mv;
  if (!encode_heads_bf16(&mq, a.q, uint64_t(a.n), a.Hq, D, uint32_t(a.G), uint32_t(tt)) ||
      !encode_rows_bf16(&mk, a.k, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok) ||
      !encode_rows_bf16(&mv, a.v, uint64_t(a.n), uint32_t(a.Hkv) * D, 64, kTok))
    return OSCAR_ERR_LAUNCH;
  const int64_t items = prompt_items(a, 1, 2 * tt) * a.Hkv;
  if (items >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  attn_prompt_tc_kernel<<<unsigned(std::min<int64_t>(items, sms[dev])), kThreads, kBytes, stream>>>(mq, mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? OSCAR_OK : OSCAR_ERR_LAUNCH;
}

}  // namespace oscar
