// C ABI: argument validation, cache layout arithmetic and kernel dispatch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <utility>

#include "internal.h"

namespace {

using oscar::Geom;

int validate(const oscar_kv_config* c) {
  if (!c) return OSCAR_ERR_INVALID;
  if (c->num_layers <= 0 || c->batch <= 0 || c->num_q_heads <= 0 || c->num_kv_heads <= 0 ||
      c->capacity <= 0 || c->sink < 0 || c->recent < 0)
    return OSCAR_ERR_INVALID;
  if (c->num_q_heads % c->num_kv_heads != 0) return OSCAR_ERR_INVALID;
  if (!(c->k_clip > 0.f && c->k_clip <= 1.f) || !(c->v_clip > 0.f && c->v_clip <= 1.f)) return OSCAR_ERR_INVALID;
  if (c->flags & ~uint32_t(OSCAR_FLAG_ABSORB_V | OSCAR_FLAG_IN_FP32 | OSCAR_FLAG_OUT_FP32 | OSCAR_FLAG_HADAMARD |
                           OSCAR_FLAG_V_BF16 | OSCAR_FLAG_LLOYD_MAX))
    return OSCAR_ERR_INVALID;
  if (c->group_size != OSCAR_KV_GROUP) return OSCAR_ERR_UNSUPPORTED;
  if (c->head_dim != 128 && c->head_dim != 256 && c->head_dim != 512) return OSCAR_ERR_UNSUPPORTED;
  if (c->num_q_heads / c->num_kv_heads > 8) return OSCAR_ERR_UNSUPPORTED;
  return OSCAR_OK;
}

Geom make_geom(const oscar_kv_config* c) {
  Geom g;
  g.B = c->batch;
  g.Hq = c->num_q_heads;
  g.Hkv = c->num_kv_heads;
  g.D = c->head_dim;
  g.G = g.Hq / g.Hkv;
  g.Dg = g.D / OSCAR_KV_GROUP;
  g.S = c->sink;
  g.W = c->recent;
  g.cap = c->capacity;
  const int64_t n = c->capacity > c->sink ? c->capacity - c->sink : 0;
  g.ncap = (n + oscar::kNcapRound - 1) / oscar::kNcapRound * oscar::kNcapRound;
  const uint64_t bh = uint64_t(g.B) * g.Hkv;
  g.sink_bytes = oscar::align256(bh * g.S * g.D * 2);
  g.ring_bytes = oscar::align256(bh * g.W * g.D * 2);
  g.codes_bytes = oscar::align256(bh * uint64_t(g.ncap) * (g.D / 4));
  g.sz_bytes = oscar::align256(bh * uint64_t(g.ncap) * g.Dg * 4);
  g.role_bytes = g.sink_bytes + g.ring_bytes + g.codes_bytes + g.sz_bytes;
  g.vb = (c->flags & OSCAR_FLAG_V_BF16) ? 1 : 0;
  g.lm = (c->flags & OSCAR_FLAG_LLOYD_MAX) ? 1 : 0;
  g.v_role_bytes = g.vb ? oscar::align256(bh * uint64_t(g.cap) * g.D * 2) : g.role_bytes;
  g.layer_bytes = g.role_bytes + g.v_role_bytes;
  return g;
}

}  // namespace

namespace oscar {
Geom geom_of(const oscar_kv_config* c) { return make_geom(c); }
}  // namespace oscar

namespace {
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

namespace {

// Validates kv_append's arguments and fills *a; launches nothing.
int prep_append(const oscar_kv_config* cfg, void* cache, int32_t layer, const void* k_new, const void* v_new,
                const int32_t* start_pos, int32_t n_new, const float* R_K, const float* R_V, float* debug_rot_out,
                int32_t* dev_status, oscar::AppendArgs* a, bool no_rows = false) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  // with the in-quant Hadamard the rotation matrices are not read (NULL allowed)
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = R_V = nullptr;
  if (!cache || (!no_rows && (!k_new || !v_new)) || !start_pos || (!had && (!R_K || !R_V))) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || n_new < 0) return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(R_K, 16) || !aligned(R_V, 16) || !aligned(k_new, 16) ||
      !aligned(v_new, 16) || (debug_rot_out && !aligned(debug_rot_out, 16)))
    return OSCAR_ERR_INVALID;
  if (n_new > cfg->capacity) return OSCAR_ERR_CAPACITY;
  a->g = make_geom(cfg);
  a->layer_base = static_cast<uint8_t*>(cache) + uint64_t(layer) * a->g.layer_bytes;
  a->k_new = k_new;
  a->v_new = v_new;
  a->start_pos = start_pos;
  a->R_K = R_K;
  a->R_V = R_V;
  a->debug_rot = debug_rot_out;
  a->status = dev_status;
  a->n_new = n_new;
  a->rows = int64_t(cfg->batch) * n_new * cfg->num_kv_heads;
  a->k_clip = cfg->k_clip;
  a->v_clip = cfg->v_clip;
  a->in_fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 1 : 0;
  a->hadamard = had ? 1 : 0;
  a->cu = nullptr;
  a->n_rows = 0;
  return OSCAR_OK;
}

// Validates attn_decode's arguments and fills *a; launches nothing.
int prep_decode(const oscar_kv_config* cfg, const void* cache, int32_t layer, const void* q,
                const int32_t* seq_lens, int32_t seq_len_hint, const float* R_K, const float* R_V, float sm_scale,
                int32_t num_splits, void* out, float* lse, void* workspace, uint64_t workspace_bytes,
                int32_t* dev_status, oscar::DecodeArgs* ap) {
  oscar::DecodeArgs& a = *ap;
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = R_V = nullptr;
  if (!cache || !q || !seq_lens || (!had && (!R_K || !R_V)) || !out || !workspace) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || num_splits < 0 || num_splits > OSCAR_KV_MAX_SPLITS ||
      seq_len_hint < 0)
    return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(workspace, 256) || !aligned(R_K, 16) || !aligned(R_V, 16) ||
      !aligned(q, 16) || !aligned(out, 16))
    return OSCAR_ERR_INVALID;
  if (seq_len_hint > cfg->capacity) return OSCAR_ERR_CAPACITY;
  const Geom g = make_geom(cfg);
  // the decode's TMA row coordinates are 32-bit: rows of each BF16 map must fit
  const uint64_t bhk = uint64_t(g.B) * g.Hkv;
  const uint64_t map_rows = bhk * uint64_t(g.vb ? (g.cap > g.S ? g.cap : g.S) : g.S);
  if (map_rows >= (uint64_t(1) << 31) || bhk * uint64_t(g.W) >= (uint64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  const int hint = seq_len_hint > 0 ? seq_len_hint : cfg->capacity;
  // partial slots per (sequence, query head): as many as the workspace holds,
  // up to OSCAR_KV_MAX_SPLITS; an explicit split count must fit in full
  if (num_splits > 0 && oscar::decode_workspace_bytes(g, num_splits) > workspace_bytes) return OSCAR_ERR_WORKSPACE;
  int ns = OSCAR_KV_MAX_SPLITS;
  while (ns > 1 && oscar::decode_workspace_bytes(g, ns) > workspace_bytes) --ns;
  if (oscar::decode_workspace_bytes(g, ns) > workspace_bytes) return OSCAR_ERR_WORKSPACE;
  const int ctas = oscar::decode_grid(g, hint, num_splits);
  if (ctas < 1) return OSCAR_ERR_LAUNCH;

  a.g = g;
  a.layer_base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * g.layer_bytes;
  a.q = q;
  a.seq_lens = seq_lens;
  a.R_K = R_K;
  a.R_V = R_V;
  a.out = out;
  a.lse = lse;
  a.status = dev_status;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const uint64_t bq = uint64_t(g.B) * g.Hq;
  const uint64_t units = uint64_t(g.B) * g.Hkv, nqt = g.G > 4 ? 2 : 1;
  a.qfrag = reinterpret_cast<uint32_t*>(ws);
  ws += oscar::align256(units * g.Dg * nqt * 2048);
  a.qbfrag = reinterpret_cast<uint32_t*>(ws);
  ws += oscar::align256(units * g.Dg * nqt * 4096);
  a.qsum = reinterpret_cast<float*>(ws);
  ws += oscar::align256(bq * g.Dg * 4);
  a.qF = reinterpret_cast<float*>(ws);
  ws += oscar::align256(bq * g.Dg * 4);
  a.ws_acc = reinterpret_cast<float*>(ws);
  ws += oscar::align256(bq * uint64_t(ns) * g.D * 4);
  a.ws_ml = reinterpret_cast<float*>(ws);
  ws += oscar::align256(bq * uint64_t(ns) * 2 * 4);
  a.ticket = reinterpret_cast<int32_t*>(ws);
  a.ns = ns;
  a.ctas = ctas;
  const float scale = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(float(g.D));
  a.qscale = scale * 1.4426950408889634f;
  a.in_fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 1 : 0;
  a.out_fp32 = (cfg->flags & OSCAR_FLAG_OUT_FP32) ? 1 : 0;
  a.absorb_v = (cfg->flags & OSCAR_FLAG_ABSORB_V) ? 1 : 0;
  a.hadamard = had ? 1 : 0;
  a.new_pos = nullptr;
  a.new_n = 0;
  a.fused = 0;
  a.wait_ns = oscar::wait_limit_ns();
  a.wait_poison = oscar::g_test_wait_poison;
  return OSCAR_OK;
}

// Workspace of the row attention: rotated queries and ns partial results per query row.
uint64_t rows_workspace(const Geom& g, int64_t rows, int ns) {
  return oscar::align256(uint64_t(rows) * g.D * 4) + oscar::align256(uint64_t(rows) * ns * g.D * 4) +
         oscar::align256(uint64_t(rows) * ns * 8);
}

// Takes `bytes` from the workspace at *ws.
template <typename T>
T* take(uint8_t** ws, uint64_t bytes) {
  T* p = reinterpret_cast<T*>(*ws);
  *ws += oscar::align256(bytes);
  return p;
}

float log2_scale(const Geom& g, float sm_scale) {
  return (sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt(float(g.D))) * 1.4426950408889634f;
}

// attn_extend's and attn_decode_prefix's common part: query rotation, row
// attention and the merge, laid out in the workspace at *ws.
struct RowsPlan {
  oscar::QrotRowsArgs q;
  oscar::RowsArgs at;
  oscar::FinishArgs fin;
};
void plan_rows(const oscar_kv_config* cfg, const Geom& g, const void* cache, int32_t layer, const void* q, int n,
               const int32_t* seq_lens, const int32_t* q_lens, const float* R_K, const float* R_V, float sm_scale, int ns,
               void* out, float* lse, int32_t* dev_status, uint8_t** ws, RowsPlan* p) {
  std::memset(p, 0, sizeof(*p));
  const int64_t rows = int64_t(g.B) * n * g.Hq;
  const int hadamard = (cfg->flags & OSCAR_FLAG_HADAMARD) ? 1 : 0;
  p->q.q = q;
  p->q.qrot = take<float>(ws, uint64_t(rows) * g.D * 4);
  p->q.R_K = R_K;
  p->q.status = dev_status;
  p->q.q_lens = q_lens;
  p->q.rows = rows;
  p->q.n = n;
  p->q.Hq = g.Hq;
  p->q.D = g.D;
  p->q.in_fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 1 : 0;
  p->q.hadamard = hadamard;
  p->q.qscale = log2_scale(g, sm_scale);
  p->at.g = g;
  p->at.layer_base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * g.layer_bytes;
  p->at.seq_lens = seq_lens;
  p->at.q_lens = q_lens;
  p->at.qrot = p->q.qrot;
  p->at.acc = take<float>(ws, uint64_t(rows) * ns * g.D * 4);
  p->at.ml = take<float>(ws, uint64_t(rows) * ns * 8);
  p->at.status = dev_status;
  p->at.n = n;
  p->at.ns = ns;
  p->at.wait_turns = oscar::wait_turns();
  p->at.wait_poison = oscar::g_test_wait_poison;
  p->fin.acc = p->at.acc;
  p->fin.ml = p->at.ml;
  p->fin.q_lens = q_lens;
  p->fin.R_V = R_V;
  p->fin.out = out;
  p->fin.lse = lse;
  p->fin.status = dev_status;
  p->fin.rows = rows;
  p->fin.n = n;
  p->fin.Hq = g.Hq;
  p->fin.D = g.D;
  p->fin.ns = ns;
  p->fin.out_fp32 = (cfg->flags & OSCAR_FLAG_OUT_FP32) ? 1 : 0;
  p->fin.absorb_v = (cfg->flags & OSCAR_FLAG_ABSORB_V) ? 1 : 0;
  p->fin.hadamard = hadamard;
}

// The row attention in float32 when the output is float32, else on the tensor cores.
int splits_of(const oscar_kv_config* cfg, const Geom& g, int64_t rows, int hint) {
  return (cfg->flags & OSCAR_FLAG_OUT_FP32) ? oscar::rows_splits(g, rows, hint) : oscar::rows_splits_tc(g, rows, hint);
}
int launch_rows(const oscar_kv_config* cfg, const oscar::RowsArgs& a, cudaStream_t st) {
  return (cfg->flags & OSCAR_FLAG_OUT_FP32) ? oscar::launch_attn_rows(a, st) : oscar::launch_attn_rows_tc(a, st);
}

// The row kernels count rows and workspace slots in ranges of these limits, and
// positions in 32 bits up to a few tiles behind the last one.
constexpr int kMostPositions = 0x7fffffff - 1024;
constexpr int kMostEvict = 0x7fffffff - 16384;  // kv_evict counts on by up to a block's loads
constexpr int kMostUnits = 65535;  // (sequence, KV head) pairs of attn_mass and kv_evict: a grid's second dimension
bool rows_supported(const Geom& g, int64_t n) {
  return n * g.G < (int64_t(1) << 30) && g.B * n * g.Hq < (int64_t(1) << 31) && g.cap <= kMostPositions;
}

// The largest split count up to `want` whose workspace fits, 0 if none does;
// an explicit count has to fit in full.
int fit_splits(const Geom& g, int64_t rows, int want, bool explicit_count, uint64_t bytes) {
  int ns = want;
  if (!explicit_count)
    while (ns > 1 && rows_workspace(g, rows, ns) > bytes) --ns;
  return rows_workspace(g, rows, ns) > bytes ? 0 : ns;
}

// Caches that kv_evict reads and writes: the same but for layers, capacity and clips.
int validate_evict(const oscar_kv_config* cfg, const oscar_kv_config* ocfg, int32_t keep) {
  int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  v = validate(ocfg);
  if (v != OSCAR_OK) return v;
  if (ocfg->batch != cfg->batch || ocfg->num_q_heads != cfg->num_q_heads || ocfg->num_kv_heads != cfg->num_kv_heads ||
      ocfg->head_dim != cfg->head_dim || ocfg->sink != cfg->sink || ocfg->recent != cfg->recent || ocfg->flags != cfg->flags ||
      keep < 0)
    return OSCAR_ERR_INVALID;
  const int64_t most = std::min<int64_t>(cfg->capacity, int64_t(cfg->sink) + cfg->recent + keep);
  if (ocfg->capacity < most) return OSCAR_ERR_CAPACITY;
  const int64_t units = int64_t(cfg->batch) * cfg->num_kv_heads;
  return units <= kMostUnits && cfg->capacity <= kMostEvict && ocfg->capacity <= kMostEvict ? OSCAR_OK : OSCAR_ERR_UNSUPPORTED;
}
int evict_list(const Geom& g, int32_t keep) { return std::min(keep, std::max(0, g.cap - g.S)); }
bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// The prefix cache has the shape of the sequences' own, with one sequence.
int validate_prefix(const oscar_kv_config* cfg, const oscar_kv_config* pcfg) {
  int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  v = validate(pcfg);
  if (v != OSCAR_OK) return v;
  if (pcfg->batch != 1 || pcfg->num_q_heads != cfg->num_q_heads || pcfg->num_kv_heads != cfg->num_kv_heads ||
      pcfg->head_dim != cfg->head_dim || pcfg->flags != cfg->flags)
    return OSCAR_ERR_INVALID;
  return rows_supported(make_geom(pcfg), cfg->batch) && cfg->capacity <= kMostPositions ? OSCAR_OK : OSCAR_ERR_UNSUPPORTED;
}

// Longest own cache that attn_decode_prefix gives to the row attention, which
// runs beside the prefix's; longer ones go to attn_decode's kernels, which take
// about 20 us more to begin with and less per position.  Row attention against
// those on a prefix of 2048 positions, us a call: 8 sequences x 8 KV heads with
// 64 / 512 / 1024 positions 37 / 47 / 49 against 52 / 55 / 55, 32 x 8 with 64 /
// 256 / 512 / 1024 57 / 71 / 82 / 94 against 65 / 68 / 72 / 75, 8 x 8 at D = 512
// with 64 / 256 / 512 / 1024 69 / 92 / 118 / 120 against 117 / 127 / 129 / 133.
constexpr int kOwnRows = 1024, kOwnTiles = 512;  // positions; tiles of 128 in all
int own_rows_limit(const Geom& g) {
  return int(std::min<int64_t>(kOwnRows, kOwnTiles / (int64_t(g.B) * g.Hkv) * 128));
}

// Workspace of attn_decode_prefix apart from the prefix's row attention: the own
// caches' partial results and a word that says that the queries are there, or
// attn_decode's outputs, lse and status word.
uint64_t own_rows_workspace(const Geom& g, int ns) {
  const uint64_t bq = uint64_t(g.B) * g.Hq;
  return oscar::align256(bq * ns * g.D * 4) + oscar::align256(bq * ns * 8) + 256;
}
uint64_t own_workspace(const Geom& g) {
  const uint64_t bq = uint64_t(g.B) * g.Hq;
  return oscar::align256(bq * g.D * 4) + oscar::align256(bq * 4) + 256;
}

}  // namespace

extern "C" {

int kv_layout_query(const oscar_kv_config* cfg, oscar_kv_layout* out) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  if (!out) return OSCAR_ERR_INVALID;
  const Geom g = make_geom(cfg);
  std::memset(out, 0, sizeof(*out));
  out->ncap = uint64_t(g.ncap);
  out->sink_bytes = g.sink_bytes;
  out->ring_bytes = g.ring_bytes;
  out->codes_bytes = g.codes_bytes;
  out->sz_bytes = g.sz_bytes;
  out->role_bytes = g.role_bytes;
  out->layer_bytes = g.layer_bytes;
  out->v_role_bytes = g.v_role_bytes;
  out->total_bytes = g.layer_bytes * uint64_t(cfg->num_layers);
  out->decode_workspace_bytes = oscar::decode_workspace_bytes(g, OSCAR_KV_MAX_SPLITS);
  out->max_splits = OSCAR_KV_MAX_SPLITS;
  return OSCAR_OK;
}

int kv_append(const oscar_kv_config* cfg, void* cache, int32_t layer, const void* k_new, const void* v_new,
              const int32_t* start_pos, int32_t n_new, const float* R_K, const float* R_V,
              float* debug_rot_out, int32_t* dev_status, void* stream) {
  oscar::AppendArgs a;
  const int v = prep_append(cfg, cache, layer, k_new, v_new, start_pos, n_new, R_K, R_V, debug_rot_out, dev_status, &a);
  if (v != OSCAR_OK) return v;
  return oscar::launch_append(a, static_cast<cudaStream_t>(stream));
}

int attn_decode(const oscar_kv_config* cfg, const void* cache, int32_t layer, const void* q,
                const int32_t* seq_lens, int32_t seq_len_hint, const float* R_K, const float* R_V,
                float sm_scale, int32_t num_splits, void* out, float* lse, void* workspace,
                uint64_t workspace_bytes, int32_t* dev_status, void* stream) {
  oscar::DecodeArgs a;
  const int v = prep_decode(cfg, cache, layer, q, seq_lens, seq_len_hint, R_K, R_V, sm_scale, num_splits, out, lse,
                            workspace, workspace_bytes, dev_status, &a);
  if (v != OSCAR_OK) return v;
  return oscar::launch_decode(a, static_cast<cudaStream_t>(stream));
}

int decode_step(const oscar_kv_config* cfg, void* cache, int32_t layer, const void* k_new, const void* v_new,
                const int32_t* start_pos, int32_t n_new, const void* q, const int32_t* seq_lens,
                int32_t seq_len_hint, const float* R_K, const float* R_V, float sm_scale, int32_t num_splits,
                void* out, float* lse, void* workspace, uint64_t workspace_bytes, int32_t* dev_status,
                void* stream) {
  oscar::AppendArgs aa;
  oscar::DecodeArgs ad;
  int v = prep_append(cfg, cache, layer, k_new, v_new, start_pos, n_new, R_K, R_V, nullptr, dev_status, &aa);
  if (v != OSCAR_OK) return v;
  v = prep_decode(cfg, cache, layer, q, seq_lens, seq_len_hint, R_K, R_V, sm_scale, num_splits, out, lse, workspace,
                  workspace_bytes, dev_status, &ad);
  if (v != OSCAR_OK) return v;
  // the decode kernels know what the append writes: they start streaming the
  // rest of the cache while it runs
  ad.new_pos = start_pos;
  ad.new_n = n_new;
  ad.fused = 1;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  v = oscar::launch_append(aa, st);
  if (v != OSCAR_OK) return v;
  return oscar::launch_decode(ad, st);
}

int kv_read(const oscar_kv_config* cfg, const void* cache, int32_t layer, const int32_t* start_pos,
            const int32_t* seq_lens, int32_t n, const float* R_K, const float* R_V, void* k_out, void* v_out,
            int32_t* dev_status, void* stream) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = R_V = nullptr;
  // no positions: the output of an empty tensor may be NULL
  if (!cache || !start_pos || !seq_lens || (!had && (!R_K || !R_V)) || (!k_out && !v_out && n != 0)) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || n < 0) return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(R_K, 16) || !aligned(R_V, 16) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return OSCAR_ERR_INVALID;
  oscar::ReadArgs a;
  a.g = make_geom(cfg);
  a.layer_base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * a.g.layer_bytes;
  a.start_pos = start_pos;
  a.seq_lens = seq_lens;
  a.R_K = R_K;
  a.R_V = R_V;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = dev_status;
  a.n = n;
  a.out_fp32 = (cfg->flags & OSCAR_FLAG_OUT_FP32) ? 1 : 0;
  a.absorb_v = (cfg->flags & OSCAR_FLAG_ABSORB_V) ? 1 : 0;
  a.hadamard = had ? 1 : 0;
  return oscar::launch_read(a, static_cast<cudaStream_t>(stream));
}

int attn_extend_workspace_query(const oscar_kv_config* cfg, int32_t n_new, uint64_t* bytes) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  if (!bytes || n_new < 0) return OSCAR_ERR_INVALID;
  if (n_new > cfg->capacity) return OSCAR_ERR_CAPACITY;
  const Geom g = make_geom(cfg);
  if (!rows_supported(g, n_new)) return OSCAR_ERR_UNSUPPORTED;
  *bytes = n_new == 0 ? 0 : rows_workspace(g, int64_t(g.B) * n_new * g.Hq, splits_of(cfg, g, int64_t(n_new) * g.G, g.cap));
  return OSCAR_OK;
}

int attn_extend(const oscar_kv_config* cfg, const void* cache, int32_t layer, const void* q, int32_t n_new,
                const int32_t* q_lens, const int32_t* seq_lens, int32_t seq_len_hint, const float* R_K,
                const float* R_V, float sm_scale, int32_t num_splits, void* out, float* lse, void* workspace,
                uint64_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = R_V = nullptr;
  // no tokens: their empty tensors may be NULL, as may the workspace, whose size is then 0
  if (!cache || !seq_lens || (!had && (!R_K || !R_V)) || (n_new != 0 && (!q || !out || !workspace))) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || n_new < 0 || num_splits < 0 || num_splits > OSCAR_KV_MAX_SPLITS ||
      seq_len_hint < 0)
    return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(workspace, 256) || !aligned(R_K, 16) || !aligned(R_V, 16) ||
      !aligned(q, 16) || !aligned(out, 16))
    return OSCAR_ERR_INVALID;
  if (n_new > cfg->capacity || seq_len_hint > cfg->capacity) return OSCAR_ERR_CAPACITY;
  const Geom g = make_geom(cfg);
  if (!rows_supported(g, n_new)) return OSCAR_ERR_UNSUPPORTED;
  if (n_new == 0) return OSCAR_OK;
  const int hint = seq_len_hint > 0 ? seq_len_hint : cfg->capacity;
  const int want = num_splits > 0 ? num_splits : splits_of(cfg, g, int64_t(n_new) * g.G, hint);
  const int ns = fit_splits(g, int64_t(g.B) * n_new * g.Hq, want, num_splits > 0, workspace_bytes);
  if (ns == 0) return OSCAR_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RowsPlan p{};
  plan_rows(cfg, g, cache, layer, q, n_new, seq_lens, q_lens, R_K, R_V, sm_scale, ns, out, lse, dev_status, &ws, &p);
  p.at.causal = 1;
  p.at.early = p.fin.dependent = 1;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int rc = oscar::launch_qrot_rows(p.q, st);
  if (rc == OSCAR_OK) rc = launch_rows(cfg, p.at, st);
  if (rc == OSCAR_OK) rc = oscar::launch_finish_rows(p.fin, st);
  return rc;
}

int attn_decode_prefix_workspace_query(const oscar_kv_config* cfg, const oscar_kv_config* prefix_cfg,
                                       uint64_t* bytes) {
  const int v = validate_prefix(cfg, prefix_cfg);
  if (v != OSCAR_OK) return v;
  if (!bytes) return OSCAR_ERR_INVALID;
  const Geom g = make_geom(cfg), pg = make_geom(prefix_cfg);
  *bytes = rows_workspace(pg, int64_t(g.B) * g.Hq, OSCAR_KV_MAX_SPLITS) +
           std::max(own_rows_workspace(g, splits_of(cfg, g, g.G, std::min(g.cap, kOwnRows))),
                    g.cap > own_rows_limit(g) ? own_workspace(g) + oscar::decode_workspace_bytes(g, OSCAR_KV_MAX_SPLITS) : 0);
  return OSCAR_OK;
}

int attn_decode_prefix(const oscar_kv_config* cfg, const void* cache, const oscar_kv_config* prefix_cfg,
                       const void* prefix_cache, int32_t layer, const void* q, const int32_t* seq_lens,
                       int32_t seq_len_hint, const int32_t* prefix_len, int32_t prefix_len_hint, const float* R_K,
                       const float* R_V, float sm_scale, int32_t num_splits, void* out, float* lse, void* workspace,
                       uint64_t workspace_bytes, int32_t* dev_status, void* stream) {
  int v = validate_prefix(cfg, prefix_cfg);
  if (v != OSCAR_OK) return v;
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = R_V = nullptr;
  if (!cache || !q || !seq_lens || !prefix_cache || !prefix_len || (!had && (!R_K || !R_V)) || !workspace || !out)
    return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || layer >= prefix_cfg->num_layers || num_splits < 0 ||
      num_splits > OSCAR_KV_MAX_SPLITS || prefix_len_hint < 0 || seq_len_hint < 0)
    return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(prefix_cache, 256) || !aligned(workspace, 256) || !aligned(R_K, 16) ||
      !aligned(R_V, 16) || !aligned(q, 16) || !aligned(out, 16))
    return OSCAR_ERR_INVALID;
  if (prefix_len_hint > prefix_cfg->capacity || seq_len_hint > cfg->capacity) return OSCAR_ERR_CAPACITY;
  const Geom g = make_geom(cfg), pg = make_geom(prefix_cfg);
  const int64_t rows = int64_t(g.B) * g.Hq;
  const int hint = prefix_len_hint > 0 ? prefix_len_hint : prefix_cfg->capacity;
  const int own_hint = seq_len_hint > 0 ? seq_len_hint : cfg->capacity;
  const int want = num_splits > 0 ? num_splits : splits_of(cfg, pg, int64_t(g.B) * g.G, hint);
  // the own caches' part has to fit with one split at least; what is left goes to the prefix
  const bool own_by_rows = own_hint <= own_rows_limit(g);
  // not more than the workspace query counts with, whatever the hint
  const int want2 = own_by_rows ? std::min(splits_of(cfg, g, g.G, own_hint), splits_of(cfg, g, g.G, std::min(g.cap, kOwnRows))) : 0;
  const uint64_t own = own_by_rows ? own_rows_workspace(g, want2) : own_workspace(g) + oscar::decode_workspace_bytes(g, 1);
  const int ns =
      workspace_bytes < own ? 0 : fit_splits(pg, rows, want, num_splits > 0, workspace_bytes - own);
  if (ns == 0) return OSCAR_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RowsPlan p{};
  // one query token per sequence: the batch is the block of query rows of the one prefix
  plan_rows(cfg, pg, prefix_cache, layer, q, g.B, prefix_len, nullptr, R_K, R_V, sm_scale, ns, out, lse, dev_status, &ws,
            &p);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (own_by_rows) {
    p.at.ready = p.q.zero_word = take<int32_t>(&ws, 256);
    oscar::RowsArgs own_at = p.at;
    own_at.g = g;
    own_at.layer_base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * g.layer_bytes;
    own_at.seq_lens = seq_lens;
    own_at.n = 1;
    p.at.early = own_at.early = own_at.beside = p.fin.dependent = 1;
    own_at.ns = want2;
    own_at.acc = take<float>(&ws, uint64_t(rows) * want2 * g.D * 4);
    own_at.ml = take<float>(&ws, uint64_t(rows) * want2 * 8);
    p.fin.acc2 = own_at.acc;
    p.fin.ml2 = own_at.ml;
    p.fin.ns2 = want2;
    int rc = oscar::launch_qrot_rows(p.q, st);
    if (rc == OSCAR_OK) rc = launch_rows(cfg, p.at, st);
    if (rc == OSCAR_OK) rc = launch_rows(cfg, own_at, st);
    if (rc == OSCAR_OK) rc = oscar::launch_finish_rows(p.fin, st);
    return rc;
  }
  float* own_o = take<float>(&ws, uint64_t(rows) * g.D * 4);
  float* own_lse = take<float>(&ws, uint64_t(rows) * 4);
  int32_t* own_status = take<int32_t>(&ws, 256);
  p.q.zero_word = own_status;
  p.fin.own_o = own_o;
  p.fin.own_lse = own_lse;
  p.fin.own_status = own_status;
  // long own caches through attn_decode's kernels, in the rotated basis and float32
  oscar_kv_config dcfg = *cfg;
  dcfg.flags |= OSCAR_FLAG_ABSORB_V | OSCAR_FLAG_OUT_FP32;
  oscar::DecodeArgs d;
  v = prep_decode(&dcfg, cache, layer, q, seq_lens, seq_len_hint, R_K, R_V, sm_scale, 0, own_o, own_lse, ws,
                  workspace_bytes - uint64_t(ws - static_cast<uint8_t*>(workspace)), own_status, &d);
  if (v != OSCAR_OK) return v;
  int rc = oscar::launch_qrot_rows(p.q, st);
  if (rc == OSCAR_OK) rc = launch_rows(cfg, p.at, st);
  if (rc == OSCAR_OK) rc = oscar::launch_decode(d, st);
  if (rc == OSCAR_OK) rc = oscar::launch_finish_rows(p.fin, st);
  return rc;
}

int qk_norm_rope(const oscar_kv_config* cfg, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                 int32_t n_rows, const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
                 const float* inv_freq, int32_t rot_dim, int32_t interleaved, void* q_out, void* k_out, void* stream) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  const int D = cfg->head_dim;
  if (n_rows < 0 || !(eps >= 0.f) || std::isinf(eps) || rot_dim < 0 || rot_dim > D || rot_dim % 16 != 0 || !q_weight || !k_weight ||
      (rot_dim > 0 && !inv_freq))
    return OSCAR_ERR_INVALID;
  if (n_rows != 0 && (!q || !k || !q_out || !k_out || (rot_dim > 0 && !positions))) return OSCAR_ERR_INVALID;
  const bool fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) != 0;
  const int64_t piece = fp32 ? 4 : 8;  // elements of 16 bytes
  if (q_stride < int64_t(cfg->num_q_heads) * D || k_stride < int64_t(cfg->num_kv_heads) * D || q_stride % piece != 0 ||
      k_stride % piece != 0)
    return OSCAR_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16))
    return OSCAR_ERR_INVALID;
  if (n_rows == 0) return OSCAR_OK;
  // a row may be written where it was read, not where another one still is
  const uint64_t size = fp32 ? 4 : 2, q_row = uint64_t(cfg->num_q_heads) * D, k_row = uint64_t(cfg->num_kv_heads) * D;
  const uint64_t q_span = (uint64_t(n_rows - 1) * q_stride + q_row) * size, k_span = (uint64_t(n_rows - 1) * k_stride + k_row) * size;
  const uint64_t q_bytes = n_rows * q_row * size, k_bytes = n_rows * k_row * size;
  const bool q_place = q_out == q && q_span == q_bytes, k_place = k_out == k && k_span == k_bytes;
  if ((!q_place && overlap(q_out, q_bytes, q, q_span)) || (!k_place && overlap(k_out, k_bytes, k, k_span)) ||
      overlap(q_out, q_bytes, k, k_span) || overlap(k_out, k_bytes, q, q_span) || overlap(q_out, q_bytes, k_out, k_bytes))
    return OSCAR_ERR_INVALID;
  oscar::NormRopeArgs a{};
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_out = k_out;
  a.eps = eps;
  a.n = n_rows;
  a.Hq = cfg->num_q_heads;
  a.Hkv = cfg->num_kv_heads;
  a.D = D;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.fp32 = fp32 ? 1 : 0;
  return oscar::launch_norm_rope(a, static_cast<cudaStream_t>(stream));
}

int attn_prompt(const oscar_kv_config* cfg, const void* q, const void* k, const void* v, int32_t n_rows,
                const int32_t* cu_seqlens, float sm_scale, void* out, float* lse, int32_t* dev_status, void* stream) {
  const int rc = validate(cfg);
  if (rc != OSCAR_OK) return rc;
  if (n_rows < 0 || !cu_seqlens || (n_rows != 0 && (!q || !k || !v || !out))) return OSCAR_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16)) return OSCAR_ERR_INVALID;
  const Geom g = make_geom(cfg);
  if (int64_t(n_rows) * g.Hq >= (int64_t(1) << 31)) return OSCAR_ERR_UNSUPPORTED;
  if (n_rows == 0) return OSCAR_OK;
  const uint64_t q_values = uint64_t(n_rows) * g.Hq * g.D, kv_values = uint64_t(n_rows) * g.Hkv * g.D;
  const uint64_t size_in = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 4 : 2, size_out = (cfg->flags & OSCAR_FLAG_OUT_FP32) ? 4 : 2;
  for (const auto& [in, values] : {std::pair(q, q_values), std::pair(k, kv_values), std::pair(v, kv_values)})
    if (overlap(in, values * size_in, out, q_values * size_out)) return OSCAR_ERR_INVALID;
  oscar::PromptArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.cu = cu_seqlens;
  a.out = out;
  a.lse = lse;
  a.status = dev_status;
  a.n = n_rows;
  a.B = g.B;
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.G = g.G;
  a.D = g.D;
  a.in_fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 1 : 0;
  a.out_fp32 = (cfg->flags & OSCAR_FLAG_OUT_FP32) ? 1 : 0;
  a.qscale = log2_scale(g, sm_scale);
  a.wait_turns = oscar::wait_turns();
  a.wait_poison = oscar::g_test_wait_poison;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.in_fp32 || a.out_fp32) return oscar::launch_attn_prompt(a, st);
  return a.D == 128 ? oscar::launch_attn_prompt_tc(a, st) : oscar::launch_attn_prompt_wide(a, st);
}

int kv_append_packed(const oscar_kv_config* cfg, void* cache, int32_t layer, const void* k_new, const void* v_new,
                     int32_t n_rows, const int32_t* cu_seqlens, const int32_t* start_pos, const float* R_K,
                     const float* R_V, int32_t* dev_status, void* stream) {
  if (!cu_seqlens || n_rows < 0) return OSCAR_ERR_INVALID;
  oscar::AppendArgs a;
  const int v = prep_append(cfg, cache, layer, k_new, v_new, start_pos, 0, R_K, R_V, nullptr, dev_status, &a, n_rows == 0);
  if (v != OSCAR_OK) return v;
  a.cu = cu_seqlens;
  a.n_rows = n_rows;
  a.rows = int64_t(n_rows) * cfg->num_kv_heads;
  return oscar::launch_append(a, static_cast<cudaStream_t>(stream));
}

int attn_mass_workspace_query(const oscar_kv_config* cfg, int32_t n_new, uint64_t* bytes) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  if (!bytes || n_new < 0) return OSCAR_ERR_INVALID;
  if (n_new > cfg->capacity) return OSCAR_ERR_CAPACITY;
  const Geom g = make_geom(cfg);
  if (!rows_supported(g, n_new) || int64_t(g.B) * g.Hkv > kMostUnits) return OSCAR_ERR_UNSUPPORTED;
  *bytes = oscar::align256(uint64_t(g.B) * n_new * g.Hq * g.D * 4) + oscar::align256(oscar::mass_frag_bytes(g, n_new));
  return OSCAR_OK;
}

int attn_mass(const oscar_kv_config* cfg, const void* cache, int32_t layer, const void* q, int32_t n_new,
              const int32_t* q_lens, const int32_t* seq_lens, int32_t seq_len_hint, const float* R_K, float sm_scale,
              const float* lse, const float* mass_in, float* mass_out, void* workspace, uint64_t workspace_bytes,
              int32_t* dev_status, void* stream) {
  uint64_t need = 0;
  const int v = attn_mass_workspace_query(cfg, n_new, &need);
  if (v != OSCAR_OK) return v;
  const bool had = (cfg->flags & OSCAR_FLAG_HADAMARD) != 0;
  if (had) R_K = nullptr;
  if (!cache || !seq_lens || !mass_out || (!had && !R_K) || (n_new != 0 && (!q || !lse || !workspace))) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || seq_len_hint < 0) return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(workspace, 256) || !aligned(R_K, 16) || !aligned(q, 16)) return OSCAR_ERR_INVALID;
  if (seq_len_hint > cfg->capacity) return OSCAR_ERR_CAPACITY;
  if (workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  const Geom g = make_geom(cfg);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  oscar::QrotRowsArgs r{};
  r.q = q;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  r.qrot = take<float>(&ws, uint64_t(g.B) * n_new * g.Hq * g.D * 4);
  r.R_K = R_K;
  r.status = dev_status;
  r.q_lens = q_lens;
  r.rows = int64_t(g.B) * n_new * g.Hq;
  r.n = n_new;
  r.Hq = g.Hq;
  r.D = g.D;
  r.in_fp32 = (cfg->flags & OSCAR_FLAG_IN_FP32) ? 1 : 0;
  r.hadamard = had ? 1 : 0;
  r.qscale = log2_scale(g, sm_scale);
  oscar::MassArgs a{};
  a.g = g;
  a.layer_base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * g.layer_bytes;
  a.seq_lens = seq_lens;
  a.q_lens = q_lens;
  a.qrot = r.qrot;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.status = dev_status;
  a.frags = ws;
  a.wait_turns = oscar::wait_turns();
  a.wait_poison = oscar::g_test_wait_poison;
  a.n = n_new;
  a.top = seq_len_hint > 0 ? seq_len_hint : g.cap;
  const int rc = n_new ? oscar::launch_qrot_rows(r, st) : OSCAR_OK;
  return rc == OSCAR_OK ? oscar::launch_attn_mass(a, st) : rc;
}

int kv_evict_workspace_query(const oscar_kv_config* cfg, int32_t keep, uint64_t* bytes) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  if (!bytes || keep < 0) return OSCAR_ERR_INVALID;
  const Geom g = make_geom(cfg);
  if (int64_t(g.B) * g.Hkv > kMostUnits || g.cap > kMostEvict) return OSCAR_ERR_UNSUPPORTED;
  *bytes = oscar::align256(uint64_t(g.B) * 4) + oscar::align256(uint64_t(g.B) * g.Hkv * evict_list(g, keep) * 4);
  return OSCAR_OK;
}

int kv_evict(const oscar_kv_config* cfg, const void* cache, int32_t layer, const float* mass, const int32_t* seq_lens,
             int32_t keep, const oscar_kv_config* out_cfg, void* out_cache, int32_t out_layer, float* out_mass,
             int32_t* kept, int32_t* new_lens, void* workspace, uint64_t workspace_bytes, int32_t* dev_status, void* stream) {
  const int v = validate_evict(cfg, out_cfg, keep);
  if (v != OSCAR_OK) return v;
  if (!cache || !out_cache || !mass || !seq_lens || !new_lens || !workspace) return OSCAR_ERR_INVALID;
  if (layer < 0 || layer >= cfg->num_layers || out_layer < 0 || out_layer >= out_cfg->num_layers) return OSCAR_ERR_INVALID;
  if (!aligned(cache, 256) || !aligned(out_cache, 256) || !aligned(workspace, 256)) return OSCAR_ERR_INVALID;
  oscar::EvictArgs a{};
  a.g = make_geom(cfg);
  a.og = make_geom(out_cfg);
  a.base = static_cast<const uint8_t*>(cache) + uint64_t(layer) * a.g.layer_bytes;
  a.out_base = static_cast<uint8_t*>(out_cache) + uint64_t(out_layer) * a.og.layer_bytes;
  const uint64_t units = uint64_t(a.g.B) * a.g.Hkv;
  if (overlap(a.base, a.g.layer_bytes, a.out_base, a.og.layer_bytes) ||
      (out_mass && overlap(mass, units * a.g.cap * 4, out_mass, units * a.og.cap * 4)))
    return OSCAR_ERR_INVALID;
  uint64_t need = 0;
  if (kv_evict_workspace_query(cfg, keep, &need) != OSCAR_OK || workspace_bytes < need) return OSCAR_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.mass = mass;
  a.seq_lens = seq_lens;
  a.new_lens = new_lens;
  a.out_mass = out_mass;
  a.kept = keep > 0 ? kept : nullptr;
  a.lens = take<int32_t>(&ws, uint64_t(a.g.B) * 4);
  a.list = reinterpret_cast<int32_t*>(ws);
  a.status = dev_status;
  a.keep = keep;
  a.list_cap = evict_list(a.g, keep);
  return oscar::launch_kv_evict(a, static_cast<cudaStream_t>(stream));
}

int oscar_kv_set_profile_events(void* split_start, void* split_stop) {
  oscar::g_prof_start = static_cast<cudaEvent_t>(split_start);
  oscar::g_prof_stop = static_cast<cudaEvent_t>(split_stop);
  return OSCAR_OK;
}

int oscar_kv_decode_kernels(const oscar_kv_config* cfg) {
  const int v = validate(cfg);
  if (v != OSCAR_OK) return v;
  return oscar::decode_kernel_count(make_geom(cfg), (cfg->flags & OSCAR_FLAG_ABSORB_V) != 0,
                                    (cfg->flags & OSCAR_FLAG_HADAMARD) != 0);
}

int oscar_kv_set_wait_test(uint64_t wait_ns, int32_t extra_bytes) {
  if (wait_ns > 10000000000ull || extra_bytes < 0 || extra_bytes > (1 << 20)) return OSCAR_ERR_INVALID;
  oscar::g_test_wait_ns = wait_ns;
  oscar::g_test_wait_poison = extra_bytes;
  return OSCAR_OK;
}
int oscar_calibrate_workspace_query(int32_t head_dim, uint64_t* bytes) {
  if (!bytes) return OSCAR_ERR_INVALID;
  if (head_dim != 128 && head_dim != 256 && head_dim != 512) return OSCAR_ERR_UNSUPPORTED;
  *bytes = oscar::calibrate_workspace_bytes(head_dim);
  return OSCAR_OK;
}

int oscar_calibrate_rk(const float* q, int64_t n_rows, int32_t head_dim, float* R_K_out, void* workspace,
                       uint64_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (head_dim != 128 && head_dim != 256 && head_dim != 512) return OSCAR_ERR_UNSUPPORTED;
  if (!q || !R_K_out || !workspace || n_rows < 1 || n_rows > OSCAR_KV_CALIB_MAX_ROWS) return OSCAR_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(R_K_out, 16) || !aligned(workspace, 256)) return OSCAR_ERR_INVALID;
  if (workspace_bytes < oscar::calibrate_workspace_bytes(head_dim)) return OSCAR_ERR_WORKSPACE;
  return oscar::launch_calibrate(q, n_rows, head_dim, R_K_out, workspace, dev_status,
                                 static_cast<cudaStream_t>(stream));
}

int oscar_calibrate_rv_workspace_query(int32_t head_dim, int64_t n_kv_rows, uint64_t* bytes) {
  if (!bytes || n_kv_rows < 1 || n_kv_rows > OSCAR_KV_CALIB_MAX_ROWS) return OSCAR_ERR_INVALID;
  if (head_dim != 128 && head_dim != 256 && head_dim != 512) return OSCAR_ERR_UNSUPPORTED;
  *bytes = oscar::calibrate_rv_workspace_bytes(head_dim, n_kv_rows);
  return OSCAR_OK;
}

int oscar_calibrate_rv(const float* q, int64_t n_q_rows, const float* k, const float* v, int64_t n_kv_rows,
                       int32_t head_dim, float* R_V_out, void* workspace, uint64_t workspace_bytes,
                       int32_t* dev_status, void* stream) {
  if (head_dim != 128 && head_dim != 256 && head_dim != 512) return OSCAR_ERR_UNSUPPORTED;
  if (!q || !k || !v || !R_V_out || !workspace) return OSCAR_ERR_INVALID;
  if (n_q_rows < 1 || n_q_rows > OSCAR_KV_CALIB_MAX_ROWS || n_kv_rows < 1 || n_kv_rows > OSCAR_KV_CALIB_MAX_ROWS)
    return OSCAR_ERR_INVALID;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(R_V_out, 16) || !aligned(workspace, 256))
    return OSCAR_ERR_INVALID;
  if (workspace_bytes < oscar::calibrate_rv_workspace_bytes(head_dim, n_kv_rows)) return OSCAR_ERR_WORKSPACE;
  return oscar::launch_calibrate_rv(q, n_q_rows, k, v, n_kv_rows, head_dim, R_V_out, workspace, dev_status,
                                    static_cast<cudaStream_t>(stream));
}

}  // extern "C"
