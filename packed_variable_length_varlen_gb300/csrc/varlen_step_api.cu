// varlen_step_api.cu -- the C entry points around a step of the paged attention
// (declared in varlen_attn.h): rotary positions, the cache write behind them, the
// step's plan, accepted rows, pages given back.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "varlen_step.h"

using namespace varlen;

namespace {

constexpr int32_t kMaxPlanBatch = 1 << 20;
constexpr int32_t kMaxMaskWords = 128;
constexpr int32_t kMaxMoveCaches = 1024;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_rotary(const varlen_rotary* r, int32_t head_dim) {
  if (r == nullptr) return VARLEN_ERR_NULL;
  if (r->rotary_dim < 8 || r->rotary_dim > head_dim || r->rotary_dim % 8 != 0) return VARLEN_ERR_SHAPE;
  if ((r->interleaved != 0 && r->interleaved != 1) || !std::isfinite(r->scale)) return VARLEN_ERR_SHAPE;
  if (r->turns == nullptr) return VARLEN_ERR_NULL;
  return aligned(r->turns, 8) ? VARLEN_OK : VARLEN_ERR_ALIGN;
}

// An input and the output it is turned into: two tensors, or one and the same.
int check_turned(const void* in, varlen_stride si, const void* out, varlen_stride so, int32_t total, int32_t heads,
                 int32_t head_dim) {
  int st;
  if ((st = check_nhd(in, si, total, heads, head_dim, false)) != VARLEN_OK) return st;
  if ((st = check_nhd(out, so, total, heads, head_dim, true)) != VARLEN_OK) return st;
  if (in != out || total == 0) return VARLEN_OK;
  return (total > 1 && si.row != so.row) || (heads > 1 && si.head != so.head) ? VARLEN_ERR_STRIDE : VARLEN_OK;
}

// What both rotary calls say of the turn itself and of the queries.
void set_rotary(RotaryLaunch& L, const varlen_rotary& r, const int32_t* positions, int32_t total, int32_t heads,
                int32_t kv_heads, int32_t head_dim, const void* q, varlen_stride sq, const void* k, varlen_stride sk,
                void* q_out, varlen_stride sqo, unsigned int* err) {
  std::memset(&L, 0, sizeof(L));
  L.interleaved = r.interleaved != 0;
  RotaryParams& p = L.p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_rs = sq.row;
  p.q_hs = sq.head;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.k_rs = sk.row;
  p.k_hs = sk.head;
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.qo_rs = sqo.row;
  p.qo_hs = sqo.head;
  p.q_same = q == q_out;
  p.positions = positions;
  p.turns = r.turns;
  p.total = total;
  p.heads = heads;
  p.kv_heads = kv_heads;
  p.head_dim = head_dim;
  p.rot = r.rotary_dim;
  p.scale = r.scale;
  p.sign = 1.f;
  p.err = err;
  p.q_span = nhd_bytes(q, sq, total, heads, head_dim);
  p.qo_span = nhd_bytes(q_out, sqo, total, heads, head_dim);
  p.k_span = nhd_bytes(k, sk, total, kv_heads, head_dim);
}

int check_pool(const varlen_page_pool* pool, int32_t batch, PoolView* view) {
  if (pool == nullptr) return VARLEN_ERR_NULL;
  const varlen_page_pool& c = *pool;
  const int shift = page_shift_of(c.page_size);
  if (shift < 0 || batch < 1 || batch > kMaxPlanBatch || c.num_pages < 1 || c.max_pages < 0) return VARLEN_ERR_SHAPE;
  if (((int64_t)c.max_pages << shift) > (int64_t(1) << 31) - 2048 || (int64_t)batch * c.max_pages > INT32_MAX) return VARLEN_ERR_SHAPE;
  if ((c.max_pages > 0 && c.block_table == nullptr) || c.seqlens == nullptr || c.seqlens_out == nullptr ||
      c.free_pages == nullptr || c.free_count == nullptr || c.free_count_out == nullptr)
    return VARLEN_ERR_NULL;
  if (c.table_stride < 0 || (batch > 1 && c.table_stride < c.max_pages) || c.table_stride >= (int64_t(1) << 40)) return VARLEN_ERR_STRIDE;
  *view = PoolView{c.block_table, c.table_stride, c.seqlens,   c.seqlens_out, c.free_pages, c.free_count,
                   c.free_count_out, c.num_pages, c.page_size, shift,         c.max_pages};
  return VARLEN_OK;
}

bool same(varlen_page_stride a, varlen_page_stride b) { return a.page == b.page && a.row == b.row && a.head == b.head; }

// f / 2 pi in whole 2^-64 turns, rounded once: 1 / 2 pi in two doubles leaves 2^-104 of the
// quotient, and the two parts of the product are brought into a turn without rounding.
uint64_t turns_of(double f) {
  constexpr double kInv = 0x1.45f306dc9c883p-3, kInvLess = -0x1.6b01ec5417056p-57;  // of 1 / 2 pi: the nearest double, the rest's
  constexpr double kUnits = 18446744073709551616.0;
  const double a = std::fabs(f), hi = a * kInv, lo = std::fma(a, kInvLess, std::fma(a, kInv, -hi));
  const double up = std::fmod(hi, 1.0) * kUnits, whole = std::floor(up);
  const double less = std::rint(std::remainder(lo, 1.0) * kUnits + (up - whole));  // at most 2^63 + 1 either way
  const uint64_t t = (uint64_t)whole + (less < 0 ? 0 - (uint64_t)-less : (uint64_t)less);  // (modulo a turn)
  return f < 0 ? 0 - t : t;
}

int done(cudaError_t e) { return e == cudaSuccess ? VARLEN_OK : cuda_fail(e); }

}  // namespace

extern "C" int varlen_attn_rotary_turns(const double* frequencies, int32_t count, uint64_t* turns) {
  if (count < 0) return VARLEN_ERR_SHAPE;
  if (count > 0 && (frequencies == nullptr || turns == nullptr)) return VARLEN_ERR_NULL;
  for (int32_t i = 0; i < count; ++i)
    if (!std::isfinite(frequencies[i])) return VARLEN_ERR_SHAPE;
  for (int32_t i = 0; i < count; ++i) turns[i] = turns_of(frequencies[i]);
  return VARLEN_OK;
}

extern "C" int varlen_attn_rotary(const void* q, varlen_stride sq, const void* k, varlen_stride sk,
                                  const int32_t* positions, const int32_t* cu_seqlens, int32_t batch, int32_t total,
                                  int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, const varlen_rotary* rotary,
                                  int32_t inverse, void* q_out, varlen_stride sqo, void* k_out, varlen_stride sko,
                                  void* stream) {
  if (total < 0 || num_heads < 0 || num_kv_heads < 0 || (int64_t)num_heads + num_kv_heads < 1 ||
      (int64_t)num_heads + num_kv_heads > (1 << 20))
    return VARLEN_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128) return VARLEN_ERR_HEAD_DIM;
  int st;
  if ((st = check_rotary(rotary, head_dim)) != VARLEN_OK) return st;
  if (positions == nullptr) {
    if (cu_seqlens == nullptr) return VARLEN_ERR_NULL;
    if (batch < 1 || batch > (1 << 30)) return VARLEN_ERR_SHAPE;
  }
  if (num_heads > 0 && (st = check_turned(q, sq, q_out, sqo, total, num_heads, head_dim)) != VARLEN_OK) return st;
  if (num_kv_heads > 0 && (st = check_turned(k, sk, k_out, sko, total, num_kv_heads, head_dim)) != VARLEN_OK) return st;
  int sms = 0;
  unsigned int* err = nullptr;
  if ((st = launch_device(&sms, &err)) != VARLEN_OK) return st;
  if (total == 0) return VARLEN_OK;
  RotaryLaunch L;
  set_rotary(L, *rotary, positions, total, num_heads, num_kv_heads, head_dim, q, sq, k, sk, q_out, sqo, err);
  L.to = kToRows;
  RotaryParams& p = L.p;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.ko_rs = sko.row;
  p.ko_hs = sko.head;
  p.k_same = k == k_out;
  p.cu = cu_seqlens;
  p.batch = batch;
  p.sign = inverse != 0 ? -1.f : 1.f;
  p.ko_span = nhd_bytes(k_out, sko, total, num_kv_heads, head_dim);
  return done(launch_rotary(L, static_cast<cudaStream_t>(stream)));
}

extern "C" int varlen_attn_rotary_cache_write(const void* q, varlen_stride sq, const void* k, varlen_stride sk,
                                              const void* v, varlen_stride sv, const int32_t* positions,
                                              const int64_t* slots, int32_t total, int32_t num_heads,
                                              const varlen_kv_cache* cache, const varlen_rotary* rotary, void* q_out,
                                              varlen_stride sqo, void* stream) {
  int shift = 0;
  int st = check_cache(cache, 1, false, &shift);
  if (st != VARLEN_OK) return st;
  const varlen_kv_cache& c = *cache;
  if (total < 0 || num_heads < 0 || (int64_t)num_heads + 2 * (int64_t)c.num_kv_heads > (1 << 20)) return VARLEN_ERR_SHAPE;
  if ((st = check_rotary(rotary, c.head_dim)) != VARLEN_OK) return st;
  if (total > 0 && (positions == nullptr || slots == nullptr)) return VARLEN_ERR_NULL;
  if (!aligned(slots, 8)) return VARLEN_ERR_ALIGN;
  if (num_heads > 0 && (st = check_turned(q, sq, q_out, sqo, total, num_heads, c.head_dim)) != VARLEN_OK) return st;
  if ((st = check_nhd(k, sk, total, c.num_kv_heads, c.head_dim, false)) != VARLEN_OK) return st;
  if ((st = check_nhd(v, sv, total, c.num_kv_heads, c.head_dim, false)) != VARLEN_OK) return st;
  int sms = 0;
  unsigned int* err = nullptr;
  if ((st = launch_device(&sms, &err)) != VARLEN_OK) return st;
  if (total == 0) return VARLEN_OK;
  const int64_t es = elem_bytes(c);
  RotaryLaunch L;
  set_rotary(L, *rotary, positions, total, num_heads, c.num_kv_heads, c.head_dim, q, sq, k, sk, q_out, sqo, err);
  L.to = c.type == VARLEN_CACHE_BF16 ? kToCacheBf16 : kToCacheE4m3;
  RotaryParams& p = L.p;
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.v_rs = sv.row;
  p.v_hs = sv.head;
  p.slots = slots;
  p.kp = static_cast<uint8_t*>(c.k);
  p.vp = static_cast<uint8_t*>(c.v);
  p.k_page = c.sk.page * es;
  p.k_row = c.sk.row * es;
  p.k_head = c.sk.head * es;
  p.v_page = c.sv.page * es;
  p.v_row = c.sv.row * es;
  p.v_head = c.sv.head * es;
  p.k_scale = static_cast<__nv_bfloat16*>(c.k_scale);
  p.v_scale = static_cast<__nv_bfloat16*>(c.v_scale);
  p.num_pages = c.num_pages;
  p.page_shift = shift;
  p.v_span = nhd_bytes(v, sv, total, c.num_kv_heads, c.head_dim);
  p.kp_span = checked_span(c.k, pages_bytes(c, c.sk));
  p.vp_span = checked_span(c.v, pages_bytes(c, c.sv));
  p.ks_span = checked_span(c.k_scale, scale_bytes(c));
  p.vs_span = checked_span(c.v_scale, scale_bytes(c));
  return done(launch_rotary(L, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t varlen_attn_cache_plan_workspace_size(int32_t batch) {
  return batch < 0 || batch > kMaxPlanBatch ? 0 : (size_t)std::max(batch, 1) * sizeof(PlanSeq);
}

extern "C" int varlen_attn_cache_plan(const varlen_page_pool* pool, const int32_t* new_lens, int32_t batch,
                                      const int32_t* parents, int32_t total, int32_t* cu_seqlens, int64_t* slots,
                                      int32_t* positions, int32_t* unplaced, uint32_t* masks, int32_t mask_words,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  PlanParams p;
  std::memset(&p, 0, sizeof(p));
  int st = check_pool(pool, batch, &p.pool);
  if (st != VARLEN_OK) return st;
  if (total < 0 || total > INT32_MAX - 2048) return VARLEN_ERR_SHAPE;
  if (parents != nullptr && (mask_words < 1 || mask_words > kMaxMaskWords)) return VARLEN_ERR_SHAPE;
  if (new_lens == nullptr || cu_seqlens == nullptr || unplaced == nullptr) return VARLEN_ERR_NULL;
  if (total > 0 && (slots == nullptr || positions == nullptr || (parents != nullptr && masks == nullptr))) return VARLEN_ERR_NULL;
  if (!aligned(slots, 8)) return VARLEN_ERR_ALIGN;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < varlen_attn_cache_plan_workspace_size(batch))
    return VARLEN_ERR_WORKSPACE;
  int sms = 0;
  if ((st = launch_device(&sms, &p.err)) != VARLEN_OK) return st;
  p.new_lens = new_lens;
  p.parents = parents;
  p.cu = cu_seqlens;
  p.slots = slots;
  p.positions = positions;
  p.unplaced = unplaced;
  p.masks = masks;
  p.batch = batch;
  p.total = total;
  p.mask_words = mask_words;
  p.seqs = static_cast<PlanSeq*>(workspace);
  p.slots_span = checked_span(slots, (int64_t)total * 8);
  p.positions_span = checked_span(positions, (int64_t)total * 4);
  p.masks_span = checked_span(masks, (int64_t)total * mask_words * 4);
  p.parents_span = checked_span(parents, (int64_t)total * 4);
  return done(launch_plan(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int varlen_attn_cache_trim(const varlen_page_pool* pool, const int32_t* lens, const int32_t* cu_seqlens,
                                      int32_t batch, void* stream) {
  TrimParams p;
  std::memset(&p, 0, sizeof(p));
  int st = check_pool(pool, batch, &p.pool);
  if (st != VARLEN_OK) return st;
  if (lens == nullptr) return VARLEN_ERR_NULL;
  int sms = 0;
  if ((st = launch_device(&sms, &p.err)) != VARLEN_OK) return st;
  p.lens = lens;
  p.cu = cu_seqlens;
  p.batch = batch;
  p.free_span = checked_span(pool->free_pages, (int64_t)pool->num_pages * 4);
  return done(launch_trim(p, static_cast<cudaStream_t>(stream)));
}

extern "C" int varlen_attn_cache_move(const varlen_kv_cache* caches, int32_t count, const int32_t* cu_seqlens,
                                      int32_t batch, int32_t total, const int32_t* kept, int64_t kept_stride,
                                      const int32_t* kept_lens, int32_t max_kept, void* stream) {
  if (count < 1 || count > kMaxMoveCaches || total < 0 || max_kept < 0) return VARLEN_ERR_SHAPE;
  if (caches == nullptr) return VARLEN_ERR_NULL;
  const varlen_kv_cache& c = caches[0];
  int shift = 0, st;
  for (int32_t i = 0; i < count; ++i) {
    const varlen_kv_cache& x = caches[i];
    if ((st = check_cache(&x, batch, true, &shift)) != VARLEN_OK) return st;
    if (x.type != c.type || x.num_pages != c.num_pages || x.page_size != c.page_size || x.max_pages != c.max_pages ||
        x.num_kv_heads != c.num_kv_heads || x.head_dim != c.head_dim || x.block_table != c.block_table ||
        x.table_stride != c.table_stride || x.seqlens != c.seqlens || !same(x.sk, c.sk) || !same(x.sv, c.sv))
      return VARLEN_ERR_SHAPE;
  }
  if (c.num_kv_heads > (1 << 20)) return VARLEN_ERR_SHAPE;
  if (cu_seqlens == nullptr || kept_lens == nullptr || (max_kept > 0 && kept == nullptr)) return VARLEN_ERR_NULL;
  if (kept_stride < 0) return VARLEN_ERR_STRIDE;
  int sms = 0;
  unsigned int* err = nullptr;
  if ((st = launch_device(&sms, &err)) != VARLEN_OK) return st;
  if (max_kept == 0 || total == 0) return VARLEN_OK;
  const int64_t es = elem_bytes(c);
  MoveLaunch L;
  std::memset(&L, 0, sizeof(L));
  MoveParams& p = L.p;
  p.k_page = c.sk.page * es;
  p.k_row = c.sk.row * es;
  p.k_head = c.sk.head * es;
  p.v_page = c.sv.page * es;
  p.v_row = c.sv.row * es;
  p.v_head = c.sv.head * es;
  p.pages = view_of(c, shift);
  p.cu = cu_seqlens;
  p.kept = kept;
  p.kept_lens = kept_lens;
  p.kept_stride = kept_stride;
  p.batch = batch;
  p.total = total;
  p.max_kept = max_kept;
  p.heads = c.num_kv_heads;
  p.row_bytes = (int32_t)(c.head_dim * es);
  p.err = err;
  p.kp_bytes = checked_span(c.k, pages_bytes(c, c.sk)).bytes;
  p.vp_bytes = checked_span(c.v, pages_bytes(c, c.sv)).bytes;
  p.s_bytes = checked_span(c.k_scale, scale_bytes(c)).bytes;
  L.e4m3 = c.type == VARLEN_CACHE_E4M3;
  for (int32_t first = 0; first < count; first += kMoveLayers) {
    L.layers = std::min(count - first, kMoveLayers);
    for (int i = 0; i < L.layers; ++i) {
      const varlen_kv_cache& x = caches[first + i];
      p.layer[i] = MoveLayer{static_cast<uint8_t*>(x.k), static_cast<uint8_t*>(x.v), static_cast<__nv_bfloat16*>(x.k_scale),
                             static_cast<__nv_bfloat16*>(x.v_scale)};
    }
    const cudaError_t e = launch_move(L, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return VARLEN_OK;
}
