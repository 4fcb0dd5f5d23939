// varlen_paged_api.cu -- the C entry points of the paged cache and of the
// attention over it (declared in varlen_attn.h): argument checks, 64-bit
// extents, launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <utility>

#include "varlen_paged.h"

using namespace varlen;

namespace {

constexpr int32_t kMaxBatch = 1 << 30;  // strides over the batch stay in int32
constexpr float kLog2e = 1.4426950408889634f;

int elem_bytes(const varlen_kv_cache& c) { return c.type == VARLEN_CACHE_BF16 ? 2 : 1; }

// Bytes from the base to the end of the last (page, row, head) vector.
int64_t pages_bytes(const varlen_kv_cache& c, varlen_page_stride s) {
  const int64_t page = c.num_pages > 1 ? (c.num_pages - 1) * s.page : 0, row = (c.page_size - 1) * s.row;
  return elem_bytes(c) * (page + row + (c.num_kv_heads > 1 ? (c.num_kv_heads - 1) * s.head : 0) + c.head_dim);
}
int64_t scale_bytes(const varlen_kv_cache& c) { return (int64_t)2 * c.num_pages * c.num_kv_heads * c.page_size; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Strides of one page array: 16-byte multiples below 2^40 bytes whose
// (page, row, head) vectors do not overlap.
int check_pages(const varlen_kv_cache& c, varlen_page_stride s) {
  const int64_t es = elem_bytes(c);
  std::pair<int64_t, int64_t> d[3] = {{s.page, c.num_pages}, {s.row, c.page_size}, {s.head, c.num_kv_heads}};  // stride, extent
  for (auto& x : d)
    if (x.first < 0 || x.first >= (int64_t(1) << 40) / es || (x.first * es & 15) != 0) return VARLEN_ERR_STRIDE;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (d[j + 1].first < d[j].first) std::swap(d[j], d[j + 1]);
  int64_t need = c.head_dim;  // elements that the dimensions so far occupy
  for (auto& x : d) {
    if (x.second <= 1) continue;
    if (x.first < need || x.first > (int64_t(1) << 60) / x.second) return VARLEN_ERR_STRIDE;
    need = x.first * x.second;
  }
  return VARLEN_OK;
}

int check_cache(const varlen_kv_cache* cache, int32_t batch, int* page_shift) {
  if (cache == nullptr) return VARLEN_ERR_NULL;
  const varlen_kv_cache& c = *cache;
  if (batch < 1 || batch > kMaxBatch || c.num_pages < 1 || c.max_pages < 0 || c.num_kv_heads < 1 || c.table_stride < 0) return VARLEN_ERR_SHAPE;
  if (c.type != VARLEN_CACHE_BF16 && c.type != VARLEN_CACHE_E4M3) return VARLEN_ERR_SHAPE;
  int shift = 4;
  while (shift < 11 && (1 << shift) != c.page_size) ++shift;
  if (shift == 11) return VARLEN_ERR_SHAPE;
  if (((int64_t)c.max_pages << shift) > (int64_t(1) << 31) - 2048) return VARLEN_ERR_SHAPE;  // tile ends stay in int32
  if (c.head_dim != 64 && c.head_dim != 96 && c.head_dim != 128) return VARLEN_ERR_HEAD_DIM;
  if (c.k == nullptr || c.v == nullptr || c.seqlens == nullptr || (c.max_pages > 0 && c.block_table == nullptr))
    return VARLEN_ERR_NULL;
  const bool scaled = c.type == VARLEN_CACHE_E4M3;
  if (scaled && (c.k_scale == nullptr || c.v_scale == nullptr)) return VARLEN_ERR_NULL;
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || (scaled && (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))))
    return VARLEN_ERR_ALIGN;
  int st;
  if ((st = check_pages(c, c.sk)) != VARLEN_OK || (st = check_pages(c, c.sv)) != VARLEN_OK) return st;
  *page_shift = shift;
  return VARLEN_OK;
}

PageView view_of(const varlen_kv_cache& c, int shift) {
  return PageView{c.block_table, c.table_stride, c.seqlens, c.num_pages, c.max_pages, c.page_size, shift};
}

// Pages as {D, heads, page rows, pages} in boxes of 128 bytes (64 bf16 or 128
// codes, zero past D) of `rows` rows of one head and page.
int encode_pages(CUtensorMap* map, const varlen_kv_cache& c, const void* base, varlen_page_stride s, int rows) {
  const cuuint64_t es = (cuuint64_t)elem_bytes(c), D = (cuuint64_t)c.head_dim;
  // (a stride over one element is never used: a legal value for it)
  const cuuint64_t head = c.num_kv_heads > 1 ? s.head * es : D * es, page = c.num_pages > 1 ? s.page * es : D * es;
  const cuuint64_t dims[4] = {D, (cuuint64_t)c.num_kv_heads, (cuuint64_t)c.page_size, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[3] = {head, s.row * es, page};
  const cuuint32_t box[4] = {(cuuint32_t)(128 / es), 1u, (cuuint32_t)rows, 1u};
  return encode_tiled(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims,
                      strides, box, true);
}

// Scales as {page rows, heads, pages} in boxes of `rows` scales.
int encode_scales(CUtensorMap* map, const varlen_kv_cache& c, const void* base, int rows) {
  const cuuint64_t n = (cuuint64_t)c.page_size;
  const cuuint64_t dims[3] = {n, (cuuint64_t)c.num_kv_heads, (cuuint64_t)c.num_pages};
  const cuuint64_t strides[2] = {n * 2, n * 2 * (cuuint64_t)c.num_kv_heads};
  const cuuint32_t box[3] = {(cuuint32_t)rows, 1u, 1u};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, false);
}

// Queries as {D, heads of a group, key heads, rows} in boxes of 64 columns of
// all rows of 128 / group tokens of one key head.
int encode_queries(CUtensorMap* map, const void* base, varlen_stride s, int32_t rows, int32_t kv_heads, int32_t group,
                   int32_t D) {
  // (a stride over one element is never used: a legal value for it)
  const cuuint64_t head = (int64_t)kv_heads * group > 1 ? s.head * 2 : D * 2, row = rows > 1 ? s.row * 2 : D * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)group, (cuuint64_t)kv_heads, (cuuint64_t)rows};
  const cuuint64_t strides[3] = {head, head * group, row};
  const cuuint32_t box[4] = {64u, (cuuint32_t)group, 1u, (cuuint32_t)(kChunkRows / 2 / group)};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, true);
}

int cache_impl(const void* k, varlen_stride sk, const void* v, varlen_stride sv, const int32_t* cu, int32_t batch,
               int32_t total, const varlen_kv_cache* cache, void* stream, bool write) {
  int shift = 0;
  int st = check_cache(cache, batch, &shift);
  if (st != VARLEN_OK) return st;
  if (total < 0) return VARLEN_ERR_SHAPE;
  if (cu == nullptr) return VARLEN_ERR_NULL;
  const varlen_kv_cache& c = *cache;
  if ((st = check_nhd(k, sk, total, c.num_kv_heads, c.head_dim, !write)) != VARLEN_OK) return st;
  if ((st = check_nhd(v, sv, total, c.num_kv_heads, c.head_dim, !write)) != VARLEN_OK) return st;
  int sms = 0;
  unsigned int* err = nullptr;
  if ((st = launch_device(&sms, &err)) != VARLEN_OK) return st;
  if (total == 0) return VARLEN_OK;
  const int64_t es = elem_bytes(c);
  CacheLaunch L;
  std::memset(&L, 0, sizeof(L));
  CacheParams& p = L.p;
  if (write) {
    p.k_new = static_cast<const __nv_bfloat16*>(k);
    p.v_new = static_cast<const __nv_bfloat16*>(v);
  } else {
    p.k_out = static_cast<__nv_bfloat16*>(const_cast<void*>(k));
    p.v_out = static_cast<__nv_bfloat16*>(const_cast<void*>(v));
  }
  p.k_rs = sk.row;
  p.k_hs = sk.head;
  p.v_rs = sv.row;
  p.v_hs = sv.head;
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.k_page = c.sk.page * es;
  p.k_row = c.sk.row * es;
  p.k_head = c.sk.head * es;
  p.v_page = c.sv.page * es;
  p.v_row = c.sv.row * es;
  p.v_head = c.sv.head * es;
  p.k_scale = static_cast<__nv_bfloat16*>(c.k_scale);
  p.v_scale = static_cast<__nv_bfloat16*>(c.v_scale);
  p.pages = view_of(c, shift);
  p.cu = cu;
  p.batch = batch;
  p.total = total;
  p.heads = c.num_kv_heads;
  p.err = err;
  p.k_span = nhd_bytes(k, sk, total, c.num_kv_heads, c.head_dim);
  p.v_span = nhd_bytes(v, sv, total, c.num_kv_heads, c.head_dim);
  p.kp_span = checked_span(c.k, pages_bytes(c, c.sk));
  p.vp_span = checked_span(c.v, pages_bytes(c, c.sv));
  p.ks_span = checked_span(c.k_scale, scale_bytes(c));
  p.vs_span = checked_span(c.v_scale, scale_bytes(c));
  L.head_dim = c.head_dim;
  L.e4m3 = c.type == VARLEN_CACHE_E4M3;
  L.write = write;
  const cudaError_t e = launch_cache(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VARLEN_OK : cuda_fail(e);
}

}  // namespace

extern "C" int varlen_attn_cache_write(const void* k, varlen_stride sk, const void* v, varlen_stride sv,
                                       const int32_t* cu_seqlens, int32_t batch, int32_t total,
                                       const varlen_kv_cache* cache, void* stream) {
  return cache_impl(k, sk, v, sv, cu_seqlens, batch, total, cache, stream, true);
}

extern "C" int varlen_attn_cache_read(const varlen_kv_cache* cache, const int32_t* cu_seqlens, int32_t batch,
                                      int32_t total, void* k, varlen_stride sk, void* v, varlen_stride sv,
                                      void* stream) {
  return cache_impl(k, sk, v, sv, cu_seqlens, batch, total, cache, stream, false);
}

extern "C" size_t varlen_attn_fwd_paged_workspace_size(int32_t batch, int32_t total_q, int32_t num_heads,
                                                       int32_t num_kv_heads, int32_t head_dim) {
  if (batch < 0 || total_q < 0 || num_heads < 0 || num_kv_heads < 1 || head_dim < 0) return 0;
  return paged_workspace((int64_t)total_q * (num_heads / num_kv_heads), head_dim).bytes;
}

extern "C" int varlen_attn_fwd_paged(const void* q, varlen_stride sq, const int32_t* cu_seqlens_q, int32_t batch,
                                     int32_t total_q, int32_t num_heads, int32_t max_seqlen_q,
                                     const varlen_kv_cache* cache, float scale, int32_t window_left,
                                     int32_t window_right, void* out, varlen_stride so, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  int shift = 0;
  int st = check_cache(cache, batch, &shift);
  if (st != VARLEN_OK) return st;
  const varlen_kv_cache& c = *cache;
  if (total_q < 0 || num_heads < 1 || num_heads % c.num_kv_heads != 0 || num_heads / c.num_kv_heads > 128)
    return VARLEN_ERR_SHAPE;
  if ((int64_t)total_q * num_heads > INT32_MAX - 256) return VARLEN_ERR_SHAPE;  // rows are counted in 32 bits
  if (!(scale > 0.f) || !std::isfinite(scale)) return VARLEN_ERR_SHAPE;
  if (cu_seqlens_q == nullptr) return VARLEN_ERR_NULL;
  if ((st = check_nhd(q, sq, total_q, num_heads, c.head_dim, false)) != VARLEN_OK) return st;
  if ((total_q > 1 && sq.row == 0) || (num_heads > 1 && sq.head == 0)) return VARLEN_ERR_STRIDE;
  if ((st = check_nhd(out, so, total_q, num_heads, c.head_dim, true)) != VARLEN_OK) return st;
  if (total_q > 0 && lse == nullptr) return VARLEN_ERR_NULL;
  const size_t need = varlen_attn_fwd_paged_workspace_size(batch, total_q, num_heads, c.num_kv_heads, c.head_dim);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < need) return VARLEN_ERR_WORKSPACE;
  int sms = 0;
  unsigned int* err = nullptr;
  if ((st = launch_device(&sms, &err)) != VARLEN_OK) return st;
  if (total_q == 0) return VARLEN_OK;
  PagedLaunch L;
  std::memset(&L, 0, sizeof(L));
  PagedParams& p = L.p;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_rs = sq.row;
  p.q_hs = sq.head;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.o_rs = so.row;
  p.o_hs = so.head;
  p.lse = lse;
  p.pages = view_of(c, shift);
  p.cu_q = cu_seqlens_q;
  p.batch = batch;
  p.total_q = total_q;
  p.kv_heads = c.num_kv_heads;
  p.group = num_heads / c.num_kv_heads;
  p.win_left = window_left < 0 ? kWinUnbounded : window_left;
  p.win_right = window_right < 0 ? kWinUnbounded : window_right;
  p.scale_log2 = scale * kLog2e;
  p.err = err;
  paged_skip_knobs(&p.debug_skip_few, &p.debug_skip_many);
  p.q_span = nhd_bytes(q, sq, total_q, num_heads, c.head_dim);
  p.out_span = nhd_bytes(out, so, total_q, num_heads, c.head_dim);
  p.lse_span = checked_span(lse, (int64_t)num_heads * total_q * 4);
  L.head_dim = c.head_dim;
  L.sms = std::min(sms, kMaxSms);
  L.e4m3 = c.type == VARLEN_CACHE_E4M3;
  // Which kernels.  Where every segment is known to have few rows, that one
  // alone; a single segment of more rows goes to the other one whatever its
  // length.  Of the rest, calls whose tables can name few key tiles go to the
  // one for many rows alone, which is two launches less; otherwise both run
  // and each takes the segments that are its own.  Measured with 13 (29, 61)
  // single tokens and 3 chunks of 10..60 tokens, 32/8 heads, us both and one, for
  // sequences of full and of ragged length: E4M3 16 x 4000 keys (27 tiles an SM)
  // 84 and 83 / 78 and 64, 16 x 6000 (40) 97 and 106 / 77 and 67, 16 x 8192 (54)
  // 115 and 135 / 77 and 88, 64 x 8192 (216) 237 and 463 / 179 and 233; bf16 16 x
  // 8192 132 and 125 / 85 and 77, 32 x 8192 (108) 206 and 224 / 121 and 110, 64 x
  // 8192 353 and 422 / 201 and 203.
  const int64_t total_rows = (int64_t)total_q * p.group;
  const bool known_few = total_rows <= kFewRows || (max_seqlen_q > 0 && (int64_t)max_seqlen_q * p.group <= kFewRows);
  L.few = known_few || batch > 1;
  L.many = !known_few;  // (so total_rows > kFewRows, and the workspace has its sections)
  const int64_t tiles = (int64_t)batch * c.num_kv_heads * ((((int64_t)c.max_pages << shift) + kChunkTile - 1) / kChunkTile);
  if (L.many && tiles <= (int64_t)(L.e4m3 ? 40 : 64) * sms) L.few = false;
  char* ws = static_cast<char*>(workspace);
  const PagedWorkspace w = paged_workspace(total_rows, c.head_dim);
  auto parts = [ws](PagedSection o, PagedSection ml, PagedSection join, int32_t rows) {
    auto span = [ws](PagedSection s) { return checked_span(ws + s.at, (int64_t)s.bytes); };
    return PagedParts{reinterpret_cast<float*>(ws + o.at), reinterpret_cast<float*>(ws + ml.at),
                      reinterpret_cast<PagedJoin*>(ws + join.at), rows, span(o), span(ml), span(join)};
  };
  L.few_parts = parts(w.few_o, w.few_ml, w.few_join, w.few_rows);
  L.chunk = parts(w.chunk_o, w.chunk_ml, w.chunk_join, kChunkRows);
  auto maps = [&](CUtensorMap* k, CUtensorMap* v, CUtensorMap* ks, CUtensorMap* vs, int tile) {
    const int box = std::min(c.page_size, tile);
    int s2;
    if ((s2 = encode_pages(k, c, c.k, c.sk, box)) != VARLEN_OK || (s2 = encode_pages(v, c, c.v, c.sv, box)) != VARLEN_OK)
      return s2;
    if (!L.e4m3) return (int)VARLEN_OK;
    if ((s2 = encode_scales(ks, c, c.k_scale, box)) != VARLEN_OK) return s2;
    return encode_scales(vs, c, c.v_scale, box);
  };
  if (L.few && (st = maps(&L.few_k, &L.few_v, &L.few_ks, &L.few_vs, kFewTile)) != VARLEN_OK) return st;
  if (L.many) {
    if ((st = maps(&L.chunk_k, &L.chunk_v, &L.chunk_ks, &L.chunk_vs, kChunkTile)) != VARLEN_OK) return st;
    if ((st = encode_queries(&L.chunk_q, q, sq, total_q, c.num_kv_heads, p.group, c.head_dim)) != VARLEN_OK) return st;
  }
  const cudaError_t e = launch_paged(L, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VARLEN_OK : cuda_fail(e);
}
