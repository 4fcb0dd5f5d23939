// varlen_paged.h -- launch structs of the paged key/value cache (write, read)
// and of the attention over it, and the device helpers that resolve a cache
// position to its page.
#pragma once

#include "varlen_attn.h"
#include "varlen_internal.h"
#include "varlen_sched.cuh"

namespace varlen {

// ------------------------------------------------- from varlen_api.cu
// SM count and error word of the current device (VARLEN_ERR_ARCH elsewhere).
int launch_device(int* sms, unsigned int** err);
// Argument checks of one NHD operand, as input and as output.
int check_nhd(const void* ptr, varlen_stride s, int64_t rows, int32_t H, int32_t D, bool output);
// A tiled tensor map of `rank` dimensions (128-byte swizzle or none), 64-bit extents.
int encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* byte_strides, const cuuint32_t* box, bool swizzle);
// Loads that the producers of CTA 0 leave out (failure test; < 0: none).
void paged_skip_knobs(int32_t* few, int32_t* many);
// [base, base + bytes), shortened by the bounds checker's self test.
Span checked_span(const void* base, int64_t bytes);
// The bytes an NHD bf16 operand occupies.
Span nhd_bytes(const void* base, varlen_stride s, int64_t rows, int32_t H, int32_t D);

// ------------------------------------------------- the cache
// (Lengths, table, cu_seqlens and queries are read by ordinary loads: the
// attention's kernels may start while earlier ones still write them, which the
// non-coherent path does not allow.)
struct PageView {
  const int32_t* table;
  int64_t table_stride;
  const int32_t* seqlens;
  int32_t num_pages, max_pages, page_size, page_shift;
};

// ------------------------------------------------- from varlen_paged_api.cu
// Argument checks of a cache; `lists`: of its table and lengths too.
int check_cache(const varlen_kv_cache* cache, int32_t batch, bool lists, int* page_shift);
// Log2 of a page size, -1 for one that is not allowed.
int page_shift_of(int32_t page_size);
// Bytes of an element, of a page array and of a scale array.
int elem_bytes(const varlen_kv_cache& c);
int64_t pages_bytes(const varlen_kv_cache& c, varlen_page_stride s);
int64_t scale_bytes(const varlen_kv_cache& c);
PageView view_of(const varlen_kv_cache& c, int shift);

// Positions sequence b holds, clamped to what its table row can name.
__device__ __forceinline__ int32_t cache_len(const PageView& c, int32_t b) {
  const int64_t cap = (int64_t)c.max_pages << c.page_shift;
  return (int32_t)min((int64_t)max(c.seqlens[b], 0), cap);
}

// Page that holds positions [i << page_shift, ...) of sequence b, 0 <= i <
// max_pages; num_pages (no page) for an entry that names none, recorded as an
// error unless it is the -1 of a plan that had no page to give (PLANNED: calls that
// come behind a plan, for which that is an ordinary outcome).
template <bool PLANNED>
__device__ __forceinline__ int32_t page_at(const PageView& c, int32_t b, int32_t i, unsigned int* err) {
  const int32_t id = c.table[(int64_t)b * c.table_stride + i];
  if ((uint32_t)id < (uint32_t)c.num_pages) return id;
  if (err != nullptr && !(PLANNED && id == -1)) atomicOr(err, (unsigned int)kErrBounds);
  return c.num_pages;
}

// The last segment b with cu[b] <= row (cu non-decreasing; any array gives
// some b in [0, batch)), found by the whole warp 32 entries at a time.
__device__ __forceinline__ int32_t warp_find_segment(const int32_t* cu, int32_t batch, int32_t total, int32_t row) {
  int32_t lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t i = (int64_t)lo + (int64_t)(threadIdx.x & 31) * step;
    const bool below = i < hi && clamp_row(cu[i], total) <= row;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int32_t k = m == 0 ? 0 : 31 - __clz(m);
    lo += k * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

struct CacheParams {
  const __nv_bfloat16 *k_new, *v_new;  // write: the new rows
  __nv_bfloat16 *k_out, *v_out;        // read: where the rows go
  int64_t k_rs, k_hs, v_rs, v_hs;      // packed rows
  uint8_t *k, *v;                      // pages
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;  // byte strides of the pages
  __nv_bfloat16 *k_scale, *v_scale;    // E4M3 only
  PageView pages;
  const int32_t* cu;
  int32_t batch, total, heads;
  unsigned int* err;
  Span k_span, v_span, kp_span, vp_span, ks_span, vs_span;  // packed rows, pages, scales (bounds-checking build)
};

struct CacheLaunch {
  CacheParams p;
  int head_dim;
  bool e4m3, write;
};

cudaError_t launch_cache(const CacheLaunch& L, cudaStream_t stream);

// ------------------------------------------------- attention over the cache
struct PagedParams {
  const __nv_bfloat16* q;
  int64_t q_rs, q_hs;
  __nv_bfloat16* out;
  int64_t o_rs, o_hs;
  float* lse;
  PageView pages;  // (keys, values and scales are read by TMA alone)
  const int32_t* cu_q;
  int32_t batch, total_q, kv_heads, group;
  int64_t win_left, win_right;
  float scale_log2;
  unsigned int* err;
  // drafted trees (their kernels only): which of the segment's new rows each row
  // sees, and where it stands (read with a bounded win_left)
  const uint32_t* masks;
  const int32_t* tree_pos;
  int32_t mask_words;
  int32_t debug_skip_few, debug_skip_many;  // < 0: off; else CTA 0's producer skips its load number n (failure test)
  Span q_span, out_span, lse_span, masks_span, pos_span;  // bounds-checking build
};

// What a kernel takes: segments of at most kFewRows rows, of more, or all.
enum PagedTake : int32_t { kTakeFew = 0, kTakeMany = 1, kTakeAll = 2 };

// Rows (queries x heads of a group) up to which the kernel for few rows takes a
// segment, and rows of its units.  us for the kernel for few rows and the one for
// many, one token a sequence, D = 128, 64 ragged sequences of up to 8192 keys
// and 8 key heads / 64 of 1000 and 8 / 32 of 8000 and 2 / 4 of 4000 and 8 / one
// of 60000 and 2: at 16 rows E4M3 166 and 220 / 52 and 82 / 50 and 61; at 17
// E4M3 272 and 225 / 80 and 89 / 78 and 64 / 38 and 29 / 34 and 37, bf16 315 and
// 192 / 94 and 72 / 90 and 59 / 27 and 26 / 27 and 36; from there to 32 rows
// neither changes by more than a tenth.
constexpr int kFewRows = 16;
constexpr int kFewTile = 64;      // keys per tile of that kernel
// its CTAs on an SM: E4M3 rows are half as long, so more of them have to be in the making
constexpr int few_ctas(bool e4m3) { return e4m3 ? 3 : 2; }
constexpr int kChunkRows = 256;   // rows of a unit of the kernel for many rows (two halves)
constexpr int kChunkTile = 128;   // keys per tile of that kernel
constexpr int kMaxSms = 160;      // the workspace is sized for this many

// What CTA c left for the join: [2 c + 1] the unit that it begins and does not
// end, [2 c] the unit that an earlier CTA began: the CTA that began it and the
// number of CTAs that hold it (0: there is no such unit).
struct PagedJoin {
  int32_t b, kh, blk, first, parts;
};

// Partial results of one kernel in the workspace: slot 2 c + (the CTA begins
// the unit) holds rows [rows][D] of the unnormalised output and [rows][2] of
// (m, l), m in the exp2 domain.
struct PagedParts {
  float* o;
  float* ml;
  PagedJoin* join;
  int32_t rows;  // rows of a slot
  Span o_span, ml_span, join_span;  // bounds-checking build
};

struct PagedLaunch {
  PagedParams p;
  int head_dim, sms;
  bool e4m3, tree;
  bool few, many;  // which kernels run; alone, each takes every segment
  CUtensorMap few_k, few_v, few_ks, few_vs;  // pages and (E4M3) scales in boxes of up to kFewTile keys
  CUtensorMap chunk_q;                       // {D, group, key heads, rows}, boxes of half a unit
  CUtensorMap chunk_k, chunk_v, chunk_ks, chunk_vs;  // the cache in boxes of up to kChunkTile keys
  PagedParts few_parts, chunk;
};

// Byte offsets of the workspace.  (A call whose rows all together are no more
// than kFewRows has no segment for the kernel for many rows.)
struct PagedSection {
  size_t at, bytes;
};
struct PagedWorkspace {
  PagedSection few_o, few_ml, few_join, chunk_o, chunk_ml, chunk_join;
  size_t bytes;
  int32_t few_rows;
};
inline PagedWorkspace paged_workspace(int64_t total_rows, int32_t head_dim) {  // of either type
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const PagedSection a{at, bytes};
    at += (bytes + 255) & ~size_t(255);
    return a;
  };
  PagedWorkspace w;
  w.few_rows = (int32_t)(total_rows < kFewRows ? (total_rows < 1 ? 1 : total_rows) : kFewRows);
  const size_t few = (size_t)few_ctas(true) * kMaxSms, many = total_rows > kFewRows ? kMaxSms : 0;
  w.few_o = take(2 * few * w.few_rows * head_dim * 4);
  w.few_ml = take(2 * few * w.few_rows * 8);
  w.few_join = take(2 * few * sizeof(PagedJoin));
  w.chunk_o = take(2 * many * kChunkRows * head_dim * 4);
  w.chunk_ml = take(2 * many * kChunkRows * 8);
  w.chunk_join = take(2 * many * sizeof(PagedJoin));
  w.bytes = at;
  return w;
}

// A kernel whose launch may begin while the one before it on the stream ends.
// Every thread of it waits (dependency_wait) before it touches global memory,
// so that a grid ends only after all those before it on the stream: what any of
// them wrote is complete where the wait returns.  (A kernel that skips the wait
// has no claim to see anything, whatever waits stand in the grids before it.)
template <class... P, class... A>
cudaError_t launch_overlapped(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

cudaError_t launch_paged_few(const PagedLaunch& L, int32_t take, cudaStream_t stream);
cudaError_t launch_paged_chunk(const PagedLaunch& L, int32_t take, cudaStream_t stream);
cudaError_t launch_paged_join(const PagedLaunch& L, cudaStream_t stream);
cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream);

}  // namespace varlen
