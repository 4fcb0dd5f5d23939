// varlen_step.h -- launch structs of the operators around a step of the paged
// attention: rotary positions and the cache write behind them, the step's plan
// (pages, slots, positions, masks), moving accepted rows, giving pages back.
#pragma once

#include "varlen_paged.h"

namespace varlen {

// ------------------------------------------------- rotary positions
struct RotaryParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16 *q_out, *k_out;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, qo_rs, qo_hs, ko_rs, ko_hs;
  const int32_t* positions;  // null: the row's index within its segment of cu
  const int32_t* cu;
  const uint64_t* turns;
  int32_t batch, total, heads, kv_heads, head_dim, rot;
  int32_t q_same, k_same;    // in place: elements behind rot are left alone
  float scale, sign;         // sign -1: turns back
  // into the cache (kv_heads of K, then of V)
  const int64_t* slots;
  uint8_t *kp, *vp;
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;  // byte strides of the pages
  __nv_bfloat16 *k_scale, *v_scale;
  int32_t num_pages, page_shift;
  unsigned int* err;
  Span q_span, k_span, v_span, qo_span, ko_span, kp_span, vp_span, ks_span, vs_span;  // bounds-checking build
};

enum RotaryTo : int { kToRows = 0, kToCacheBf16 = 1, kToCacheE4m3 = 2 };

struct RotaryLaunch {
  RotaryParams p;
  bool interleaved;
  RotaryTo to;
};

cudaError_t launch_rotary(const RotaryLaunch& L, cudaStream_t stream);

// ------------------------------------------------- the step's lists
struct PoolView {
  int32_t* table;
  int64_t table_stride;
  const int32_t* seqlens;
  int32_t* seqlens_out;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t num_pages, page_size, page_shift, max_pages;
};

// What the plan's first kernel finds out about a sequence.
struct PlanSeq {
  int32_t old;   // positions before the call
  int32_t row0;  // first packed row
  int32_t n;     // new rows
  int32_t top;   // place on the stack of its first new page (the next ones lie below); -1: it gets none
};

struct PlanParams {
  PoolView pool;
  const int32_t *new_lens, *parents;
  int32_t* cu;
  int64_t* slots;
  int32_t *positions, *unplaced;
  uint32_t* masks;
  int32_t batch, total, mask_words;
  PlanSeq* seqs;  // workspace
  unsigned int* err;
  Span slots_span, positions_span, masks_span, parents_span;  // bounds-checking build
};

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream);

struct TrimParams {
  PoolView pool;
  const int32_t *lens, *cu;
  int32_t batch;
  unsigned int* err;
  Span free_span;  // bounds-checking build
};

cudaError_t launch_trim(const TrimParams& p, cudaStream_t stream);

// ------------------------------------------------- accepted rows
constexpr int kMoveLayers = 64;  // caches of one launch (2 KB of its parameters)

struct MoveLayer {
  uint8_t *k, *v;
  __nv_bfloat16 *k_scale, *v_scale;
};

struct MoveParams {
  MoveLayer layer[kMoveLayers];
  int64_t k_page, k_row, k_head, v_page, v_row, v_head;  // byte strides of the pages
  PageView pages;
  const int32_t *cu, *kept, *kept_lens;
  int64_t kept_stride;
  int32_t batch, total, max_kept, heads, row_bytes;  // row_bytes: of one head's row of K or V
  unsigned int* err;
  int64_t kp_bytes, vp_bytes, s_bytes;  // extents (bounds-checking build)
};

struct MoveLaunch {
  MoveParams p;
  int layers;
  bool e4m3;
};

cudaError_t launch_move(const MoveLaunch& L, cudaStream_t stream);

}  // namespace varlen
