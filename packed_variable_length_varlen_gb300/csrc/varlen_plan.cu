// varlen_plan.cu -- the lists of a step of the paged attention, built on the
// GPU: where each new row goes and stands (plan), which pages come back (trim),
// and accepted rows moved behind the context (move).
//
// Plan and trim write a few bytes a row and are bound by latency: one launch, two
// or three prefix sums over the batch and a few dependent loads.  One CTA sums
// up (rows, then pages needed, so that every sequence knows its first row and its
// place on the stack of free pages), and small steps without trees are finished by
// the same CTA: 3.4 us for 512 rows, 4.3 for 2000, where a second kernel, a thread a
// row, makes it 4.5 to 6.4 (for 262144 rows).  (Trees want all SMs even when small: one
// CTA took 5.6 us for 2 trees of 32 rows and 8.6 for 62, two kernels take 5.2.)  A row finds its page from its
// sequence's sums alone, so rows depend on nothing but those; the row that opens
// a page writes the table's entry.
//
// Masks: the rows above a row in its tree.  A warp takes 32 rows of a sequence,
// one word of the mask.  Within the word it follows all parents at once, twice as
// far each time (five steps), which leaves for each row the bits of the word that
// are above it and the one row before the word that the topmost of them continues.
// A row's mask is then put together word by word, from the right: at most one look-up
// for each word before its own, whatever the depth of the tree.
#include <algorithm>

#include "sm103_ptx.cuh"
#include "varlen_step.h"

namespace varlen {

namespace {

constexpr int kPlanThreads = 1024;  // of the CTA that sums up; fewer sequences take fewer,
constexpr int kPlanFew = 256;       // whose barriers cost less
constexpr int kPlanSmall = 2048;    // rows up to which it does the rest as well
constexpr int kRowThreads = 256;    // of the second kernel

__device__ __forceinline__ int32_t pool_len(const PoolView& c, int32_t b) {
  return (int32_t)min((int64_t)max(c.seqlens[b], 0), (int64_t)c.max_pages << c.page_shift);
}
__device__ __forceinline__ int32_t pool_free(const PoolView& c) { return min(max(*c.free_count, 0), c.num_pages); }
__device__ __forceinline__ int64_t pages_of(const PoolView& c, int64_t len) {
  return (len + c.page_size - 1) >> c.page_shift;
}

// Inclusive sum over the CTA's THREADS threads; `all` is the whole one.
template <int THREADS>
__device__ __forceinline__ long long block_inclusive(long long v, long long* sums, long long& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  long long s = lane < THREADS / 32 ? sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  all = __shfl_sync(0xffffffffu, s, 31);
  const long long before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  __syncthreads();
  return v + (warp > 0 ? before : 0);
}

// What a row of a tree leaves for the rows after it: the bits of its own word
// that are above it (itself included) and the row before the word that the topmost
// of them continues, -1 for none.
struct TreeNode {
  uint32_t bits;
  int32_t up;
};

// A warp works out the 32 rows from 32 * w on of a sequence of n rows; first: the
// sequence's first packed row.
__device__ __forceinline__ TreeNode tree_word(const PlanParams& p, int32_t first, int32_t n, int32_t w) {
  const int lane = threadIdx.x & 31;
  const int32_t i = 32 * w + lane;
  int32_t up = -1;
  if (i < n) {
    const int32_t* a = p.parents + first + i;
    up = in_span(p.parents_span, a, 4, p.err) ? *a : -1;
    if (up >= i) {
      record_error(p.err, kErrBounds);
      up = -1;
    }
    up = max(up, -1);
  }
  int jump = up >= 32 * w ? up - 32 * w : -1;  // a lane before this one
  uint32_t bits = 1u << lane;
#pragma unroll
  for (int s = 0; s < 5; ++s) {
    const int from = max(jump, 0);
    const uint32_t more = __shfl_sync(0xffffffffu, bits, from);
    const int next = __shfl_sync(0xffffffffu, jump, from);
    if (jump >= 0) {
      bits |= more;
      jump = next;
    }
  }
  const int32_t out = up >= 32 * w ? -1 : up;
  return TreeNode{bits, __shfl_sync(0xffffffffu, out, __ffs(bits) - 1)};
}

// The mask of a row and its depth; nodes: of the sequence's rows, w the row's word.
__device__ __forceinline__ int32_t write_mask(const PlanParams& p, int64_t row, const TreeNode* nodes, TreeNode x, int32_t w) {
  uint32_t* out = p.masks + row * p.mask_words;
  int32_t depth = -1;
  const bool wide = (p.mask_words & 3) == 0 && (reinterpret_cast<uintptr_t>(p.masks) & 15) == 0;
  for (int32_t k = p.mask_words - 1; k >= 0;) {
    uint32_t v[4];
    const int32_t take = wide ? 4 : 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e >= take) break;
      v[e] = 0;
      if (k - e == w) {
        v[e] = x.bits;
        depth += __popc(x.bits);
        if (x.up >= 0) {
          w = x.up >> 5;
          x = nodes[x.up];
        } else {
          w = -1;
        }
      }
    }
    uint32_t* a = out + k - (take - 1);
    if (in_span(p.masks_span, a, 4 * take, p.err)) {
      if (wide) *reinterpret_cast<uint4*>(a) = make_uint4(v[3], v[2], v[1], v[0]);
      else *a = v[0];
    }
    k -= take;
  }
  return depth;
}

__device__ __forceinline__ void clear_mask(const PlanParams& p, int64_t row) {
  for (int32_t k = 0; k < p.mask_words; ++k)
    if (in_span(p.masks_span, p.masks + row * p.mask_words + k, 4, p.err)) p.masks[row * p.mask_words + k] = 0;
}

// Slot and position of row i of sequence b, and the table's entry where it opens a page.
__device__ __forceinline__ void write_row(const PlanParams& p, const PlanSeq& s, int32_t b, int32_t i, int32_t depth) {
  const PoolView& c = p.pool;
  const int64_t at = (int64_t)s.old + i, pg = at >> c.page_shift, have = pages_of(c, s.old);
  const int64_t row = (int64_t)s.row0 + i;
  const int32_t in_page = (int32_t)(at & (c.page_size - 1));
  int32_t id = -1;
  if (pg < c.max_pages) {
    int32_t* entry = c.table + (int64_t)b * c.table_stride + pg;
    if (pg < have) {
      id = *entry;
    } else {
      if (s.top >= 0) id = c.free_pages[max(s.top - (int32_t)(pg - have), 0)];
      if (in_page == 0) *entry = id;
    }
    if ((uint32_t)id >= (uint32_t)c.num_pages) {
      if (pg < have || s.top >= 0) record_error(p.err, kErrBounds);
      id = -1;
    }
  }
  if (in_span(p.slots_span, p.slots + row, 8, p.err))
    p.slots[row] = id < 0 ? -1 : ((int64_t)id << c.page_shift) + in_page;
  if (in_span(p.positions_span, p.positions + row, 4, p.err))
    p.positions[row] = (int32_t)min((int64_t)s.old + (p.parents != nullptr ? depth : i), (int64_t)INT32_MAX);
}

// A row behind the last sequence's.
__device__ __forceinline__ void write_padding(const PlanParams& p, int64_t row) {
  if (in_span(p.slots_span, p.slots + row, 8, p.err)) p.slots[row] = -1;
  if (in_span(p.positions_span, p.positions + row, 4, p.err)) p.positions[row] = 0;
  if (p.parents != nullptr) clear_mask(p, row);
}

// The rows of one word of a tree; nodes: of the sequence.
__device__ __forceinline__ void write_tree_rows(const PlanParams& p, const PlanSeq& s, int32_t b, int32_t w, const TreeNode* nodes,
                                                int32_t n) {
  const int32_t i = 32 * w + (threadIdx.x & 31);
  if (i >= s.n) return;
  int32_t depth = 0;
  if (i < n) depth = write_mask(p, (int64_t)s.row0 + i, nodes, nodes[i], w);
  else clear_mask(p, (int64_t)s.row0 + i);
  write_row(p, s, b, i, depth);
}

// The last entry of first[0 .. n) (non-decreasing) that is at most x.
template <class F>
__device__ __forceinline__ int32_t last_at_most(int32_t n, int64_t x, F first) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (first(mid) <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ plan

// Sums up; with `small`, which needs a batch of at most THREADS and no trees, does the
// rows as well.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) varlen_plan_kernel(const __grid_constant__ PlanParams p, int small) {
  __shared__ long long sums[32];
  __shared__ PlanSeq seqs[THREADS];
  dependency_wait();
  const PoolView& c = p.pool;
  const int32_t count = pool_free(c);
  long long rows = 0, need_before = 0;
  int32_t used = 0;  // pages that this thread's sequences bring the hand-out to
  for (int32_t base = 0; base < p.batch; base += THREADS) {
    const int32_t b = base + threadIdx.x;
    const bool live = b < p.batch;
    const int32_t old = live ? pool_len(c, b) : 0;
    long long all;
    const long long want_rows = live ? max(p.new_lens[b], 0) : 0;
    const long long end = rows + block_inclusive<THREADS>(want_rows, sums, all);
    rows += all;
    const int32_t r0 = (int32_t)min(end - want_rows, (long long)p.total), r1 = (int32_t)min(end, (long long)p.total);
    const int32_t n = r1 - r0;
    const int64_t have = pages_of(c, old), want = pages_of(c, (int64_t)old + n);
    const bool fits = want <= c.max_pages;
    const int64_t need = fits ? want - have : 0;
    const long long upto = need_before + block_inclusive<THREADS>(need, sums, all);
    need_before += all;
    const bool given = fits && (need == 0 || upto <= count);
    if (given && need > 0) used = max(used, (int32_t)upto);
    const PlanSeq s{old, r0, n, given ? (int32_t)(count - 1 - (upto - need)) : -1};
    if (live) {
      p.cu[b] = r0;
      if (b + 1 == p.batch) p.cu[p.batch] = r1;
      c.seqlens_out[b] = (int32_t)min((int64_t)old + n, (int64_t)INT32_MAX);
      // (a sequence that needs no page has all its rows in pages of its own)
      p.unplaced[b] = given ? 0 : (int32_t)max((int64_t)old + n - max((int64_t)old, have << c.page_shift), (int64_t)0);
      if (small) seqs[b] = s;
      else p.seqs[b] = s;
      if (p.parents != nullptr && n > 32 * p.mask_words) record_error(p.err, kErrBounds);
    }
  }
  dependents_may_launch();
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) used = max(used, __shfl_xor_sync(0xffffffffu, used, o));
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = used;
  __syncthreads();
  if (threadIdx.x < 32) {
    used = threadIdx.x < THREADS / 32 ? (int32_t)sums[threadIdx.x] : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) used = max(used, __shfl_xor_sync(0xffffffffu, used, o));
    if (threadIdx.x == 0) *c.free_count_out = count - used;
  }
  if (!small) return;
  const int32_t last = (int32_t)min(rows, (long long)p.total);
  for (int32_t row = threadIdx.x; row < last; row += THREADS) {
    const int32_t b = last_at_most(p.batch, row, [&](int32_t i) { return seqs[i].row0; });
    write_row(p, seqs[b], b, row - seqs[b].row0, 0);
  }
  for (int32_t row = last + threadIdx.x; row < p.total; row += THREADS) write_padding(p, row);
}

// A thread a row, without trees.
__global__ void __launch_bounds__(kRowThreads) varlen_plan_rows_kernel(const __grid_constant__ PlanParams p) {
  dependency_wait();
  dependents_may_launch();
  for (int64_t row = (int64_t)blockIdx.x * kRowThreads + threadIdx.x; row < p.total; row += (int64_t)gridDim.x * kRowThreads) {
    const int32_t b = last_at_most(p.batch, row, [&](int32_t i) { return p.seqs[i].row0; });
    const PlanSeq s = p.seqs[b];
    if (row - s.row0 < s.n) write_row(p, s, b, (int32_t)(row - s.row0), 0);
    else write_padding(p, row);
  }
}

// A row of CTAs a sequence, with trees: each works out all words' nodes in shared
// memory and writes its share of the rows.  The rows behind the last sequence's are
// shared out among all.
__global__ void __launch_bounds__(kRowThreads) varlen_plan_trees_kernel(const __grid_constant__ PlanParams p) {
  extern __shared__ TreeNode nodes[];
  dependency_wait();
  dependents_may_launch();
  const int32_t b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const PlanSeq s = p.seqs[b];
  const int32_t n = min(s.n, 32 * p.mask_words);
  for (int32_t w = warp; w < (n + 31) / 32; w += kRowThreads / 32) {
    const TreeNode x = tree_word(p, s.row0, n, w);
    if (32 * w + lane < n) nodes[32 * w + lane] = x;
  }
  __syncthreads();
  for (int32_t w = blockIdx.y * (kRowThreads / 32) + warp; w < (s.n + 31) / 32; w += gridDim.y * (kRowThreads / 32))
    write_tree_rows(p, s, b, w, nodes, n);
  const PlanSeq e = p.seqs[p.batch - 1];
  const int64_t cta = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, ctas = (int64_t)gridDim.x * gridDim.y;
  for (int64_t row = e.row0 + (int64_t)e.n + cta * kRowThreads + threadIdx.x; row < p.total; row += ctas * kRowThreads)
    write_padding(p, row);
}

// ------------------------------------------------------------------ trim

// One CTA: the pages that come back, from the last sequence's last to the first's
// first, form a list; entries that name a page are numbered and go onto the stack.
// Made for the few pages that come back behind a step (3.7 us for 256 sequences of 4 pages); many
// are taken THREADS at a time, a dependent load and two barriers each: 64 sequences of 64 pages
// 15 us, 256 of 512 184 us.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) varlen_trim_kernel(const __grid_constant__ TrimParams p) {
  __shared__ long long sums[32];
  __shared__ int32_t first[THREADS], have[THREADS];  // place in the list; pages before the call
  dependency_wait();
  dependents_may_launch();
  const PoolView& c = p.pool;
  const int32_t count = pool_free(c);
  long long pushed = 0;
  for (int32_t base = 0; base < p.batch; base += THREADS) {
    const int32_t b = p.batch - 1 - base - (int32_t)threadIdx.x;
    const bool live = b >= 0;
    int64_t held = 0, keep = 0;
    if (live) {
      const int32_t old = pool_len(c, b);
      int64_t left = p.lens[b];
      if (p.cu != nullptr) left = (int64_t)max(c.seqlens[b], 0) - max((int64_t)p.cu[b + 1] - p.cu[b], (int64_t)0) + max(left, (int64_t)0);
      left = min(max(left, (int64_t)0), (int64_t)old);
      held = pages_of(c, old);
      keep = pages_of(c, left);
      c.seqlens_out[b] = (int32_t)left;
    }
    long long all;
    const long long end = block_inclusive<THREADS>(held - keep, sums, all);
    first[threadIdx.x] = (int32_t)(end - (held - keep));  // (batch * max_pages < 2^31)
    have[threadIdx.x] = (int32_t)held;
    __syncthreads();
    const int32_t live_n = min(p.batch - base, THREADS);
    for (long long f0 = 0; f0 < all; f0 += THREADS) {  // CTA-uniform
      const long long f = f0 + threadIdx.x;
      int32_t id = -1;
      if (f < all) {
        const int32_t k = last_at_most(live_n, f, [&](int32_t i) { return first[i]; });
        const int32_t entry = have[k] - 1 - (int32_t)(f - first[k]);
        id = c.table[(int64_t)(p.batch - 1 - base - k) * c.table_stride + entry];
        if (id < -1 || id >= c.num_pages) {
          record_error(p.err, kErrBounds);
          id = -1;
        }
      }
      long long kept;
      const long long rank = block_inclusive<THREADS>(id >= 0 ? 1 : 0, sums, kept) - 1;
      if (id >= 0) {
        const long long to = count + pushed + rank;
        if (to < c.num_pages) {
          if (in_span(p.free_span, c.free_pages + to, 4, p.err)) c.free_pages[to] = id;
        } else {
          record_error(p.err, kErrBounds);
        }
      }
      pushed += kept;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *c.free_count_out = (int32_t)min(count + pushed, (long long)c.num_pages);
}

// ------------------------------------------------------------------ move

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;      // accepted rows looked up at once
constexpr int kMoveLoads = 8;      // pieces of 16 bytes that a thread holds at once
constexpr int kMovePieces = 1024;  // of a CTA

// Moves pieces t, t + kMoveThreads, ... (GROUPS of them at once) of the listed rows.
// A thread takes a piece through all rows in order, kMoveLoads / GROUPS rows loaded
// before any is stored: the place of row i lies at or before its source, so what a
// thread has still to read it has not yet overwritten, and no other thread touches it.
template <bool E4M3, int GROUPS>
__device__ __forceinline__ void move_pieces(const MoveParams& p, const MoveLayer& layer, int32_t t, int32_t end,
                                            int32_t rows, const int2* from, const int2* to) {
  constexpr int ROWS = kMoveLoads / GROUPS;
  const int32_t chunks = p.row_bytes / 16, items = 2 * chunks + (E4M3 ? 2 : 0);  // pieces of a head's rows
  for (; t < end; t += GROUPS * kMoveThreads) {
    uint8_t* base[GROUPS];
    int64_t ps[GROUPS], rs[GROUPS];  // byte strides of pages and rows
    Span s[GROUPS];
    bool scale[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int32_t at = min(t + g * kMoveThreads, end - 1), h = at / items, item = at - h * items;
      scale[g] = E4M3 && item >= 2 * chunks;
      const bool is_v = scale[g] ? item > 2 * chunks : item >= chunks;
      if (scale[g]) {
        uint8_t* a = reinterpret_cast<uint8_t*>(is_v ? layer.v_scale : layer.k_scale);
        s[g] = Span{a, p.s_bytes};
        base[g] = a + ((int64_t)h << (p.pages.page_shift + 1));
        ps[g] = (int64_t)p.heads << (p.pages.page_shift + 1);
        rs[g] = 2;
      } else {
        uint8_t* a = is_v ? layer.v : layer.k;
        s[g] = Span{a, is_v ? p.vp_bytes : p.kp_bytes};
        base[g] = a + h * (is_v ? p.v_head : p.k_head) + (item - (is_v ? chunks : 0)) * 16;
        ps[g] = is_v ? p.v_page : p.k_page;
        rs[g] = is_v ? p.v_row : p.k_row;
      }
    }
    for (int32_t j0 = 0; j0 < rows; j0 += ROWS) {
      uint4 x[GROUPS][ROWS];
#pragma unroll
      for (int e = 0; e < ROWS; ++e) {
        const int2 f = from[min(j0 + e, rows - 1)];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          const uint8_t* a = base[g] + f.x * ps[g] + f.y * rs[g];
          x[g][e] = make_uint4(0, 0, 0, 0);
          if (scale[g]) {
            if (in_span(s[g], a, 2, p.err)) x[g][e].x = *reinterpret_cast<const unsigned short*>(a);
          } else {
            if (in_span(s[g], a, 16, p.err)) x[g][e] = *reinterpret_cast<const uint4*>(a);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < ROWS; ++e) {
        if (j0 + e >= rows) break;
        const int2 f = to[j0 + e];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
          if (t + g * kMoveThreads >= end) break;
          uint8_t* a = base[g] + f.x * ps[g] + f.y * rs[g];
          if (scale[g]) {
            if (in_span(s[g], a, 2, p.err)) *reinterpret_cast<unsigned short*>(a) = (unsigned short)x[g][e].x;
          } else {
            if (in_span(s[g], a, 16, p.err)) *reinterpret_cast<uint4*>(a) = x[g][e];
          }
        }
      }
    }
  }
}

// A CTA takes some of the pieces (16 bytes of a head's row of K or V, or its scale) of
// one sequence's rows in one layer.  It looks up 32 accepted rows at a time and lists
// those that do not stay.  Bound by the memory where there is much to move: 732 rows of
// 56 heads of 128 in four bf16 layers, 168 MB, 31 us, 5.4 TB/s (a piece a thread 38.8;
// 512 or 2048 pieces a CTA 34); else by four dependent loads: 214 rows of 8 E4M3 heads 3.6 us.
template <bool E4M3>
__global__ void __launch_bounds__(kMoveThreads) varlen_move_kernel(const __grid_constant__ MoveParams p) {
  __shared__ int2 from_at[kMoveRows], to_at[kMoveRows];  // (page, row in it)
  __shared__ int32_t listed;
  dependency_wait();
  dependents_may_launch();
  const int32_t b = blockIdx.x;
  const MoveLayer& layer = p.layer[blockIdx.z];
  // (an accepted row is read before it is known to be one: it lies within kept's rows)
  int32_t k = threadIdx.x < min(kMoveRows, p.max_kept) ? p.kept[(int64_t)b * p.kept_stride + threadIdx.x] : 0;
  const int32_t r0 = clamp_row(p.cu[b], p.total), n = max(clamp_row(p.cu[b + 1], p.total) - r0, 0);
  const int32_t kept = min(max(p.kept_lens[b], 0), p.max_kept);
  const int64_t start = (int64_t)max(p.pages.seqlens[b], 0) - n;  // position of new row 0
  const int32_t all = p.heads * (2 * (p.row_bytes / 16) + (E4M3 ? 2 : 0));  // (heads are bounded: no overflow)
  auto place = [&](int32_t i, int32_t& page, int32_t& row) {  // of new row i, or no page
    const int64_t at = start + i;
    page = p.pages.num_pages;
    row = (int32_t)(at & (p.pages.page_size - 1));
    if (at < 0 || (at >> p.pages.page_shift) >= p.pages.max_pages) return;  // (the plan found it no place)
    page = page_at<true>(p.pages, b, (int32_t)(at >> p.pages.page_shift), p.err);
  };
  for (int32_t i0 = 0; i0 < kept; i0 += kMoveRows) {  // CTA-uniform
    if (threadIdx.x < 32) {
      const int32_t i = i0 + threadIdx.x;
      if (i0 > 0 && i < kept) k = p.kept[(int64_t)b * p.kept_stride + i];
      int32_t from = p.pages.num_pages, to = from, rf = 0, rt = 0;
      if (i < kept) {
        if (k < i || k >= n) {
          record_error(p.err, kErrBounds);
        } else if (k != i) {
          place(k, from, rf);
          place(i, to, rt);
        }
      }
      const bool moves = from < p.pages.num_pages && to < p.pages.num_pages;
      const unsigned who = __ballot_sync(0xffffffffu, moves);
      if (moves) {
        const int at = __popc(who & ((1u << threadIdx.x) - 1u));
        from_at[at] = make_int2(from, rf);
        to_at[at] = make_int2(to, rt);
      }
      if (threadIdx.x == 0) listed = __popc(who);
    }
    __syncthreads();
    const int32_t rows = listed;
    for (int32_t w = blockIdx.y * kMovePieces; w < all && rows > 0; w += gridDim.y * kMovePieces) {
      const int32_t t = w + (int32_t)threadIdx.x, end = min(w + kMovePieces, all);
      if (rows <= 2) move_pieces<E4M3, 4>(p, layer, t, end, rows, from_at, to_at);
      else if (rows <= 4) move_pieces<E4M3, 2>(p, layer, t, end, rows, from_at, to_at);
      else move_pieces<E4M3, 1>(p, layer, t, end, rows, from_at, to_at);
    }
    __syncthreads();  // the lists are read
  }
}

}  // namespace

cudaError_t launch_plan(const PlanParams& p, cudaStream_t stream) {
  const bool small = p.batch <= kPlanThreads && p.total <= kPlanSmall && p.parents == nullptr;
  const bool few = p.batch <= kPlanFew && (!small || p.total <= kPlanFew);
  const cudaError_t e = few ? launch_overlapped(varlen_plan_kernel<kPlanFew>, dim3(1), kPlanFew, 0, stream, p, small ? 1 : 0)
                            : launch_overlapped(varlen_plan_kernel<kPlanThreads>, dim3(1), kPlanThreads, 0, stream, p, small ? 1 : 0);
  if (e != cudaSuccess || small || p.total == 0) return e;
  if (p.parents == nullptr) {
    const int64_t blocks = ((int64_t)p.total + kRowThreads - 1) / kRowThreads;
    return launch_overlapped(varlen_plan_rows_kernel, dim3((unsigned)std::min<int64_t>(blocks, 1 << 20)), kRowThreads, 0, stream, p);
  }
  const int32_t cap = std::min(p.total, 32 * p.mask_words);  // rows of a sequence that have nodes
  const int64_t share = ((int64_t)p.total / p.batch + kRowThreads - 1) / kRowThreads;
  const unsigned y = (unsigned)std::min<int64_t>(std::max<int64_t>(share, 1), 64);
  return launch_overlapped(varlen_plan_trees_kernel, dim3((unsigned)p.batch, y), kRowThreads, cap * sizeof(TreeNode), stream, p);
}

cudaError_t launch_trim(const TrimParams& p, cudaStream_t stream) {
  // (a few pages come back from each sequence)
  return p.batch <= kPlanFew / 4 ? launch_overlapped(varlen_trim_kernel<kPlanFew>, dim3(1), kPlanFew, 0, stream, p)
                                 : launch_overlapped(varlen_trim_kernel<kPlanThreads>, dim3(1), kPlanThreads, 0, stream, p);
}

cudaError_t launch_move(const MoveLaunch& L, cudaStream_t stream) {
  const int64_t items = (int64_t)L.p.heads * (2 * (L.p.row_bytes / 16) + (L.e4m3 ? 2 : 0));
  const dim3 grid((unsigned)L.p.batch, (unsigned)std::min<int64_t>((items + kMovePieces - 1) / kMovePieces, 65535), (unsigned)L.layers);
  return L.e4m3 ? launch_overlapped(varlen_move_kernel<true>, grid, kMoveThreads, 0, stream, L.p)
                : launch_overlapped(varlen_move_kernel<false>, grid, kMoveThreads, 0, stream, L.p);
}

}  // namespace varlen
