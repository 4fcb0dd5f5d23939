// varlen_paged_walk.cuh -- how the paged attention kernels share out their
// work.
//
// A unit is one block of rows of one (segment, key head); a row is one (query
// token, query head of the key head's group), token-major: row r is token r /
// group, head r % group.  A unit works through the key tiles that some of its
// rows see.  The units of a launch in a fixed order (segment, key head, row
// block), each with its tiles (at least one, so that a unit without keys is
// visited and writes its zeros), form one long list of T places, and each of N
// CTAs takes T / N neighbouring ones of it (the first T % N one more): the tiles
// whose first place these are.  A tile has one place, so that every CTA has the same
// number of them, whatever the lengths; with trees, whose units are many and short, more, by
// what it costs, and so has the end of a unit.  A CTA's part starts and ends inside a unit
// in general; what it has of a unit that it does not hold whole goes to the
// workspace as a partial result (its running maximum, sum and unnormalised
// output), in one of two slots: 1 for the unit that it begins and a later CTA
// ends, 0 for one that an earlier CTA began.  varlen_paged_join_kernel adds the
// partial results of a unit in the order of the CTAs.
//
// The lengths are device data: each CTA sums the costs itself (one segment
// per thread) and finds where its part begins.
#pragma once

#include "sm103_ptx.cuh"
#include "varlen_paged.h"

namespace varlen {

struct PagedSeg {
  int32_t q0, n, sk;   // first packed query row, queries, keys (TREE: positions)
  int32_t blocks;      // row blocks
  int64_t per_head;    // places of all row blocks of one key head
};

struct PagedUnit {
  int32_t t0, t1;        // first and last query token (within the segment)
  int32_t lo, hi;        // keys that some row of the unit sees
  int32_t tile0, tiles;  // first key tile and number of key tiles
};

// n / d: 64-bit division is a long subroutine, and hardly ever needed here.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (((uint64_t)n | (uint64_t)d) >> 32 == 0) return (int64_t)((uint32_t)n / (uint32_t)d);
  return n / d;
}

// CTAs that share `total` places: no more than leave each `least`.
__device__ __forceinline__ int32_t paged_ctas(int64_t total, int32_t grid, int32_t least) {
  const int64_t n = quotient(total + least - 1, least);
  return (int32_t)(n < 1 ? 1 : (n < grid ? n : grid));
}

// Geometry of a kernel's units: ROWS rows per block, or, with BY_TOKEN, the
// rows of two halves of whole tokens (ROWS / 2 / group tokens each); TILE keys
// per tile.  TREE: the keys are those from where a row at the context's end would
// begin to see them to the last new row, whichever of them the masks name; sk counts a
// sequence's positions, its new rows last, although its table may name fewer.
template <int ROWS, int TILE, bool BY_TOKEN, bool TREE>
struct PagedGeom {
  __device__ static __forceinline__ int32_t half_tokens(const PagedParams& p) { return ROWS / 2 / p.group; }
  __device__ static __forceinline__ int32_t blocks(const PagedParams& p, int32_t n) {
    const uint32_t rows = BY_TOKEN ? n : n * p.group, per = BY_TOKEN ? 2 * half_tokens(p) : ROWS;
    return (int32_t)((rows + per - 1) / per);
  }
  __device__ static __forceinline__ PagedUnit unit(const PagedParams& p, int32_t n, int32_t sk, int32_t blk) {
    PagedUnit u;
    if (BY_TOKEN) {
      const int32_t bt = 2 * half_tokens(p);
      u.t0 = blk * bt;
      u.t1 = min(n - u.t0, bt) + u.t0 - 1;
    } else {
      const uint32_t r0 = (uint32_t)blk * ROWS, r1 = min((uint32_t)(n * p.group), r0 + ROWS) - 1;
      u.t0 = (int32_t)(r0 / (uint32_t)p.group);
      u.t1 = (int32_t)(r1 / (uint32_t)p.group);
    }
    if (TREE) {
      band_keys(0, 0, n, sk, p.win_left, kWinUnbounded, &u.lo, &u.hi);
      u.hi = min(u.hi, p.pages.max_pages << p.pages.page_shift);  // (below 2^31)
    } else band_keys(u.t0, u.t1, n, sk, p.win_left, p.win_right, &u.lo, &u.hi);
    u.tile0 = u.lo / TILE;
    u.tiles = u.hi > u.lo ? (u.hi - 1) / TILE + 1 - u.tile0 : 0;
    return u;
  }
  // Places that a tile and a unit take in the list: one a tile or, with trees, what they
  // cost: a tile of two halves 5, of one 4 (2.4 and 1.9 us in E4M3, 2.1 and 1.75 in bf16), a
  // unit's start and end two such tiles; in the kernel for few rows 1 and 3.  For 64 trees
  // of 16..64 rows, 4 heads a key head, over 1..8192 keys, us, tiles alone, tiles and ends, all
  // three: E4M3 350, 326, 320, bf16 270, 248, 235; trees of 33..64 336, 301, 300 and 260, 226, 227; of
  // 1..4 140, 130 and 160, 152.
  static constexpr bool kTree = TREE;
  static constexpr int32_t kTilePlaces = TREE && BY_TOKEN ? 5 : 1, kHalfPlaces = TREE && BY_TOKEN ? 4 : 1,
                           kEndPlaces = TREE ? (BY_TOKEN ? 10 : 3) : 0;
  __device__ static __forceinline__ int32_t per_tile(const PagedParams& p, const PagedUnit& u) {
    return kHalfPlaces != kTilePlaces && u.t1 - u.t0 < half_tokens(p) ? kHalfPlaces : kTilePlaces;
  }
  __device__ static __forceinline__ int32_t weight(const PagedParams& p, const PagedUnit& u) {
    return max(u.tiles, 1) * per_tile(p, u) + kEndPlaces;
  }
  // CTAs that share a list of `total` places: no more than leave each `least` tiles.
  __device__ static __forceinline__ int32_t ctas(int64_t total, int32_t grid, int32_t least) {
    // (with trees no part is shorter than that: each then holds the first place of some tile of
    // a unit that goes on before and behind it, as the join takes for granted)
    return paged_ctas(TREE ? max(total - (kTilePlaces * least - 1), (int64_t)1) : total, grid, kTilePlaces * least);
  }
};

template <class G>
__device__ __forceinline__ PagedSeg paged_seg(const PagedParams& p, int32_t b, int32_t take) {
  PagedSeg s;
  const int32_t a = clamp_row(p.cu_q[b], p.total_q), e = clamp_row(p.cu_q[b + 1], p.total_q);
  s.q0 = a;
  s.n = max(e - a, 0);
  s.sk = G::kTree ? max(p.pages.seqlens[b], 0) : cache_len(p.pages, b);
  const bool few = s.n * p.group <= kFewRows;  // (total_q * num_heads < 2^31)
  if ((take == kTakeFew && !few) || (take == kTakeMany && few)) s.n = 0;
  s.blocks = G::blocks(p, s.n);
  s.per_head = 0;
  for (int32_t i = 0; i < s.blocks; ++i) s.per_head += G::weight(p, G::unit(p, s.n, s.sk, i));
  return s;
}

// One CTA's part of a unit: tiles [j0, j1) of the unit's list (which has
// `cost` of them, at least one).
struct PagedPiece {
  PagedUnit u;
  int32_t b, kh, blk;
  int32_t q0, n, sk;
  int32_t j0, j1, cost;
  __device__ __forceinline__ bool begins() const { return j0 == 0; }
  __device__ __forceinline__ bool ends() const { return j1 == cost; }
  __device__ __forceinline__ bool whole() const { return begins() && ends(); }
};

// Where a CTA's part begins, shared by its threads.
struct PagedStart {
  int64_t total, first, count;  // places of the launch; first and number of this CTA's
  int64_t off;                  // the first one's place within segment b
  int32_t b, ctas;              // segment; CTAs that have work
  PagedSeg seg;                 // of segment b
  long long sums[16];
};

// First place of CTA c: the parts have total / ctas places, the first total %
// ctas of them one more.
struct PagedShares {
  int64_t each, more;
  __device__ __forceinline__ PagedShares(int64_t total, int32_t ctas) {
    each = quotient(total, ctas);
    more = total - each * ctas;
  }
  __device__ __forceinline__ int64_t first(int32_t c) const { return each * c + min((int64_t)c, more); }
  __device__ __forceinline__ int32_t owner(int64_t x) const {
    const int64_t big = more * (each + 1);
    return (int32_t)(x < big ? quotient(x, each + 1) : more + quotient(x - big, each));
  }
};

__device__ __forceinline__ long long warp_inclusive(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += t;
  }
  return v;
}

// Fills `st` (shared memory).  Every thread of the CTA (a whole number of
// warps, at most 16) calls it; the CTA is synchronised when it returns.
template <class G>
__device__ __forceinline__ void paged_start(PagedStart& st, const PagedParams& p, int32_t take, int32_t least) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  // batches of at most a thread's segment each are scanned once; larger ones
  // are summed first and then searched
  const bool one = p.batch <= (int32_t)blockDim.x;
  PagedSeg seg;
  seg.per_head = 0;
  long long mine = 0;
  for (int32_t b = threadIdx.x; b < p.batch; b += blockDim.x) {
    seg = paged_seg<G>(p, b, take);
    mine += (long long)p.kv_heads * seg.per_head;
  }
  long long incl = warp_inclusive(mine);
  if (lane == 31) st.sums[warp] = incl;
  if (threadIdx.x == 0) st.b = st.off = 0;
  __syncthreads();
  long long total = 0, excl = incl - mine;
  for (int w = 0; w < warps; ++w) {
    if (w < warp) excl += st.sums[w];
    total += st.sums[w];
  }
  const int32_t ctas = G::ctas(total, gridDim.x, least);
  const bool works = total > 0 && (int32_t)blockIdx.x < ctas;
  const PagedShares shares(total, ctas);
  const int64_t first = works ? shares.first(blockIdx.x) : 0;
  if (threadIdx.x == 0) {
    st.total = total;
    st.ctas = ctas;
    st.first = first;
    st.count = works ? shares.first(blockIdx.x + 1) - first : 0;
  }
  if (one || !works) {  // CTA-uniform
    if (works && first >= excl && first < excl + mine) {
      st.b = threadIdx.x;
      st.off = first - excl;
      st.seg = seg;
    }
    __syncthreads();
    return;
  }
  __syncthreads();
  long long before = 0;
  for (int32_t base = 0; base < p.batch; base += blockDim.x) {
    const int32_t b = base + threadIdx.x;
    long long c = 0;
    if (b < p.batch) {
      seg = paged_seg<G>(p, b, take);
      c = (long long)p.kv_heads * seg.per_head;
    }
    incl = warp_inclusive(c);
    if (lane == 31) st.sums[warp] = incl;
    __syncthreads();
    long long e = before + incl - c, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) e += st.sums[w];
      all += st.sums[w];
    }
    if (first >= e && first < e + c) {
      st.b = b;
      st.off = first - e;
      st.seg = seg;
    }
    before += all;
    __syncthreads();
    if (before > first) break;  // CTA-uniform
  }
}

// Walks a CTA's part piece by piece.  Every role of the CTA runs its own.
template <class G>
struct PagedWalk {
  PagedSeg s;
  int32_t b, kh, blk, at, take;  // at: the part's place within its next unit
  int64_t left;                  // its places from there on
  __device__ __forceinline__ void init(const PagedStart& st, const PagedParams& p, int32_t take_) {
    take = take_;
    left = st.count;
    b = st.b;
    kh = blk = 0;
    at = 0;
    if (left <= 0) return;
    s = st.seg;
    int64_t off = st.off;
    kh = (int32_t)quotient(off, s.per_head);
    off -= (int64_t)kh * s.per_head;
    while (true) {
      const int32_t w = G::weight(p, G::unit(p, s.n, s.sk, blk));
      if (off < w) break;
      off -= w;
      ++blk;
    }
    at = (int32_t)off;
  }
  __device__ __forceinline__ bool next(const PagedParams& p, PagedPiece& x) {
    while (left > 0) {
      while (blk >= s.blocks) {
        blk = 0;
        if (s.blocks > 0 && kh + 1 < p.kv_heads) {
          ++kh;
          break;
        }
        if (++b >= p.batch) return false;
        s = paged_seg<G>(p, b, take);
        kh = 0;
      }
      x.u = G::unit(p, s.n, s.sk, blk);
      x.b = b;
      x.kh = kh;
      x.blk = blk;
      x.q0 = s.q0;
      x.n = s.n;
      x.sk = s.sk;
      x.cost = max(x.u.tiles, 1);
      // the tiles whose first place lies in the part
      const int32_t w = G::weight(p, x.u), per = G::per_tile(p, x.u), end = (int32_t)min((int64_t)w, at + left);
      x.j0 = min((at + per - 1) / per, x.cost);
      x.j1 = min((end + per - 1) / per, x.cost);
      left -= w - at;  // (0 or less: this is the last)
      at = 0;
      ++blk;
      if (x.j0 < x.j1) return true;
    }
    return false;
  }
};

// ------------------------------------------------- drafted trees
// ctx: position of a segment's new row 0 (its positions less its new rows; negative
// where rows are missing, past a table that is too short for them).  A row sees the keys
// [tree_lo, ctx) and those new rows j, key ctx + j, whose bit its mask has, where the table
// names them (below the unit's hi).
__device__ __forceinline__ int32_t tree_lo(const PagedParams& p, int64_t row, int32_t ctx) {
  if (p.win_left >= kWinUnbounded) return 0;
  const int32_t* a = p.tree_pos + row;
  const int64_t at = in_span(p.pos_span, a, 4, p.err) ? *a : 0;
  // (a row whose window begins behind the context sees none of it: ctx)
  return (int32_t)max(min(max(at, (int64_t)ctx) - p.win_left, (int64_t)ctx), (int64_t)0);
}

__device__ __forceinline__ uint32_t tree_word_at(const PagedParams& p, int64_t row, int32_t w) {
  const uint32_t* a = p.masks + row * p.mask_words + w;
  return (uint32_t)w < (uint32_t)p.mask_words && in_span(p.masks_span, a, 4, p.err) ? *a : 0u;
}

// Brings the first 512 bytes of a row's mask as far as L1 (a hint: nothing waits for it).
__device__ __forceinline__ void tree_prefetch(const PagedParams& p, int64_t row) {
  const uint32_t* a = p.masks + row * p.mask_words;
  for (int32_t w = 0; w < min(p.mask_words, 128); w += 32)
    if (in_span(p.masks_span, a + w, 4, p.err)) asm volatile("prefetch.global.L1 [%0];" ::"l"(a + w));
}

// 32 bits of a packed row's mask, from new row `rel` on; those before new row 0
// (the context's) are set.
__device__ __forceinline__ uint32_t tree_bits(const PagedParams& p, int64_t row, int32_t rel) {
  if (rel <= -32) return ~0u;
  if (rel < 0) return (tree_word_at(p, row, 0) << -rel) | ((1u << -rel) - 1u);
  const uint32_t lo = tree_word_at(p, row, rel >> 5);
  return (rel & 31) == 0 ? lo : __funnelshift_r(lo, tree_word_at(p, row, (rel >> 5) + 1), rel & 31);
}

// Bits [lo, hi) of a word.
__device__ __forceinline__ uint32_t bits_between(int32_t lo, int32_t hi) {
  const uint32_t below = hi >= 32 ? ~0u : (hi <= 0 ? 0u : (1u << hi) - 1u);
  return lo <= 0 ? below : (lo >= 32 ? 0u : below & ~((1u << lo) - 1u));
}

// A whole warp: the first key that some row of the unit sees of the context.
__device__ __forceinline__ int32_t tree_unit_lo(const PagedParams& p, const PagedPiece& x) {
  if (p.win_left >= kWinUnbounded) return x.u.lo;
  int32_t lo = INT32_MAX;
  for (int32_t t = x.u.t0 + (int32_t)(threadIdx.x & 31); t <= x.u.t1; t += 32) lo = min(lo, tree_lo(p, (int64_t)x.q0 + t, x.sk - x.n));
  return max(__reduce_min_sync(0xffffffffu, lo), x.u.lo);
}

// A whole warp: which of the 128 keys from key0 on some row of the unit sees.
__device__ __forceinline__ void tree_unit_bits(const PagedParams& p, const PagedPiece& x, int32_t unit_lo, int32_t key0, uint32_t (&any)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) any[k] = 0;
  for (int32_t t = x.u.t0 + (int32_t)(threadIdx.x & 31); t <= x.u.t1; t += 32)
#pragma unroll
    for (int k = 0; k < 4; ++k) any[k] |= tree_bits(p, (int64_t)x.q0 + t, key0 + 32 * k - (x.sk - x.n));
#pragma unroll
  for (int k = 0; k < 4; ++k)
    any[k] = __reduce_or_sync(0xffffffffu, any[k]) & bits_between(unit_lo - key0 - 32 * k, x.u.hi - key0 - 32 * k);
}

// 32 bytes in one store, to an address aligned to them.
__device__ __forceinline__ void store_sector(float* a, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
               "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// Entry i of the join's list.
__device__ __forceinline__ void put_join(const PagedParams& p, const PagedParts& parts, int32_t i, const PagedJoin& u) {
  if (in_span(parts.join_span, parts.join + i, sizeof(PagedJoin), p.err)) parts.join[i] = u;
}
__device__ __forceinline__ PagedJoin get_join(const PagedParams& p, const PagedParts& parts, int32_t i) {
  return in_span(parts.join_span, parts.join + i, sizeof(PagedJoin), p.err) ? parts.join[i] : PagedJoin{0, 0, 0, 0, 0};
}
// This CTA's entries, empty: no unit that the join would have to look at.
__device__ __forceinline__ void clear_join(const PagedParams& p, const PagedParts& parts) {
  put_join(p, parts, 2 * blockIdx.x, PagedJoin{0, 0, 0, 0, 0});
  put_join(p, parts, 2 * blockIdx.x + 1, PagedJoin{0, 0, 0, 0, 0});
}

// A CTA that cannot work: an error, and no unit for the join (which would take
// what the workspace happens to hold for one).
__device__ __forceinline__ void paged_refuse(const PagedParams& p, const PagedParts& parts) {
  dependency_wait();
  if (threadIdx.x != 0) return;
  clear_join(p, parts);
  record_error(p.err, kErrBounds);
}

// Left for the join by the one thread that calls it, for every piece: the
// units that the CTA holds a part of (its first and its last piece, if any).
template <class G>
__device__ __forceinline__ void paged_note(const PagedParams& p, const PagedParts& parts, const PagedStart& st,
                                           const PagedWalk<G>& walk, const PagedPiece& x) {
  if (x.whole()) return;
  const PagedShares shares(st.total, st.ctas);
  const int64_t begin = st.first + st.count - walk.left - G::weight(p, x.u);  // the unit's first place (walk stands behind it)
  const int32_t first = shares.owner(begin);
  put_join(p, parts, 2 * blockIdx.x + (x.begins() ? 1 : 0),
           PagedJoin{x.b, x.kh, x.blk, first, shares.owner(begin + (int64_t)(x.cost - 1) * G::per_tile(p, x.u)) - first + 1});
}

}  // namespace varlen
