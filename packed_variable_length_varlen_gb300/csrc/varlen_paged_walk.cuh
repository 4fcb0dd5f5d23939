// varlen_paged_walk.cuh -- how the paged attention kernels share out their
// work.
//
// A unit is one block of rows of one (segment, key head); a row is one (query
// token, query head of the key head's group), token-major: row r is token r /
// group, head r % group.  A unit works through the key tiles that some of its
// rows see.  The units of a launch in a fixed order (segment, key head, row
// block), each with its tiles (at least one, so that a unit without keys is
// visited and writes its zeros), form one long list of T tiles, and each of N
// CTAs takes T / N neighbouring ones of it (the first T % N one more): every CTA
// has the same number of tiles, whatever the lengths.  A CTA's part starts and ends inside a unit
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
  int32_t q0, n, sk;   // first packed query row, queries, keys
  int32_t blocks;      // row blocks
  int64_t per_head;    // tiles of all row blocks of one key head
};

struct PagedUnit {
  int32_t t0, t1;        // first and last query token (within the segment)
  int32_t lo, hi;        // keys that some row of the unit sees
  int32_t tile0, tiles;  // first key tile and number of key tiles
};

// Geometry of a kernel's units: ROWS rows per block, or, with BY_TOKEN, the
// rows of two halves of whole tokens (ROWS / 2 / group tokens each); TILE keys
// per tile.
template <int ROWS, int TILE, bool BY_TOKEN>
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
    band_keys(u.t0, u.t1, n, sk, p.win_left, p.win_right, &u.lo, &u.hi);
    u.tile0 = u.lo / TILE;
    u.tiles = u.hi > u.lo ? (u.hi - 1) / TILE + 1 - u.tile0 : 0;
    return u;
  }
};

template <class G>
__device__ __forceinline__ PagedSeg paged_seg(const PagedParams& p, int32_t b, int32_t take) {
  PagedSeg s;
  const int32_t a = clamp_row(p.cu_q[b], p.total_q), e = clamp_row(p.cu_q[b + 1], p.total_q);
  s.q0 = a;
  s.n = max(e - a, 0);
  s.sk = cache_len(p.pages, b);
  const bool few = s.n * p.group <= kFewRows;  // (total_q * num_heads < 2^31)
  if ((take == kTakeFew && !few) || (take == kTakeMany && few)) s.n = 0;
  s.blocks = G::blocks(p, s.n);
  s.per_head = 0;
  for (int32_t i = 0; i < s.blocks; ++i) s.per_head += max(G::unit(p, s.n, s.sk, i).tiles, 1);
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
  int64_t total, first, count;  // tiles of the launch; first tile and number of tiles of this CTA
  int64_t off;                  // first tile's place within segment b
  int32_t b, ctas;              // segment; CTAs that have work
  PagedSeg seg;                 // of segment b
  long long sums[16];
};

// n / d: 64-bit division is a long subroutine, and hardly ever needed here.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (((uint64_t)n | (uint64_t)d) >> 32 == 0) return (int64_t)((uint32_t)n / (uint32_t)d);
  return n / d;
}

// CTAs that share `total` tiles: no more than leave each `least`.
__device__ __forceinline__ int32_t paged_ctas(int64_t total, int32_t grid, int32_t least) {
  const int64_t n = quotient(total + least - 1, least);
  return (int32_t)(n < 1 ? 1 : (n < grid ? n : grid));
}
// First tile of CTA c: the parts have total / ctas tiles, the first total %
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
  const int32_t ctas = paged_ctas(total, gridDim.x, least);
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
  int32_t b, kh, blk, j, take;
  int64_t left;
  __device__ __forceinline__ void init(const PagedStart& st, const PagedParams& p, int32_t take_) {
    take = take_;
    left = st.count;
    b = st.b;
    kh = blk = j = 0;
    if (left <= 0) return;
    s = st.seg;
    int64_t off = st.off;
    kh = (int32_t)quotient(off, s.per_head);
    off -= (int64_t)kh * s.per_head;
    while (true) {
      const int32_t c = max(G::unit(p, s.n, s.sk, blk).tiles, 1);
      if (off < c) break;
      off -= c;
      ++blk;
    }
    j = (int32_t)off;
  }
  __device__ __forceinline__ bool next(const PagedParams& p, PagedPiece& x) {
    if (left <= 0) return false;
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
    x.j0 = j;
    x.j1 = (int32_t)min((int64_t)x.cost, j + left);
    left -= x.j1 - x.j0;
    if (x.j1 == x.cost) {
      ++blk;
      j = 0;
    } else {
      j = x.j1;
    }
    return true;
  }
};

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
__device__ __forceinline__ void paged_note(const PagedParams& p, const PagedParts& parts, const PagedStart& st,
                                           const PagedPiece& x) {
  if (x.whole()) return;
  // the unit's first and last tile in the launch's list (x is the CTA's last
  // piece where it begins the unit, its first where it does not)
  const int64_t begin = x.begins() ? st.first + st.count - x.j1 : st.first - x.j0;
  const PagedShares shares(st.total, st.ctas);
  const int32_t first = shares.owner(begin);
  put_join(p, parts, 2 * blockIdx.x + (x.begins() ? 1 : 0),
           PagedJoin{x.b, x.kh, x.blk, first, shares.owner(begin + x.cost - 1) - first + 1});
}

}  // namespace varlen
