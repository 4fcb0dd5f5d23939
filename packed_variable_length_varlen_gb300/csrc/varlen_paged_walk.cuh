// varlen_paged_walk.cuh -- how the paged attention kernels share out their
// work.
//
// A unit is one block of rows of one (segment, key head); a row is one (query
// token, query head of the key head's group), token-major: row r is token r /
// group, head r % group.  A unit works through the key tiles that some of its
// rows see.  The units of a launch in a fixed order (segment, key head, row
// block), each with its tiles (at least one, so that a unit without keys is
// visited and writes its zeros), form one long list of tiles, and CTA c of N
// takes the tiles [c T / N, (c + 1) T / N): every CTA has the same number of
// tiles, whatever the lengths.  A CTA's part starts and ends inside a unit
// in general; what it has of a unit that it does not hold whole goes to the
// workspace as a partial result (its running maximum, sum and unnormalised
// output), in one of two slots: 1 for the unit that it begins and a later CTA
// ends, 0 for one that an earlier CTA began.  varlen_paged_join_kernel adds the
// partial results of a unit in the order of the CTAs.
//
// The lengths are device data: each CTA sums the costs itself (one segment
// per thread) and finds where its part begins.
#pragma once

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
  static constexpr int kRows = ROWS, kTile = TILE;
  __device__ static __forceinline__ int32_t half_tokens(const PagedParams& p) { return ROWS / 2 / p.group; }
  __device__ static __forceinline__ int32_t blocks(const PagedParams& p, int32_t n) {
    if (BY_TOKEN) return (int32_t)(((int64_t)n + 2 * half_tokens(p) - 1) / (2 * half_tokens(p)));
    return (int32_t)(((int64_t)n * p.group + ROWS - 1) / ROWS);
  }
  __device__ static __forceinline__ PagedUnit unit(const PagedParams& p, int32_t n, int32_t sk, int32_t blk) {
    PagedUnit u;
    if (BY_TOKEN) {
      const int32_t bt = 2 * half_tokens(p);
      u.t0 = blk * bt;
      u.t1 = min(n - u.t0, bt) + u.t0 - 1;
    } else {
      const int64_t r0 = (int64_t)blk * ROWS, r1 = min((int64_t)n * p.group, r0 + ROWS) - 1;
      u.t0 = (int32_t)(r0 / p.group);
      u.t1 = (int32_t)(r1 / p.group);
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
  const int32_t a = clamp_row(__ldg(p.cu_q + b), p.total_q), e = clamp_row(__ldg(p.cu_q + b + 1), p.total_q);
  s.q0 = a;
  s.n = max(e - a, 0);
  s.sk = cache_len(p.pages, b);
  const bool few = (int64_t)s.n * p.group <= kFewRows;
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
  int64_t after;  // tiles of the CTA's part that follow this piece
  __device__ __forceinline__ bool begins() const { return j0 == 0; }
  __device__ __forceinline__ bool ends() const { return j1 == cost; }
  __device__ __forceinline__ bool whole() const { return begins() && ends(); }
};

// Where a CTA's part begins, shared by its threads.
struct PagedStart {
  int64_t total, first, count;  // tiles of the launch; first tile and number of tiles of this CTA
  int64_t off;                  // first tile's place within segment b
  int32_t b, ctas;              // segment; CTAs that have work
  long long sums[32];
};

// CTAs that share `total` tiles: no more than leave each `least`.
__device__ __forceinline__ int32_t paged_ctas(int64_t total, int32_t grid, int32_t least) {
  const int64_t n = (total + least - 1) / least;
  return (int32_t)(n < 1 ? 1 : (n < grid ? n : grid));
}
// (total * c cannot overflow: fewer than 2^31 tokens of 2^7 rows over 2^31
// keys would take years; any launch that ends has total < 2^50, c < 2^10)
__device__ __forceinline__ int64_t paged_first(int64_t total, int32_t ctas, int32_t c) { return total * c / ctas; }
// The CTA that has tile x.
__device__ __forceinline__ int32_t paged_owner(int64_t total, int32_t ctas, int64_t x) {
  int32_t c = (int32_t)(x * ctas / total);
  while (c + 1 < ctas && paged_first(total, ctas, c + 1) <= x) ++c;
  while (c > 0 && paged_first(total, ctas, c) > x) --c;
  return c;
}

__device__ __forceinline__ long long warp_inclusive(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += t;
  }
  return v;
}

// Fills `st` (shared memory).  Every thread of the CTA (a whole number of
// warps) calls it; the CTA is synchronised when it returns.
template <class G>
__device__ __forceinline__ void paged_start(PagedStart& st, const PagedParams& p, int32_t take, int32_t least) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  long long mine = 0, mine_first = 0;
  for (int32_t b = threadIdx.x; b < p.batch; b += blockDim.x) {
    const long long c = (long long)p.kv_heads * paged_seg<G>(p, b, take).per_head;
    if (b < (int)blockDim.x) mine_first = c;
    mine += c;
  }
  long long incl = warp_inclusive(mine);
  if (lane == 31) st.sums[warp] = incl;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < warps; ++w) total += st.sums[w];
  const int32_t ctas = paged_ctas(total, gridDim.x, least);
  const bool works = total > 0 && (int32_t)blockIdx.x < ctas;
  const int64_t first = works ? paged_first(total, ctas, blockIdx.x) : 0;
  const int64_t last = works ? paged_first(total, ctas, blockIdx.x + 1) : 0;
  if (threadIdx.x == 0) {
    st.total = total;
    st.ctas = ctas;
    st.first = first;
    st.count = last - first;
    st.off = 0;
    st.b = 0;
  }
  __syncthreads();
  if (!works) return;  // CTA-uniform
  long long before = 0;
  for (int32_t base = 0; base < p.batch; base += blockDim.x) {
    const int32_t b = base + threadIdx.x;
    const long long c =
        b >= p.batch ? 0 : (base == 0 ? mine_first : (long long)p.kv_heads * paged_seg<G>(p, b, take).per_head);
    incl = warp_inclusive(c);
    if (lane == 31) st.sums[warp] = incl;
    __syncthreads();
    long long excl = before + incl - c, all = 0;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) excl += st.sums[w];
      all += st.sums[w];
    }
    if (first >= excl && first < excl + c) {
      st.b = b;
      st.off = first - excl;
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
    s = paged_seg<G>(p, b, take);
    int64_t off = st.off;
    kh = (int32_t)(off / s.per_head);
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
    x.after = left;
    if (x.j1 == x.cost) {
      ++blk;
      j = 0;
    } else {
      j = x.j1;
    }
    return true;
  }
};

// Left for the join by the one thread that calls it, for every piece: the
// unit that the CTA begins and does not end (its last piece, if any).
__device__ __forceinline__ void paged_note(PagedJoin* join, const PagedStart& st, const PagedPiece& x) {
  if (!x.begins() || x.ends()) return;
  const int64_t end = st.first + st.count + (x.cost - x.j1) - 1;  // the unit's last tile
  join[blockIdx.x] =
      PagedJoin{x.b, x.kh, x.blk, paged_owner(st.total, st.ctas, end) - (int32_t)blockIdx.x + 1};
}

}  // namespace varlen
