// varlen_paged_few.cu -- attention over the paged cache for few query rows:
// single tokens, drafted tokens, short chunks.
//
// Bound: every key and value is read once for at most 16 rows (query tokens
// times the query heads that share a key head), so the memory's rate decides and
// the matrix products only have to keep up with it.  At 6.8 TB/s an SM receives
// 44.7 bytes a nanosecond, 12 bf16 or 23 E4M3 elements a cycle.  The warp-level
// m16n8k16 products take keys (then columns of V) as their 16 rows and query
// rows as their 8 columns, S^T = K Q^T and O^T = V^T P^T: a step of 16 keys for 8
// rows is 16 products at D = 128 (bf16 24, for P's second part), and o takes 32
// registers, so that enough warps stay resident to hide the chain of products,
// softmax and products.  (The other
// way round, 16 query rows by 8 keys, costs twice the products and registers
// while most of the 16 rows are empty: 214 us where this form took 190 for 64
// ragged E4M3 sequences, and 124 with the third CTA an SM that its registers leave
// room for.)
// Measured: 8 sequences of 17580 bf16 keys, 56 heads of 128, one token: 564-585 us
// across machines, 6.9-7.1 TB/s, the copy rate.  64 E4M3 sequences of 1..8192 keys,
// 8 key heads: 115-120 us, 4.3-4.5 TB/s.  What holds E4M3 back, from runs in which
// the consumers only gave the slots back (TB/s whole / stream alone): pages whose
// rows of one head lie apart come in pieces of 128 bytes, bf16 in 256; 64 x 4096
// keys, 8 key heads 5.1 / 5.3, with head-major pages 5.5 / 6.0, bf16 6.3 / 6.4; 8 x
// 17580 keys, 56 heads 5.8 / 5.9 and head-major 6.5 / 6.9, bf16 6.9 / 6.9.  The
// stream decides, then; in short calls the start (4 us until the first tile) and the
// join (5 us) weigh besides, and among ragged lengths the ends of many short units
// (64 of up to 8192 keys 4.4 / 5.3).
//
// A CTA is four consumer warps and a producer warp; two (bf16) or three (E4M3)
// CTAs share an SM.
// The producer streams tiles of K and of V, page piece by page piece, through
// a ring of shared-memory slots by TMA (an entry that names no page, and
// positions past the sequence, become an out-of-range page: zeros, no
// traffic).  Rows are taken in tiles of 8; the warps that share a row tile split
// each key tile, every one with its own online softmax (m, l, o in registers,
// 32-bit), and join theirs through shared memory at the end of a unit, in a
// fixed order.
//
// Operands need no shuffling but for P, which is transposed in registers.  S
// sums over d, so both operands may take d in any order: a lane reads 16
// consecutive bytes of its key's row, and Q is loaded to match.  The same holds
// for the order of O's columns: with E4M3 a lane reads D/8 consecutive bytes of
// each of its four keys, which stand for its row of D/8 different half-tiles.
//
// bf16: the products want P in V's type.  One bf16 of it would put 2^-9 of each
// weight's size into O, as much again as O's own rounding, so P comes in two
// parts of 8 bits, hi + lo, and V is multiplied by both: twice the products of
// that half, which the memory hides (8 sequences of 17580 keys 584 us either
// way; 4 drafted tokens of 4 sequences 15.8 and 15.9).
//
// E4M3 codes become f16 (exact, two a conversion) and both products run in
// f16 with 32-bit sums.  What f16 lacks in range the scales make up for:
//   S: a row of Q is multiplied by the power of two that brings its largest
//      element to 2^14 (f16 then holds all of a bf16 that is not 2^-28 of the
//      largest), and S by that power's inverse and the key's scale.
//   P V: the weight of key j is P_j s_j / R * 2^13, with R the largest scale
//      that the warp has met (o is kept in units of R 2^-13): at most 2^15, as P
//      stays below 2^2 (the maximum follows when a key passes it by more), and
//      f16 holds it in 11 bits down to P_j s_j / R = 2^-27, as well as bf16 would
//      down to 2^-29, and with an error of 2^-38 below.  Where a key's scale lies
//      more than 2^8 below R (or is NaN), the step's products run in bf16
//      instead, so that P_j is held to bf16's 8 bits or better down to 2^-21 of
//      the row's largest weight whatever the scales are: a code's bits s eeee mmm
//      moved to s 0000eeee mmm0000 are the bf16 code * 2^-120, subnormals too,
//      times 2^127 s / R, and P times 2^6 (one bf16 of P: there are no registers
//      left for a second).  A vector of zeros has a scale of 1
//      that says nothing of its neighbours' size: it counts as one that is not
//      there, and R does not follow it.
#include <cuda_fp8.h>

#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

constexpr int kLeastTiles = 2;  // tiles per CTA when there are few
constexpr int kMaxSlots = 8;

template <int D, bool E4M3>
struct FewCfg {
  static constexpr int WARPS = 4;                           // consumer warps
  static constexpr int THREADS = (WARPS + 1) * 32;
  static constexpr int KT = kFewTile;                       // keys per tile
  static constexpr int STEP = 16;                           // keys a warp takes at a time
  static constexpr int ROWS = kFewRows;
  using Geom = PagedGeom<ROWS, KT, false>;
  static constexpr int CK = E4M3 ? 1 : (D + 63) / 64;       // 128-byte column chunks of a row
  static constexpr int CHUNK = KT * 128;
  static constexpr int TILE = CK * CHUNK;
  static constexpr int SCALES = E4M3 ? KT * 8 : 0;          // page pieces of at least 16 keys, 128 bytes apart
  // Slots of K or V tiles: four are enough to cover the memory's latency, and
  // more are slower (64 E4M3 sequences 116 us with four, 118 with five, 125 with
  // seven; 56 bf16 heads 584 with four, 592 with five).
  static constexpr int NSLOT = E4M3 ? 4 : (CK == 1 ? 6 : 4);
  static constexpr int KSTEPS = E4M3 ? (D == 64 ? 4 : 8) : CK * 4;
  static constexpr int MT = D / 16;                         // m-tiles of O^T
  static constexpr int XCHG = (MT * 4 + 4) * 32 * 4;        // one warp's (o, m, l)
  static constexpr int SMEM = 1024 + NSLOT * (TILE + SCALES) + WARPS / 2 * XCHG;
};

struct FewShared {
  uint64_t full[kMaxSlots], empty[kMaxSlots], join;
  int abort;
  PagedStart start;
};
static_assert(sizeof(FewShared) <= 1024, "barrier block too large");

// d += A B: A 16 x 16 (a: rows r, r + 8 of its first eight columns, then of its
// last), B 16 x 8 (b), bf16 or f16 with 32-bit sums.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements, two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// mbar_wait_warp whose loop stands apart, so that the way through a tile stays
// short.
__device__ __noinline__ bool warp_wait_long(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_long(bar, parity, abort);
}

template <class T>
__device__ __forceinline__ T lds(const uint8_t* p) {
  return *reinterpret_cast<const T*>(p);
}

// Byte offset of bytes [off, ...) of row `row` in a tile of 128-byte rows
// in the 128-byte swizzle (off within one 16-byte chunk).
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t off) { return row * 128 + (off ^ ((row & 7) << 4)); }

// Codes in bits 8..15 and 24..31 of x as bf16 pairs code * 2^-120 (the
// other bits of x do not matter).
__device__ __forceinline__ uint32_t raw_pair(uint32_t x) { return (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u); }

__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}

// Four codes as f16: the first two and the last two.
__device__ __forceinline__ void f16_pairs(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Shared-memory offset of the scale of key r of a tile whose page pieces hold
// 1 << shift keys.
__device__ __forceinline__ uint32_t scale_at(uint32_t r, int shift) {
  return ((r >> shift) << 7) + ((r & ((1u << shift) - 1)) << 1);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(FewCfg<D, E4M3>::THREADS, few_ctas(E4M3))
    varlen_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                            const PagedParams p, const PagedParts parts, int32_t take) {
  using C = FewCfg<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_addr(smem) & 1023u) != 0) {
    paged_refuse(p, parts);
    return;
  }
  FewShared& sh = *reinterpret_cast<FewShared*>(smem);
  uint8_t* ring = smem + 1024;
  uint8_t* scales = ring + C::NSLOT * C::TILE;
  float* xchg = reinterpret_cast<float*>(scales + C::NSLOT * C::SCALES);
  volatile int* abort = &sh.abort;
  const int warp = warp_id(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], C::WARPS);
    }
    mbar_init(&sh.join, C::WARPS * 32);
    sh.abort = 0;
    fence_barrier_init();
  }
  dependency_wait();  // nothing above reads or writes global memory
  paged_start<typename C::Geom>(sh.start, p, take, kLeastTiles);
  dependents_may_launch();
  PagedWalk<typename C::Geom> walk;
  PagedPiece x;
  const int box_shift = min(p.pages.page_shift, 6);  // keys of one page piece of a tile

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      clear_join(p, parts);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int pieces = C::KT >> box_shift;
    const bool loads = lane < pieces * C::CK, loads_scale = E4M3 && lane < pieces;
    const int piece = lane % pieces, cc = lane / pieces;
    uint32_t pos = 0;
    bool ok = true;
    walk.init(sh.start, p, take);
    while (ok && walk.next(p, x)) {
      if (lane == 0) paged_note(p, parts, sh.start, x);
      const int32_t tiles = min(x.j1, x.u.tiles);
      for (int32_t j = x.j0; ok && j < tiles; ++j) {
        const int32_t key = (x.u.tile0 + j) * C::KT + (piece << box_shift);
        int32_t page = p.pages.num_pages;
        if (loads && key < x.u.hi && key + (1 << box_shift) > x.u.lo)
          page = page_at(p.pages, x.b, key >> p.pages.page_shift, p.err);
        const int32_t row = key & (p.pages.page_size - 1);
#pragma unroll
        for (int which = 0; which < 2; ++which, ++pos) {
          const uint32_t slot = pos % C::NSLOT;
          if (!mbar_wait_warp(&sh.empty[slot], ((pos / C::NSLOT) & 1) ^ 1, abort)) {
            ok = false;
            break;
          }
          // (failure test: CTA 0 leaves one load out)
          if (blockIdx.x == 0 && (int64_t)pos == (int64_t)p.debug_skip_few) continue;
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], C::TILE + (E4M3 ? C::KT * 2 : 0));
          __syncwarp();
          if (loads)
            tma_load_4d(ring + slot * C::TILE + cc * C::CHUNK + ((piece << box_shift) * 128), which ? &tm_v : &tm_k,
                        &sh.full[slot], cc * 64, x.kh, row, page);
          if (loads_scale)
            tma_load_3d(scales + slot * C::SCALES + piece * 128, which ? &tm_vs : &tm_ks, &sh.full[slot], row, x.kh,
                        page);
        }
      }
    }
    if (!ok && lane == 0) {
      // every copy in flight lands before the CTA's shared memory is released (bounded)
      for (uint32_t s = 0; s < C::NSLOT && s < pos; ++s) {
        const uint32_t last = pos - 1 - ((pos - 1 - s) % C::NSLOT);
        int dummy = 0;
        mbar_wait(&sh.full[s], (last / C::NSLOT) & 1, &dummy, 100000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ consumers
    const int r = lane >> 2, c = lane & 3;
    uint32_t pos = 0, joins = 0;
    bool ok = true;
    walk.init(sh.start, p, take);
    while (ok && walk.next(p, x)) {
      // rows of the unit: first is row `skip` of token t0
      const int32_t skip = x.blk * C::ROWS - x.u.t0 * p.group;
      const int32_t rows = min((x.n - x.u.t0) * p.group - skip, C::ROWS);
      const int mt = rows <= 8 ? 1 : 2;  // row tiles
      const int rt = warp & (mt - 1), kg = warp / mt, share = C::WARPS / mt;
      const bool works = rt * 8 < rows;
      // the operand B holds row r of the tile; the sums hold rows 2c, 2c + 1
      int32_t tok[2], klo[2], khi[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tok[i] = x.u.t0 + (skip + min(rt * 8 + 2 * c + i, rows - 1)) / p.group;
        band_keys(tok[i], tok[i], x.n, x.sk, p.win_left, p.win_right, &klo[i], &khi[i]);
      }
      uint32_t qf[C::KSTEPS][2];
      float rowf[2] = {p.scale_log2, p.scale_log2};
      if (works) {
        const bool live = rt * 8 + r < rows;
        const int32_t at = skip + min(rt * 8 + r, rows - 1), t = at / p.group;
        const __nv_bfloat16* qa =
            p.q + (int64_t)(x.q0 + x.u.t0 + t) * p.q_rs + (int64_t)(x.kh * p.group + at - t * p.group) * p.q_hs;
        auto load = [&](int d0) {
          return live && d0 < D && in_span(p.q_span, qa + d0, 16, p.err) ? *reinterpret_cast<const uint4*>(qa + d0)
                                                                        : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int s = 0; s < C::KSTEPS / 2; ++s) {  // eight elements of this lane
          const uint4 u = load(E4M3 ? (C::KSTEPS == 4 ? c : 2 * c + (s >> 1)) * 16 + (s & 1) * 8
                                    : (s >> 1) * 64 + (2 * c + (s & 1)) * 8);
          qf[2 * s][0] = u.x;
          qf[2 * s][1] = u.y;
          qf[2 * s + 1][0] = u.z;
          qf[2 * s + 1][1] = u.w;
        }
        if constexpr (E4M3) {  // to f16, the row's largest element at 2^14
          uint32_t top = 0;
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k)
            top = __vmaxu2(top, __vmaxu2(qf[k][0] & 0x7fff7fffu, qf[k][1] & 0x7fff7fffu));
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // its biased exponent, within what leaves both powers normal
          const int e = min(max((int)(max(top & 0xffffu, top >> 16) >> 7), 15), 254);
          const float up = __uint_as_float((uint32_t)(254 + 14 - e) << 23);
#pragma unroll
          for (int k = 0; k < C::KSTEPS; ++k)
#pragma unroll
            for (int y = 0; y < 2; ++y) qf[k][y] = pack_f16x2(bf16_lo(qf[k][y]) * up, bf16_hi(qf[k][y]) * up);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            rowf[i] *= __uint_as_float((uint32_t)(__shfl_sync(0xffffffffu, e, (2 * c + i) * 4) - 14) << 23);
        }
      }
      float vref = 0.f, vinv = 0.f;  // E4M3: R and 1 / R (finite: R >= 2^-127)
      float o[C::MT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < C::MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
      // keys that every row of the unit sees: no select needed
      int32_t all_lo, all_hi;
      {
        int32_t a, e;
        band_keys(x.u.t1, x.u.t1, x.n, x.sk, p.win_left, p.win_right, &all_lo, &e);
        band_keys(x.u.t0, x.u.t0, x.n, x.sk, p.win_left, p.win_right, &a, &all_hi);
      }
      const int32_t tiles = min(x.j1, x.u.tiles);
      if (!works) {  // no rows: only gives the slots back
        for (int32_t j = 2 * x.j0; ok && j < 2 * tiles; ++j, ++pos) {
          const uint32_t slot = pos % C::NSLOT;
          ok = warp_wait(&sh.full[slot], (pos / C::NSLOT) & 1, abort);
          if (ok && lane == 0) mbar_arrive(&sh.empty[slot]);
        }
      }
      for (int32_t j = works ? x.j0 : tiles; j < tiles; ++j, pos += 2) {
        const uint32_t ks = pos % C::NSLOT, vs = (pos + 1) % C::NSLOT;
        if (!warp_wait(&sh.full[ks], (pos / C::NSLOT) & 1, abort)) {
          ok = false;
          break;
        }
        __syncwarp();
        const uint8_t *kt = ring + ks * C::TILE, *vt = ring + vs * C::TILE;
        const uint8_t *ksc = scales + ks * C::SCALES, *vsc = scales + vs * C::SCALES;
        const int32_t key0 = (x.u.tile0 + j) * C::KT;
        const bool edge = key0 < all_lo || key0 + C::KT > all_hi;
        // rows of V that no row of the unit sees may hold anything: cleared
        const bool vedge = key0 < x.u.lo || key0 + C::KT > x.u.hi;
        bool v_here = false;
        // the steps of this warp: kg, kg + share, ...
#pragma unroll 1
        for (int a = kg * C::STEP; a < C::KT; a += share * C::STEP) {
          float s[4], s2[4];  // keys a + r and a + r + 8 of rows 2c, 2c + 1; s2: a second chain of products
          {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = s2[e] = 0.f;
            constexpr int NL = E4M3 ? C::KSTEPS / 4 : C::KSTEPS / 2;  // 16-byte loads of a key
            uint4 u[NL], v[NL];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
              const uint32_t at = E4M3 ? swz(a + r, (C::KSTEPS == 4 ? c : 2 * c + i) * 16)
                                       : (i >> 1) * C::CHUNK + swz(a + r, (2 * c + (i & 1)) * 16);
              u[i] = lds<uint4>(kt + at);
              v[i] = lds<uint4>(kt + at + 8 * 128);  // eight rows on: the same place in the swizzle
            }
#pragma unroll
            for (int i = 0; i < NL; ++i) {
              if constexpr (E4M3) {
                const uint32_t x0[4] = {u[i].x, u[i].y, u[i].z, u[i].w}, x1[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t a0, a1, a2, a3;
                  f16_pairs(x0[k], a0, a2);
                  f16_pairs(x1[k], a1, a3);
                  mma16816<true>((k & 1) ? s2 : s, a0, a1, a2, a3, qf[i * 4 + k][0], qf[i * 4 + k][1]);
                }
              } else {
                mma16816<false>(s, u[i].x, v[i].x, u[i].y, v[i].y, qf[2 * i][0], qf[2 * i][1]);
                mma16816<false>(s2, u[i].z, v[i].z, u[i].w, v[i].w, qf[2 * i + 1][0], qf[2 * i + 1][1]);
              }
            }
            if constexpr (E4M3) {
              // the row's and the key's factor first: either alone may take the sum out of range
              const float k0 = __bfloat162float(lds<__nv_bfloat16>(ksc + scale_at(a + r, box_shift)));
              const float k1 = __bfloat162float(lds<__nv_bfloat16>(ksc + scale_at(a + r + 8, box_shift)));
#pragma unroll
              for (int e = 0; e < 4; ++e) s[e] = (s[e] + s2[e]) * (rowf[e & 1] * (e < 2 ? k0 : k1));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) s[e] = (s[e] + s2[e]) * rowf[e & 1];
            }
          }
          if (a + share * C::STEP >= C::KT) {  // the warp's last step on this K tile
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[ks]);
          }
          {
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int32_t key = key0 + a + r + (e >> 1) * 8;
                s[e] = key >= klo[e & 1] && key < khi[e & 1] ? s[e] : -INFINITY;
              }
            }
            // The maximum follows only when a key passes it by more than 2^8, with E4M3
            // 2^2 (o and l carry the same factor, so nothing is lost): the lanes of a
            // row need to look at one another's keys only then.
            constexpr float kLag = E4M3 ? 2.f : 8.f;
            float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kLag || mx[1] > m[1] + kLag)) {
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) {
                mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], w));
                mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], w));
              }
              float al[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[i], mx[i]);
                al[i] = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
                m[i] = mn;
                l[i] *= al[i];
              }
#pragma unroll
              for (int t = 0; t < C::MT; ++t) {
                o[t][0] *= al[0];
                o[t][1] *= al[1];
                o[t][2] *= al[0];
                o[t][3] *= al[1];
              }
            }
            const float sub[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = ex2(s[e] - sub[e & 1]);
            l[0] += s[0] + s[2];
            l[1] += s[1] + s[3];
          }
          if (!v_here) {
            v_here = warp_wait(&sh.full[vs], ((pos + 1) / C::NSLOT) & 1, abort);
            ok = ok && v_here;
          }
          if (!ok) break;
          __syncwarp();
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // keys 2c, 2c+1 and 2c+8, 2c+9
          if (vedge) {
            auto in = [&](int k) { return key0 + a + k >= x.u.lo && key0 + a + k < x.u.hi; };
            keep0 = (in(2 * c) ? 0xffffu : 0u) | (in(2 * c + 1) ? 0xffff0000u : 0u);
            keep1 = (in(2 * c + 8) ? 0xffffu : 0u) | (in(2 * c + 9) ? 0xffff0000u : 0u);
          }
          if constexpr (E4M3) {
            uint32_t w[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t row = a + 2 * c + (k & 1) + (k >> 1) * 8;
              if constexpr (D == 128) {
                const uint4 u = lds<uint4>(vt + swz(row, r * 16));
                w[k][0] = u.x;
                w[k][1] = u.y;
                w[k][2] = u.z;
                w[k][3] = u.w;
              } else if constexpr (D == 64) {
                const uint2 u = lds<uint2>(vt + swz(row, r * 8));
                w[k][0] = u.x;
                w[k][1] = u.y;
              } else {
#pragma unroll
                for (int i = 0; i < 3; ++i) w[k][i] = lds<uint32_t>(vt + swz(row, r * 12 + i * 4));
              }
            }
            // scales of keys a + r, a + r + 8, the rows of P; 0 stands for a vector that is not there
            float sv[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) sv[k] = __bfloat162float(lds<__nv_bfloat16>(vsc + scale_at(a + r + 8 * k, box_shift)));
            if (vedge) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
                sv[k] = key0 + a + r + 8 * k >= x.u.lo && key0 + a + r + 8 * k < x.u.hi ? sv[k] : 0.f;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const bool keep = ((k >> 1) ? keep1 : keep0) & ((k & 1) ? 0xffff0000u : 0xffffu);
#pragma unroll
                for (int i = 0; i < D / 32; ++i) w[k][i] = keep ? w[k][i] : 0u;
              }
            }
            auto odd = [&] {
              const float least = vref * 0x1p-8f;
              return __any_sync(0xffffffffu, !(sv[0] <= vref) || !(sv[1] <= vref) || (sv[0] < least && sv[0] != 0.f) ||
                                                 (sv[1] < least && sv[1] != 0.f));
            };
            bool wide = odd();
            if (wide) {
              // Vectors of zeros (with a finite scale) drop out: bit k of `here` says
              // that key 2c + (k & 1) + 8 (k >> 1) has a code that is not zero, then
              // each lane asks for the keys of its scales, and tells which drop.
              uint32_t here = 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) any |= w[k][i];
                here |= (any & 0x7f7f7f7fu) != 0 ? 1u << k : 0u;
              }
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) here |= __shfl_xor_sync(0xffffffffu, here, k);
              here = __shfl_sync(0xffffffffu, here, r >> 1) >> (r & 1);
              uint32_t drop = 0;  // bit 0: key a + r, bit 1: a + r + 8
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (((here >> (2 * k)) & 1u) == 0 && sv[k] == sv[k]) {
                  sv[k] = 0.f;
                  drop |= 1u << k;
                }
              const uint32_t d0 = __shfl_sync(0xffffffffu, drop, 8 * c), d1 = __shfl_sync(0xffffffffu, drop, 8 * c + 4);
              keep0 &= ((d0 & 1u) ? 0u : 0xffffu) | ((d1 & 1u) ? 0u : 0xffff0000u);
              keep1 &= ((d0 & 2u) ? 0u : 0xffffu) | ((d1 & 2u) ? 0u : 0xffff0000u);
              // a new largest scale: o to its units; and look again
              float top = fmaxf(sv[0], sv[1]);
#pragma unroll
              for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
              if (top > vref) {
                const float f = vref / top;  // powers of two (or 0)
                vref = top;
                vinv = 1.f / top;
#pragma unroll
                for (int t = 0; t < C::MT; ++t)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[t][e] *= f;
              }
              wide = odd();
            }
            if (!wide) {
              const float f0 = sv[0] * vinv * 0x1p13f, f1 = sv[1] * vinv * 0x1p13f;
              const uint32_t p0 = transpose8(pack_f16x2(s[0] * f0, s[1] * f0));
              const uint32_t p1 = transpose8(pack_f16x2(s[2] * f1, s[3] * f1));
#pragma unroll
              for (int t = 0; t < C::MT; ++t) {
                const uint32_t sel = (t & 1) ? 0x7362u : 0x5140u;
                const uint32_t u0 = __byte_perm(w[0][t >> 1], w[1][t >> 1], sel);
                const uint32_t u1 = __byte_perm(w[2][t >> 1], w[3][t >> 1], sel);
                uint32_t a0, a1, a2, a3;
                f16_pairs(u0, a0, a1);
                f16_pairs(u1, a2, a3);
                mma16816<true>(o[t], a0, a1, a2, a3, p0, p1);
              }
            } else {
              const float up = vref > 0.f ? vinv : 1.f;
              // the factors of keys 2c, 2c + 1 and 2c + 8, 2c + 9
              uint32_t f[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t sc = lds<uint32_t>(vsc + scale_at(a + 2 * c + 8 * k, box_shift)) & (k ? keep1 : keep0);
                f[k] = pack_bf16x2(bf16_lo(sc) * up * 0x1p127f, bf16_hi(sc) * up * 0x1p127f);
              }
              const uint32_t p0 = transpose8(pack_bf16x2(s[0] * 0x1p6f, s[1] * 0x1p6f));
              const uint32_t p1 = transpose8(pack_bf16x2(s[2] * 0x1p6f, s[3] * 0x1p6f));
#pragma unroll
              for (int t = 0; t < C::MT; ++t) {
                uint32_t b[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // half-tile k & 1, keys k >> 1
                  const int y = 2 * t + (k & 1);
                  constexpr uint32_t kSel[4] = {0x4000u, 0x5010u, 0x6020u, 0x7030u};
                  b[k] = mul_pair(raw_pair(__byte_perm(w[k & 2][y >> 2], w[(k & 2) + 1][y >> 2], kSel[y & 3])), f[k >> 1]);
                }
                mma16816<false>(o[t], b[0], b[1], b[2], b[3], p0, p1);
              }
            }
          } else {
            const uint32_t row = a + (lane & 15);
            // P in two bf16 parts, the second what the first leaves: 16 bits of it
            const uint32_t h0 = pack_bf16x2(s[0], s[1]), h1 = pack_bf16x2(s[2], s[3]);
            const uint32_t p0 = transpose8(h0), p1 = transpose8(h1);
            const uint32_t e0 = transpose8(pack_bf16x2(s[0] - bf16_lo(h0), s[1] - bf16_hi(h0)));
            const uint32_t e1 = transpose8(pack_bf16x2(s[2] - bf16_lo(h1), s[3] - bf16_hi(h1)));
#pragma unroll
            for (int t = 0; t < C::MT; ++t) {
              uint32_t b[4];
              ldsm_x4_t(b, smem_addr(vt) + (t >> 2) * C::CHUNK + swz(row, ((2 * t & 7) + (lane >> 4)) * 16));
              mma16816<false>(o[t], b[0] & keep0, b[2] & keep0, b[1] & keep1, b[3] & keep1, p0, p1);
              mma16816<false>(o[t], b[0] & keep0, b[2] & keep0, b[1] & keep1, b[3] & keep1, e0, e1);
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[vs]);
      }
      if (!ok) break;
      if constexpr (E4M3) {
        const float f = vref * 0x1p-13f;
#pragma unroll
        for (int t = 0; t < C::MT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] *= f;
      }
      // row sums over the lanes of a row
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], w);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], w);
      }
      // join the warps that share these rows
      for (int step = share >> 1; step >= 1 && ok; step >>= 1) {
        float* buf = xchg + ((kg & (step - 1)) * mt + rt) * (C::XCHG / 4) + lane;
        if (kg >= step && kg < 2 * step) {
#pragma unroll
          for (int t = 0; t < C::MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) buf[(t * 4 + e) * 32] = o[t][e];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            buf[(C::MT * 4 + i) * 32] = m[i];
            buf[(C::MT * 4 + 2 + i) * 32] = l[i];
          }
        }
        mbar_arrive(&sh.join);
        if (!warp_wait(&sh.join, joins++ & 1, abort)) {
          ok = false;
          break;
        }
        if (kg < step) {
          float a0[2], a1[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m1 = buf[(C::MT * 4 + i) * 32], mn = fmaxf(m[i], m1);
            a0[i] = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
            a1[i] = mn == -INFINITY ? 1.f : ex2(m1 - mn);
            m[i] = mn;
            l[i] = l[i] * a0[i] + buf[(C::MT * 4 + 2 + i) * 32] * a1[i];
          }
#pragma unroll
          for (int t = 0; t < C::MT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = o[t][e] * a0[e & 1] + buf[(t * 4 + e) * 32] * a1[e & 1];
        }
        mbar_arrive(&sh.join);
        if (!warp_wait(&sh.join, joins++ & 1, abort)) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      if (kg != 0 || !works) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t rr = rt * 8 + 2 * c + i;  // row of the unit; this lane's columns of it:
        if (rr >= rows) continue;
        if (x.whole()) {
          const int32_t at = skip + rr, t0 = at / p.group, hd = x.kh * p.group + at - t0 * p.group;
          const int64_t row = x.q0 + x.u.t0 + t0;
          const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // no key: 0; NaN stays
          __nv_bfloat16* oa = p.out + row * p.o_rs + (int64_t)hd * p.o_hs;
          if constexpr (E4M3) {  // D/8 consecutive ones
#pragma unroll
            for (int t = 0; t < C::MT; t += 2) {
              __nv_bfloat16* d = oa + r * (D / 8) + 2 * t;
              if (in_span(p.out_span, d, 8, p.err))
                *reinterpret_cast<uint2*>(d) = make_uint2(pack_bf16x2(o[t][i] * inv, o[t][2 + i] * inv),
                                                          pack_bf16x2(o[t + 1][i] * inv, o[t + 1][2 + i] * inv));
            }
          } else {  // r, r + 8 of each 16
#pragma unroll
            for (int t = 0; t < C::MT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                __nv_bfloat16* d = oa + t * 16 + e * 8 + r;
                if (in_span(p.out_span, d, 2, p.err)) *d = __float2bfloat16_rn(o[t][2 * e + i] * inv);
              }
          }
          float* la = p.lse + (int64_t)hd * p.total_q + row;
          if (r == 0 && in_span(p.lse_span, la, 4, p.err))
            *la = l[i] == 0.f ? -INFINITY : (m[i] + __log2f(l[i])) * 0.69314718055994531f;
        } else {
          const int64_t row = (2 * (int64_t)blockIdx.x + (x.begins() ? 1 : 0)) * parts.rows + rr;
          float* oa = parts.o + row * D;
          if constexpr (E4M3) {
#pragma unroll
            for (int t = 0; t < C::MT; t += 2) {
              float* d = oa + r * (D / 8) + 2 * t;
              if (in_span(parts.o_span, d, 16, p.err))
                *reinterpret_cast<float4*>(d) = make_float4(o[t][i], o[t][2 + i], o[t + 1][i], o[t + 1][2 + i]);
            }
          } else {
#pragma unroll
            for (int t = 0; t < C::MT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float* d = oa + t * 16 + e * 8 + r;
                if (in_span(parts.o_span, d, 4, p.err)) *d = o[t][2 * e + i];
              }
          }
          float* ml = parts.ml + row * 2;
          if (r == 0 && in_span(parts.ml_span, ml, 8, p.err)) *reinterpret_cast<float2*>(ml) = make_float2(m[i], l[i]);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && sh.abort) record_error(p.err, kErrTimeout);
}

template <int D, bool E4M3>
cudaError_t launch_few_d(const PagedLaunch& L, int32_t take, cudaStream_t stream) {
  using C = FewCfg<D, E4M3>;
  auto kern = varlen_paged_few_kernel<D, E4M3>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, (unsigned)(L.sms * few_ctas(E4M3)), C::THREADS, C::SMEM, stream, L.few_k, L.few_v, L.few_ks,
                           L.few_vs, L.p, L.few_parts, take);
}

}  // namespace

cudaError_t launch_paged_few(const PagedLaunch& L, int32_t take, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return L.e4m3 ? launch_few_d<64, true>(L, take, stream) : launch_few_d<64, false>(L, take, stream);
    case 96: return L.e4m3 ? launch_few_d<96, true>(L, take, stream) : launch_few_d<96, false>(L, take, stream);
    case 128: return L.e4m3 ? launch_few_d<128, true>(L, take, stream) : launch_few_d<128, false>(L, take, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace varlen
