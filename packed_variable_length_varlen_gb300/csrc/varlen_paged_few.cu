// varlen_paged_few.cu -- attention over the paged cache for few query rows:
// single tokens, drafted tokens, short chunks.
//
// Bound: every key and value is read once for at most 64 rows (query tokens
// times the query heads that share a key head), so the memory's rate decides
// and the matrix products only have to keep up with it.  At 6.8 TB/s an SM
// receives 44.7 bytes a nanosecond, 12 bf16 or 23 E4M3 elements a cycle; with
// 16 rows the warp-level m16n8k16 products cost 16 multiply-adds an element,
// a fraction of their rate, which is why they are used here and the
// tcgen05 units, whose tiles have 128 rows, are not.
//
// A CTA is four consumer warps and a producer warp; two CTAs share an SM.
// The producer streams 64-key tiles of K and of V, page piece by page piece,
// through a ring of shared-memory slots by TMA (an entry that names no page,
// and positions past the sequence, become an out-of-range page: zeros, no
// traffic).  Rows are taken in tiles of 16: a unit of up to 16 rows splits each
// tile's keys over the four warps, of up to 32 rows over two pairs, and 64 rows
// give every warp its own rows and all keys.  Each warp runs its own online
// softmax (m, l, o in registers, 32-bit); at the end of a unit the warps that
// share rows join theirs through shared memory, in a fixed order.
//
// Operands need no shuffling.  The product S = Q K^T sums over d, so both
// operands may take d in any order: a lane reads 16 consecutive bytes of its
// key's row, and Q is loaded to match.  The same holds for the columns of
// O = P V: with E4M3 a lane reads D/8 consecutive bytes of each of its four
// keys, which stand for its column of D/8 different n-tiles.  An E4M3 code s
// eeee mmm becomes a bf16 by moving its bits to s 0000eeee mmm0000, which is
// code * 2^-120 exactly (subnormals too), times 2^120 * scale.
#include <cuda_fp8.h>

#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

using FewGeom = PagedGeom<kFewRows, kFewTile, false>;

constexpr int kWarps = 4;                         // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kLeastTiles = 2;                    // tiles per CTA when there are few

template <int D, bool E4M3>
struct FewCfg {
  static constexpr int CK = E4M3 ? 1 : (D + 63) / 64;       // 128-byte column chunks of a row
  static constexpr int CHUNK = kFewTile * 128;
  static constexpr int TILE = CK * CHUNK;
  static constexpr int SCALES = E4M3 ? 512 : 0;             // up to four page pieces, 128 bytes apart
  static constexpr int NSLOT = E4M3 ? 8 : (CK == 1 ? 8 : 5);
  static constexpr int KSTEPS = E4M3 ? (D == 64 ? 4 : 8) : CK * 4;
  static constexpr int NT = D / 8;                          // n-tiles of O
  static constexpr int XCHG = (NT * 4 + 4) * 32 * 4;        // one warp's (o, m, l)
  static constexpr int SMEM = 1024 + NSLOT * (TILE + SCALES) + 2 * XCHG;
};

struct FewShared {
  uint64_t full[8], empty[8], join;
  int abort;
  PagedStart start;
};
static_assert(sizeof(FewShared) <= 1024, "barrier block too large");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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

// 2^120 * scale as two bf16 factors: f, and a rest that is 1 unless the
// product passes 2^127 (a scale above 2^7).
struct Factor {
  uint32_t f, rest;  // pairs
};
__device__ __forceinline__ Factor factor_of(uint32_t scales) {  // two bf16 scales
  const float a = __uint_as_float(scales << 16) * 0x1p120f, b = __uint_as_float(scales & 0xffff0000u) * 0x1p120f;
  const bool la = a > 0x1p127f, lb = b > 0x1p127f;
  Factor x;
  x.f = pack_bf16x2(la ? 0x1p127f : a, lb ? 0x1p127f : b);
  x.rest = pack_bf16x2(la ? __uint_as_float(scales << 16) * 0x1p-7f : 1.f,
                       lb ? __uint_as_float(scales & 0xffff0000u) * 0x1p-7f : 1.f);
  return x;
}

// Shared-memory offset of the scale of key r of a tile whose page pieces hold
// 1 << shift keys.
__device__ __forceinline__ uint32_t scale_at(uint32_t r, int shift) {
  return ((r >> shift) << 7) + ((r & ((1u << shift) - 1)) << 1);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, kFewCtasPerSm)
    varlen_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs,
                            const PagedParams p, const PagedParts parts, int32_t take) {
  using C = FewCfg<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_addr(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) record_error(p.err, kErrBounds);
    return;
  }
  FewShared& sh = *reinterpret_cast<FewShared*>(smem);
  uint8_t* ring = smem + 1024;
  uint8_t* scales = ring + C::NSLOT * C::TILE;
  float* xchg = reinterpret_cast<float*>(scales + C::NSLOT * C::SCALES);
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    mbar_init(&sh.join, kWarps * 32);
    sh.abort = 0;
    fence_barrier_init();
  }
  dependency_wait();  // nothing above reads or writes global memory
  paged_start<FewGeom>(sh.start, p, take, kLeastTiles);
  dependents_may_launch();
  PagedWalk<FewGeom> walk;
  PagedPiece x;
  const int box_shift = min(p.pages.page_shift, 6);  // keys of one page piece of a tile

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      parts.join[blockIdx.x].parts = 0;
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    const int pieces = kFewTile >> box_shift;
    const bool loads = lane < pieces * C::CK, loads_scale = E4M3 && lane < pieces;
    const int piece = lane % pieces, cc = lane / pieces;
    uint32_t pos = 0;
    bool ok = true;
    walk.init(sh.start, p, take);
    while (ok && walk.next(p, x)) {
      if (lane == 0) paged_note(parts.join, sh.start, x);
      const int32_t tiles = min(x.j1, x.u.tiles);
      for (int32_t j = x.j0; ok && j < tiles; ++j) {
        const int32_t key = (x.u.tile0 + j) * kFewTile + (piece << box_shift);
        int32_t page = p.pages.num_pages;
        if (loads && key < x.u.hi && key + (1 << box_shift) > x.u.lo)
          page = page_at(p.pages, x.b, key >> p.pages.page_shift, p.err);
        const int32_t row = key & (p.pages.page_size - 1);
#pragma unroll
        for (int which = 0; which < 2; ++which, ++pos) {
          const uint32_t slot = pos % C::NSLOT;
          if (!mbar_wait(&sh.empty[slot], ((pos / C::NSLOT) & 1) ^ 1, abort)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], C::TILE + (E4M3 ? kFewTile * 2 : 0));
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
    ok = __all_sync(0xffffffffu, ok);
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
      const int32_t rows = (int32_t)min((int64_t)x.n * p.group - (int64_t)x.blk * kFewRows, (int64_t)kFewRows);
      const int mt = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);  // row tiles; kWarps / mt warps share each
      const int rt = warp & (mt - 1), kg = warp / mt, share = kWarps / mt;
      const bool works = rt * 16 < rows;
      // this lane's two rows
      int32_t tok[2], hd[2];
      bool live[2];
      int32_t klo[2], khi[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t rr = rt * 16 + r + i * 8;
        live[i] = rr < rows;
        const int64_t row = (int64_t)x.blk * kFewRows + min(rr, rows - 1);
        tok[i] = (int32_t)(row / p.group);
        hd[i] = x.kh * p.group + (int32_t)(row - (int64_t)tok[i] * p.group);
        band_keys(tok[i], tok[i], x.n, x.sk, p.win_left, p.win_right, &klo[i], &khi[i]);
      }
      uint32_t qf[C::KSTEPS][4];
      if (works) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __nv_bfloat16* qa = p.q + (int64_t)(x.q0 + tok[i]) * p.q_rs + (int64_t)hd[i] * p.q_hs;
          if constexpr (E4M3) {
#pragma unroll
            for (int s = 0; s < C::KSTEPS / 4; ++s) {
              const int d0 = (C::KSTEPS == 4 ? c : 2 * c + s) * 16;  // 16 elements of this lane
              uint4 u[2];
#pragma unroll
              for (int k = 0; k < 2; ++k)
                u[k] = live[i] && d0 < D && in_span(p.q_span, qa + d0 + k * 8, 16, p.err)
                           ? __ldg(reinterpret_cast<const uint4*>(qa + d0 + k * 8))
                           : make_uint4(0, 0, 0, 0);
              const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // elements 1, 3 then 0, 2 of each four
                qf[s * 4 + k][i] = __byte_perm(w[2 * k], w[2 * k + 1], 0x7632);
                qf[s * 4 + k][2 + i] = __byte_perm(w[2 * k], w[2 * k + 1], 0x5410);
              }
            }
          } else {
#pragma unroll
            for (int s = 0; s < C::KSTEPS / 2; ++s) {
              const int d0 = (s >> 1) * 64 + (2 * c + (s & 1)) * 8;
              const uint4 u = live[i] && d0 < D && in_span(p.q_span, qa + d0, 16, p.err)
                                  ? __ldg(reinterpret_cast<const uint4*>(qa + d0))
                                  : make_uint4(0, 0, 0, 0);
              qf[s * 2][i] = u.x;
              qf[s * 2][2 + i] = u.y;
              qf[s * 2 + 1][i] = u.z;
              qf[s * 2 + 1][2 + i] = u.w;
            }
          }
        }
      }
      float o[C::NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < C::NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
      // keys that every row of the unit sees: no select needed
      int32_t all_lo, all_hi;
      {
        int32_t a, e;
        band_keys(x.u.t1, x.u.t1, x.n, x.sk, p.win_left, p.win_right, &all_lo, &e);
        band_keys(x.u.t0, x.u.t0, x.n, x.sk, p.win_left, p.win_right, &a, &all_hi);
      }
      const int32_t tiles = min(x.j1, x.u.tiles);
      for (int32_t j = x.j0; j < tiles; ++j, pos += 2) {
        const uint32_t ks = pos % C::NSLOT, vs = (pos + 1) % C::NSLOT;
        if (!mbar_wait(&sh.full[ks], (pos / C::NSLOT) & 1, abort)) {
          ok = false;
          break;
        }
        __syncwarp();
        const uint32_t kt = smem_addr(ring + ks * C::TILE), vt = smem_addr(ring + vs * C::TILE);
        const uint32_t ksc = smem_addr(scales + ks * C::SCALES), vsc = smem_addr(scales + vs * C::SCALES);
        const int32_t key0 = (x.u.tile0 + j) * kFewTile;
        const bool edge = key0 < all_lo || key0 + kFewTile > all_hi;
        // rows of V that no row of the unit sees may hold anything: cleared
        const bool vedge = key0 < x.u.lo || key0 + kFewTile > x.u.hi;
        bool v_here = false;
        // the 16-key steps of this warp: kg, kg + share, ...
#pragma unroll 1
        for (int a = kg * 16; a < kFewTile; a += share * 16) {
          float s[2][4];
          if (works) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
              const uint32_t row = a + h * 8 + r;
              if constexpr (E4M3) {
                uint32_t sc;
                asm volatile("ld.shared.u16 %0, [%1];" : "=r"(sc) : "r"(ksc + scale_at(row, box_shift)) : "memory");
                const Factor f = factor_of(sc | (sc << 16));
                const bool rest = __any_sync(0xffffffffu, f.rest != 0x3f803f80u);
#pragma unroll
                for (int i = 0; i < C::KSTEPS / 4; ++i) {
                  const uint4 u = lds128(kt + swz(row, (C::KSTEPS == 4 ? c : 2 * c + i) * 16));
                  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    uint32_t b0 = mul_pair(raw_pair(w[k]), f.f);
                    uint32_t b1 = mul_pair(raw_pair(w[k] << 8), f.f);
                    if (rest) {
                      b0 = mul_pair(b0, f.rest);
                      b1 = mul_pair(b1, f.rest);
                    }
                    mma16816(s[h], qf[i * 4 + k], b0, b1);
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < C::KSTEPS / 2; ++i) {
                  const uint4 u = lds128(kt + (i >> 1) * C::CHUNK + swz(row, (2 * c + (i & 1)) * 16));
                  mma16816(s[h], qf[2 * i], u.x, u.y);
                  mma16816(s[h], qf[2 * i + 1], u.z, u.w);
                }
              }
            }
          }
          if (a + share * 16 >= kFewTile) {  // the warp's last step on this K tile
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[ks]);
          }
          uint32_t pf[4];
          if (works) {
            // columns of this lane: keys a + h*8 + 2c, +1
            float mx[2] = {-INFINITY, -INFINITY}, sub[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float v = s[h][e] * p.scale_log2;
                if (edge) {
                  const int32_t key = key0 + a + h * 8 + 2 * c + (e & 1);
                  v = key >= klo[e >> 1] && key < khi[e >> 1] ? v : -INFINITY;
                }
                s[h][e] = v;
                mx[e >> 1] = fmaxf(mx[e >> 1], v);
              }
            bool grow = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
              mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
              // the maximum follows only when it grew by more than 2^8: o and l
              // carry the same factor, so nothing is lost
              grow |= mx[i] > m[i] + 8.f;
            }
            if (__any_sync(0xffffffffu, grow)) {
              float al[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[i], mx[i]);
                al[i] = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
                m[i] = mn;
                l[i] *= al[i];
              }
#pragma unroll
              for (int t = 0; t < C::NT; ++t) {
                o[t][0] *= al[0];
                o[t][1] *= al[0];
                o[t][2] *= al[1];
                o[t][3] *= al[1];
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) sub[i] = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 4; ++e) s[h][e] = ex2(s[h][e] - sub[e >> 1]);
              l[0] += s[h][0] + s[h][1];
              l[1] += s[h][2] + s[h][3];
              pf[2 * h] = pack_bf16x2(s[h][0], s[h][1]);
              pf[2 * h + 1] = pack_bf16x2(s[h][2], s[h][3]);
            }
          }
          if (!v_here) {
            v_here = mbar_wait(&sh.full[vs], ((pos + 1) / C::NSLOT) & 1, abort);
            ok = ok && v_here;
          }
          if (!ok) break;
          __syncwarp();
          if (!works) continue;
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;  // keys 2c, 2c+1 and 2c+8, 2c+9
          if (vedge) {
            auto in = [&](int k) { return key0 + a + k >= x.u.lo && key0 + a + k < x.u.hi; };
            keep0 = (in(2 * c) ? 0xffffu : 0u) | (in(2 * c + 1) ? 0xffff0000u : 0u);
            keep1 = (in(2 * c + 8) ? 0xffffu : 0u) | (in(2 * c + 9) ? 0xffff0000u : 0u);
          }
          if constexpr (E4M3) {
            const uint32_t sc0 = lds32(vsc + scale_at(a + 2 * c, box_shift)) & keep0;
            const uint32_t sc1 = lds32(vsc + scale_at(a + 2 * c + 8, box_shift)) & keep1;
            const Factor f0 = factor_of(sc0), f1 = factor_of(sc1);
            const bool rest = __any_sync(0xffffffffu, f0.rest != 0x3f803f80u || f1.rest != 0x3f803f80u);
            uint32_t w[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t row = a + 2 * c + (k & 1) + (k >> 1) * 8;
              if constexpr (D == 128) {
                const uint4 u = lds128(vt + swz(row, r * 16));
                w[k][0] = u.x;
                w[k][1] = u.y;
                w[k][2] = u.z;
                w[k][3] = u.w;
              } else if constexpr (D == 64) {
                const uint2 u = lds64(vt + swz(row, r * 8));
                w[k][0] = u.x;
                w[k][1] = u.y;
              } else {
#pragma unroll
                for (int i = 0; i < 3; ++i) w[k][i] = lds32(vt + swz(row, r * 12 + i * 4));
              }
            }
#pragma unroll
            for (int t = 0; t < C::NT; ++t) {
              constexpr uint32_t kSel[4] = {0x4000u, 0x5010u, 0x6020u, 0x7030u};
              uint32_t b0 = mul_pair(raw_pair(__byte_perm(w[0][t >> 2], w[1][t >> 2], kSel[t & 3])), f0.f);
              uint32_t b1 = mul_pair(raw_pair(__byte_perm(w[2][t >> 2], w[3][t >> 2], kSel[t & 3])), f1.f);
              if (rest) {
                b0 = mul_pair(b0, f0.rest);
                b1 = mul_pair(b1, f1.rest);
              }
              mma16816(o[t], pf, b0, b1);
            }
          } else {
            const uint32_t row = a + (lane & 15);
#pragma unroll
            for (int t = 0; t < C::NT; t += 2) {
              uint32_t b[4];
              ldsm_x4_t(b, vt + (t >> 3) * C::CHUNK + swz(row, ((t & 7) + (lane >> 4)) * 16));
              mma16816(o[t], pf, b[0] & keep0, b[1] & keep1);
              mma16816(o[t + 1], pf, b[2] & keep0, b[3] & keep1);
            }
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[vs]);
      }
      if (!ok) break;
      // row sums over the four lanes of a row
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      }
      // join the warps that share these rows
      for (int step = share >> 1; step >= 1 && ok; step >>= 1) {
        float* buf = xchg + ((kg & (step - 1)) * mt + rt) * (C::XCHG / 4) + lane;
        if (kg >= step && kg < 2 * step) {
#pragma unroll
          for (int t = 0; t < C::NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) buf[(t * 4 + e) * 32] = o[t][e];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            buf[(C::NT * 4 + i) * 32] = m[i];
            buf[(C::NT * 4 + 2 + i) * 32] = l[i];
          }
        }
        mbar_arrive(&sh.join);
        if (!mbar_wait(&sh.join, joins++ & 1, abort)) {
          ok = false;
          break;
        }
        if (kg < step) {
          float a0[2], a1[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m1 = buf[(C::NT * 4 + i) * 32], mn = fmaxf(m[i], m1);
            a0[i] = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
            a1[i] = mn == -INFINITY ? 1.f : ex2(m1 - mn);
            m[i] = mn;
            l[i] = l[i] * a0[i] + buf[(C::NT * 4 + 2 + i) * 32] * a1[i];
          }
#pragma unroll
          for (int t = 0; t < C::NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = o[t][e] * a0[e >> 1] + buf[(t * 4 + e) * 32] * a1[e >> 1];
        }
        mbar_arrive(&sh.join);
        if (!mbar_wait(&sh.join, joins++ & 1, abort)) {
          ok = false;
          break;
        }
      }
      if (!ok) break;
      if (kg != 0 || !works) continue;
      // column of element e of n-tile t: d_of(t, e & 1)
      auto d_of = [&](int t, int e) { return E4M3 ? (2 * c + e) * (D / 8) + t : t * 8 + 2 * c + e; };
      if (x.whole()) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!live[i]) continue;
          const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);  // no key: 0; NaN stays
          __nv_bfloat16* oa = p.out + (int64_t)(x.q0 + tok[i]) * p.o_rs + (int64_t)hd[i] * p.o_hs;
          if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int t = 0; t < C::NT; t += 4) {
                const uint2 w = make_uint2(pack_bf16x2(o[t][2 * i + e] * inv, o[t + 1][2 * i + e] * inv),
                                           pack_bf16x2(o[t + 2][2 * i + e] * inv, o[t + 3][2 * i + e] * inv));
                __nv_bfloat16* a = oa + d_of(t, e);
                if (in_span(p.out_span, a, 8, p.err)) *reinterpret_cast<uint2*>(a) = w;
              }
          } else {
#pragma unroll
            for (int t = 0; t < C::NT; ++t) {
              __nv_bfloat16* a = oa + d_of(t, 0);
              if (in_span(p.out_span, a, 4, p.err))
                *reinterpret_cast<uint32_t*>(a) = pack_bf16x2(o[t][2 * i] * inv, o[t][2 * i + 1] * inv);
            }
          }
          float* la = p.lse + (int64_t)hd[i] * p.total_q + x.q0 + tok[i];
          if (c == 0 && in_span(p.lse_span, la, 4, p.err))
            *la = l[i] == 0.f ? -INFINITY : (m[i] + __log2f(l[i])) * 0.69314718055994531f;
        }
      } else {
        const int64_t slot = 2 * (int64_t)blockIdx.x + (x.begins() ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!live[i]) continue;
          const int64_t row = slot * parts.rows + rt * 16 + r + i * 8;
          float* oa = parts.o + row * D;
          if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int t = 0; t < C::NT; t += 4)
                *reinterpret_cast<float4*>(oa + d_of(t, e)) =
                    make_float4(o[t][2 * i + e], o[t + 1][2 * i + e], o[t + 2][2 * i + e], o[t + 3][2 * i + e]);
          } else {
#pragma unroll
            for (int t = 0; t < C::NT; ++t)
              *reinterpret_cast<float2*>(oa + d_of(t, 0)) = make_float2(o[t][2 * i], o[t][2 * i + 1]);
          }
          if (c == 0) *reinterpret_cast<float2*>(parts.ml + row * 2) = make_float2(m[i], l[i]);
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
  return launch_overlapped(kern, (unsigned)(L.sms * kFewCtasPerSm), kThreads, C::SMEM, stream, L.few_k, L.few_v, L.few_ks,
                           L.few_vs, L.p, L.few, take);
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
