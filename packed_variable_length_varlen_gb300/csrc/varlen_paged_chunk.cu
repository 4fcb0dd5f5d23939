// varlen_paged_chunk.cu -- attention over the paged cache for many query rows:
// chunks of a prompt.
//
// Bound: 4 D operations for every visible (row, key) pair on the tensor cores;
// the keys are read from L2 by most units.  Measured at D = 128: four chunks of
// 1500..2048 tokens (32 heads, 8 key heads) over 4096..16384 bf16 keys, causal,
// 850-927 us across machines, 1160-1260 TFLOP/s; 250 tokens of 56 heads over 77000
// E4M3 keys 474-494 us, 1115-1160 TFLOP/s.  Under ncu two chunks of 2048 tokens
// over 8192 bf16 keys have the tensor pipe active 52% of the time (issue slots 30%,
// the tensor core's operand reads 39% of shared memory's cycles), 250 tokens of
// 56 heads over 40000 E4M3 keys 46% (issue slots 46%, operand reads 35% and the
// conversion 22%): no unit is full, the softmax and the products of a half wait
// for one another, and with two halves in flight they overlap only in part.  The
// structure is the packed
// forward's (varlen_fwd.cu): a unit is two halves A and B of 128 rows that share
// every 128-key tile, S and P of a half in one TMEM region, the next S of a
// half issued right behind its P V product, so that the tensor core works on one
// half while the other's softmax runs.  What differs:
//   * A row is one (query token, head of the key head's group), token-major,
//     so that all heads of a group share the keys' way through shared memory.
//     A half holds the rows of 128 / group whole tokens; TMA loads them as one
//     box {64 columns, group heads, 128 / group tokens}.
//   * Key tiles are gathered from pages: 128 / page_size boxes for pages of less
//     than a tile, issued by as many lanes of the producer warp.
//   * Units are shared out by tiles (varlen_paged_walk.cuh), so that a few units over
//     a long cache fill all SMs; a unit that a CTA does not hold whole goes to
//     the workspace and is joined.
//   * E4M3: a warpgroup turns the codes of each tile into bf16 in the layout that
//     the products read: s eeee mmm moved to s 0000eeee mmm0000 is code * 2^-120,
//     times 2^120 * scale; with power-of-two scales the result is exact, so the
//     softmax does not know of scales at all.
//   * Rows of V outside the unit's keys are cleared (by the converting warps, or
//     for bf16 by warps 2 and 3) before the product reads them: they may hold
//     anything, and 0 * NaN would poison O.
//
// TREE, drafted trees: in tiles with new rows (the last of a unit) a row's scores are
// selected by its mask's bits, and rows of V whose bit no row of the unit has are cleared
// too: warps 2 and 3, or the converting warps, unite the unit's masks.  The masks are
// brought into L1 while the context's tiles are worked through.  The kernel is sensitive to
// its code's size (one stall in eight waits for instructions), so this form has one select
// for all masks, and softmax and conversion read their piece where it lies instead of keeping
// it in registers: 64 trees of 64 rows, 4 heads a key head, over 8192 keys 458 us in bf16
// and 501 in E4M3, where the causal band takes 470 and 515 (a second select in the
// softmax and pieces in registers: 488 and 641).  256 rows of 7 heads over 77000 bf16
// keys 456-474 from a graph, 497-523 a call.
//
// P is rounded to bf16, V's type, which the second product asks for: each weight
// is off by at most 2^-9 of its binade, O by 2e-3 to 2.4e-3 relative to 64 bits
// where rounding O alone gives 1.65e-3.  The sum l takes P before that rounding.  A
// second bf16 part, as in the kernel for few rows, would be half as many tensor
// operations again where those are the bound.
//
// Warps: 0 producer, 1 MMA issuer, 2 and 3 clearing (bf16), 4..7 softmax of half
// A, 8..11 of half B, 12..15 converting (E4M3).  The producer walks the CTA's
// part and hands each piece to the other roles through a ring in shared memory.
#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

// Tiles per CTA when there are few.  With trees the last one takes longer, and each is better off
// alone: 4 trees of 13 rows under a window of 1024 18.4 and 15.3 us, one over 500 keys 18.9 and 15.3.
template <bool TREE>
constexpr int kLeastTiles = TREE ? 1 : 2;
constexpr int kPieces = 4;      // pieces that the producer may be ahead

template <int D, bool E4M3>
struct ChunkCfg {
  static constexpr int THREADS = E4M3 ? 512 : 384;
  static constexpr int NC = (D + 63) / 64;           // 64-column chunks of a bf16 tile
  static constexpr int CHUNK = 128 * 128;            // 128 rows x 128 bytes
  static constexpr int TILE = NC * CHUNK;            // one Q / K / V tile in bf16
  static constexpr int NSLOT = E4M3 ? 4 : (NC == 1 ? 8 : 4);  // bf16 K/V ring (even for bf16: K and V slots alternate)
  static constexpr int NRAW = E4M3 ? 2 : 0;          // ring of codes
  static constexpr int SCALES = 1024;                // page pieces of at least 16 keys, 128 bytes apart
  static constexpr int O_COL = 256;                  // TMEM column of O_A (O_B at +128)
  static constexpr int KSTEPS = D / 16;
  static constexpr int SMEM = 1024 + TILE * (2 + NSLOT) + NRAW * (CHUNK + SCALES);
  // Registers (threads x registers at launch is all there is to share out):
  // bf16 384 x 168 = 128 x (120 + 192 + 192); E4M3 512 x 128 = 128 x (80 + 184 + 184 + 64).
  static constexpr uint32_t REGS_LAUNCH = E4M3 ? 128 : 168, REGS_CTL = E4M3 ? 80 : 120, REGS_SOFTMAX = E4M3 ? 184 : 192,
                            REGS_CONVERT = 64;
  static_assert(REGS_CTL + 2 * REGS_SOFTMAX + (E4M3 ? REGS_CONVERT : 0) <= (THREADS / 128) * REGS_LAUNCH,
                "warpgroup register split exceeds the launch allocation");
};

struct ChunkShared {
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t mma_done;
  uint64_t kv_full[8], kv_empty[8], v_ok[8];
  uint64_t raw_full[2], raw_empty[2];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint32_t tmem_base;
  int abort;
  PagedPiece piece[kPieces];
  PagedStart start;
};
static_assert(sizeof(ChunkShared) <= 1024, "barrier block too large");

// The next piece from the ring (b < 0: there is none); false on giving up.
// WARP: a whole warp reads it, and gives up as one; else a single thread does.
template <bool WARP>
struct PieceReader {
  uint32_t n = 0;
  __device__ __forceinline__ bool next(ChunkShared& sh, PagedPiece& x, volatile int* abort) {
    const uint32_t i = n % kPieces, parity = (n / kPieces) & 1;
    if (!(WARP ? mbar_wait_warp(&sh.piece_full[i], parity, abort) : mbar_wait(&sh.piece_full[i], parity, abort))) return false;
    x = sh.piece[i];
    mbar_arrive(&sh.piece_empty[i]);
    ++n;
    return x.b >= 0;
  }
  // The same for a reader that leaves the piece where it lies until it calls done().
  __device__ __forceinline__ bool wait(ChunkShared& sh, volatile int* abort) {
    const uint32_t i = n % kPieces, parity = (n / kPieces) & 1;
    return mbar_wait_warp(&sh.piece_full[i], parity, abort) && sh.piece[i].b >= 0;
  }
  __device__ __forceinline__ void done(ChunkShared& sh) {
    mbar_arrive(&sh.piece_empty[n % kPieces]);
    ++n;
  }
};

__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&x);
}

template <int D, bool E4M3, bool TREE>
__global__ void __launch_bounds__(ChunkCfg<D, E4M3>::THREADS, 1)
    varlen_paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_ks,
                              const __grid_constant__ CUtensorMap tm_vs, const PagedParams p, const PagedParts parts,
                              int32_t take) {
  using C = ChunkCfg<D, E4M3>;
  using ChunkGeom = PagedGeom<kChunkRows, kChunkTile, true, TREE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_addr(smem) & 1023u) != 0) {
    paged_refuse(p, parts);
    return;
  }
  ChunkShared& sh = *reinterpret_cast<ChunkShared*>(smem);
  uint8_t* q_smem = smem + 1024;  // Q_A then Q_B
  uint8_t* ring = q_smem + 2 * C::TILE;
  uint8_t* raw = ring + C::NSLOT * C::TILE;          // codes
  uint8_t* scales = raw + C::NRAW * C::CHUNK;
  volatile int* abort = &sh.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kReaders = 1 + 256 + (E4M3 ? 128 : 64);  // threads that read each piece

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 1);
    mbar_init(&sh.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 128);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.mma_done, 1);
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&sh.kv_full[i], E4M3 ? 128 : 1);
      mbar_init(&sh.kv_empty[i], 1);
      mbar_init(&sh.v_ok[i], 64);
    }
    for (int i = 0; i < C::NRAW; ++i) {
      mbar_init(&sh.raw_full[i], 1);
      mbar_init(&sh.raw_empty[i], 128);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&sh.piece_full[i], 1);
      mbar_init(&sh.piece_empty[i], kReaders);
    }
    sh.abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&sh.tmem_base, 512);
  tc_fence_before();
  dependency_wait();  // nothing above reads or writes global memory
  paged_start<ChunkGeom>(sh.start, p, take, kLeastTiles<TREE>);
  __syncthreads();
  tc_fence_after();
  dependents_may_launch();
  const uint32_t tmem = sh.tmem_base;
  const int32_t half_tokens = ChunkGeom::half_tokens(p);

  if (warp < 4) {
    warpgroup_set_regs<C::REGS_CTL, C::REGS_LAUNCH>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        clear_join(p, parts);
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      const int box_shift = min(p.pages.page_shift, 7);
      const int pieces = kChunkTile >> box_shift;  // page pieces of a tile
      const int piece = lane % pieces, cc = lane / pieces;
      const bool loads = cc < (E4M3 ? 1 : C::NC), loads_scale = E4M3 && lane < pieces;
      constexpr int kRing = E4M3 ? C::NRAW : C::NSLOT;
      uint64_t* full = E4M3 ? sh.raw_full : sh.kv_full;
      uint64_t* empty = E4M3 ? sh.raw_empty : sh.kv_empty;
      const uint32_t q_bytes = 2u * C::NC * 128u * (uint32_t)(half_tokens * p.group);
      PagedWalk<ChunkGeom> walk;
      PagedPiece x;
      uint32_t pos = 0, q_loads = 0, handed = 0;
      bool ok = true;
      walk.init(sh.start, p, take);
      while (ok) {
        const bool more = walk.next(p, x);
        if (!more) x.b = -1;
        const uint32_t slot = handed % kPieces;
        if (!mbar_wait_warp(&sh.piece_empty[slot], ((handed / kPieces) & 1) ^ 1, abort)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) {
          if (more) paged_note(p, parts, sh.start, walk, x);
          sh.piece[slot] = x;
          mbar_arrive(&sh.piece_full[slot]);
        }
        ++handed;
        if (!more) break;
        const int32_t tiles = min(x.j1, x.u.tiles);
        if (x.j0 >= tiles) continue;  // no key: nothing to load
        if (q_loads > 0 && !mbar_wait_warp(&sh.q_empty, (q_loads - 1) & 1, abort)) {
          ok = false;
          break;
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, q_bytes);
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int c = 0; c < C::NC; ++c)
              tma_load_4d(q_smem + hf * C::TILE + c * C::CHUNK, &tm_q, &sh.q_full, c * 64, 0, x.kh,
                          x.q0 + x.u.t0 + hf * half_tokens);
        }
        ++q_loads;
        for (int32_t j = x.j0; ok && j < tiles; ++j) {
          const int32_t key = (x.u.tile0 + j) * kChunkTile + (piece << box_shift);
          int32_t page = p.pages.num_pages;
          if (loads && key < x.u.hi && key + (1 << box_shift) > x.u.lo)
            page = page_at<TREE>(p.pages, x.b, key >> p.pages.page_shift, p.err);
          const int32_t row = key & (p.pages.page_size - 1);
#pragma unroll
          for (int which = 0; which < 2; ++which, ++pos) {
            const uint32_t s = pos % kRing;
            if (!mbar_wait_warp(&empty[s], ((pos / kRing) & 1) ^ 1, abort)) {
              ok = false;
              break;
            }
            // (failure test: CTA 0 leaves one load out)
            if (blockIdx.x == 0 && (int64_t)pos == (int64_t)p.debug_skip_many) continue;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], E4M3 ? C::CHUNK + kChunkTile * 2 : C::TILE);
            __syncwarp();
            uint8_t* dst = (E4M3 ? raw + s * C::CHUNK : ring + s * C::TILE) + cc * C::CHUNK + (piece << box_shift) * 128;
            if (loads) tma_load_4d(dst, which ? &tm_v : &tm_k, &full[s], cc * 64, x.kh, row, page);
            if (loads_scale)
              tma_load_3d(scales + s * C::SCALES + piece * 128, which ? &tm_vs : &tm_ks, &full[s], row, x.kh, page);
          }
        }
      }
      if (*abort && lane == 0) {
        // every copy in flight lands before the CTA's shared memory is released (bounded)
        int dummy = 0;
        for (uint32_t s = 0; s < kRing && s < pos; ++s) {
          const uint32_t last = pos - 1 - ((pos - 1 - s) % kRing);
          mbar_wait(&full[s], (last / kRing) & 1, &dummy, 100000000ull);
        }
        if (q_loads > 0) mbar_wait(&sh.q_full, (q_loads - 1) & 1, &dummy, 100000000ull);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0) {
        constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t kIdescO = idesc_bf16_f32(128, D, false, true);
        const uint32_t qlo = sw128_desc_lo(smem_addr(q_smem), 16);     // Q_A (Q_B at +TILE), K-major A
        const uint32_t rK = sw128_desc_lo(smem_addr(ring), 16);        // slot 0 as K-major B
        const uint32_t rV = sw128_desc_lo(smem_addr(ring), C::CHUNK);  // slot 0 as MN-major B
        auto issue_s = [&](int hf, uint32_t slot) {
#pragma unroll
          for (int kk = 0; kk < C::KSTEPS; ++kk) {
            const uint32_t off = ((kk >> 2) * C::CHUNK + (kk & 3) * 32) >> 4;
            mma_ss_lo(tmem + hf * 128, qlo + ((hf * C::TILE) >> 4) + off, rK + ((slot * C::TILE) >> 4) + off, kIdescS,
                      kk > 0 ? 1u : 0u);
          }
          mma_commit(&sh.s_full[hf]);
        };
        // O += P V over the 16-row steps of the keys below `nk` (TREE: over all of them, as
        // only a unit's last tile has others, whose P is 0 and whose rows of V are clear: a
        // branch before each product costs 3 to 7% of the whole)
        auto issue_pv = [&](int hf, uint32_t slot, bool first, int nk) {
#pragma unroll
          for (int kk = 0; kk < kChunkTile / 16; ++kk)
            if (TREE || kk < nk)
              mma_ts_lo(tmem + C::O_COL + hf * 128, tmem + hf * 128 + kk * 8, rV + ((slot * C::TILE + kk * 2048) >> 4),
                        kIdescO, (!first || kk > 0) ? 1u : 0u);
          mma_commit(&sh.pv_done[hf]);
        };
        PieceReader<false> pieces;
        PagedPiece x;
        uint32_t q_loads = 0, pos = 0, g[2] = {0, 0};  // steps of each half so far
        bool ok = true;
        while (ok && pieces.next(sh, x, abort)) {
          const int32_t tiles = min(x.j1, x.u.tiles) - x.j0;
          if (tiles <= 0) continue;
          const int nh = x.u.t1 - x.u.t0 >= half_tokens ? 2 : 1;  // halves that have rows
          if (!mbar_wait(&sh.q_full, q_loads & 1, abort)) break;
          ++q_loads;
          {
            const uint32_t s = pos % C::NSLOT;
            if (!mbar_wait(&sh.kv_full[s], (pos / C::NSLOT) & 1, abort)) break;
            tc_fence_after();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
              if (hf < nh) issue_s(hf, s);
            mma_commit(&sh.kv_empty[s]);
            if (tiles == 1) mma_commit(&sh.q_empty);
          }
          for (int32_t j = 0; j < tiles; ++j) {
            const bool more = j + 1 < tiles;
            const uint32_t vpos = pos + 2 * j + 1, vs = vpos % C::NSLOT, kpos = vpos + 1, ks = kpos % C::NSLOT;
            if (!mbar_wait(&sh.kv_full[vs], (vpos / C::NSLOT) & 1, abort)) { ok = false; break; }
            if (!E4M3 && !mbar_wait(&sh.v_ok[vs], (vpos / C::NSLOT) & 1, abort)) { ok = false; break; }
            const int nk = (min(kChunkTile, x.u.hi - (x.u.tile0 + x.j0 + j) * kChunkTile) + 15) >> 4;
            if (more && !mbar_wait(&sh.kv_full[ks], (kpos / C::NSLOT) & 1, abort)) { ok = false; break; }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              if (hf >= nh) break;
              if (!mbar_wait(&sh.p_full[hf], (g[hf] + j) & 1, abort)) { ok = false; break; }
              tc_fence_after();
              issue_pv(hf, vs, j == 0, nk);
              if (more) issue_s(hf, ks);
            }
            if (!ok) break;
            mma_commit(&sh.kv_empty[vs]);
            if (more) {
              mma_commit(&sh.kv_empty[ks]);
              if (j + 2 == tiles) mma_commit(&sh.q_empty);
            }
          }
          g[0] += tiles;
          if (nh == 2) g[1] += tiles;
          pos += 2 * tiles;
        }
        // Drain: every MMA this thread issued completes before TMEM is freed.
        mma_commit(&sh.mma_done);
        int dummy = 0;
        mbar_wait(&sh.mma_done, 0, &dummy);
      }
    } else if constexpr (!E4M3) {
      // ---------------------------------------------------------- clearing (bf16)
      PieceReader<true> pieces;
      PagedPiece x;
      uint32_t pos = 0;
      bool ok = true;
      const int t = threadIdx.x - 64;  // 0..63
      while (ok && pieces.next(sh, x, abort)) {
        const int32_t tiles = min(x.j1, x.u.tiles);
        const int32_t unit_lo = TREE ? tree_unit_lo(p, x) : x.u.lo;
        for (int32_t j = x.j0; j < tiles; ++j, pos += 2) {
          const uint32_t vpos = pos + 1, s = vpos % C::NSLOT;
          const int32_t key0 = (x.u.tile0 + j) * kChunkTile;
          const bool tail = TREE && key0 + kChunkTile > x.sk - x.n;  // has new rows
          const int lo = min(max(unit_lo - key0, 0), kChunkTile), hi = min(x.u.hi - key0, kChunkTile);
          uint32_t any[4] = {0, 0, 0, 0};
          if (tail) tree_unit_bits(p, x, unit_lo, key0, any);
          if (!mbar_wait_warp(&sh.kv_full[s], (vpos / C::NSLOT) & 1, abort)) { ok = false; break; }
          uint4* base = reinterpret_cast<uint4*>(ring + s * C::TILE);
          if (tail) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              for (int u = t; any[k] != ~0u && u < 32 * 8; u += 64)
                if (((any[k] >> (u >> 3)) & 1u) == 0)
#pragma unroll
                  for (int c = 0; c < C::NC; ++c) base[c * (C::CHUNK / 16) + k * 256 + u] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          } else if (lo > 0 || hi < kChunkTile) {
#pragma unroll
            for (int c = 0; c < C::NC; ++c) {
              for (int u = t; u < lo * 8; u += 64) base[c * (C::CHUNK / 16) + u] = make_uint4(0, 0, 0, 0);
              for (int u = hi * 8 + t; u < kChunkTile * 8; u += 64) base[c * (C::CHUNK / 16) + u] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          mbar_arrive(&sh.v_ok[s]);
        }
      }
    }
  } else if (warp < 12) {
    warpgroup_set_regs<C::REGS_SOFTMAX, C::REGS_LAUNCH>();
    // ------------------------------------------------------------ softmax
    const int hf = (warp - 4) >> 2;  // 0: half A (warps 4..7), 1: half B (warps 8..11)
    const int row = (warp & 3) * 32 + lane;  // TMEM lane = row within the half
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = hf * 128, o_col = C::O_COL + hf * 128;
    const float c2 = p.scale_log2;
    const int32_t row_tok = row / p.group, row_head = row - row_tok * p.group;
    PieceReader<true> pieces;
    PagedPiece copy;
    uint32_t g = 0;
    bool ok = true;
    while (ok && (TREE ? pieces.wait(sh, abort) : pieces.next(sh, copy, abort))) {
      // (TREE needs a few registers more: what the piece says is read again where it is needed)
      const PagedPiece& x = TREE ? sh.piece[pieces.n % kPieces] : copy;
      const int32_t tok = x.u.t0 + hf * half_tokens + row_tok;
      const bool live = row_tok < half_tokens && tok <= x.u.t1;
      const int32_t tiles = min(x.j1, x.u.tiles) - x.j0;
      if (hf == 1 && x.u.t1 - x.u.t0 < half_tokens) {  // no rows in this half
        if (TREE) pieces.done(sh);
        continue;
      }
      float m_use = -INFINITY, l = 0.f;
      // a row that is none sees all keys: what it computes goes nowhere, and its
      // warp is spared the selects
      int32_t key_lo = 0, key_hi = INT32_MAX;
      const int32_t ctx = x.sk - x.n, edge = min(ctx, x.u.hi);  // (edge: of the keys that every row sees)
      if (live && TREE) {
        key_lo = tree_lo(p, (int64_t)x.q0 + tok, ctx);
        key_hi = x.u.hi;
      } else if (live) {
        band_keys(tok, tok, x.n, x.sk, p.win_left, p.win_right, &key_lo, &key_hi);
      }
      const int32_t key0 = (x.u.tile0 + x.j0) * kChunkTile;
      // TREE: the masks come near while the context's tiles are worked through
      if (TREE && live && key0 + tiles * kChunkTile > ctx) tree_prefetch(p, (int64_t)x.q0 + tok);
      for (int32_t j = 0; j < tiles; ++j) {
        if (!mbar_wait_warp(&sh.s_full[hf], (g + j) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        uint32_t s[128];
        {
          uint32_t(&s0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[0]);
          uint32_t(&s1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[32]);
          uint32_t(&s2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[64]);
          uint32_t(&s3)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[96]);
          const uint32_t ta = tmem + lane_off + s_col;
          tmem_ld32(ta + 0, s0);
          tmem_ld32(ta + 32, s1);
          tmem_ld32(ta + 64, s2);
          tmem_ld32(ta + 96, s3);
          tmem_wait_ld();
        }
        float v[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(s[i]);
        // keys that the row does not see are set to -inf by select
        const int32_t lim = key_hi - (key0 + j * kChunkTile), lim_lo = key_lo - (key0 + j * kChunkTile);
        if (TREE) {
          if (key0 + (j + 1) * kChunkTile > edge || __any_sync(0xffffffffu, lim_lo > 0)) {  // new rows, or a window's edge
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t see = live ? tree_bits(p, (int64_t)x.q0 + tok, key0 + j * kChunkTile + 32 * k - ctx) &
                                              bits_between(lim_lo - 32 * k, lim - 32 * k) : ~0u;
#pragma unroll
              for (int i = 0; i < 32; ++i) v[32 * k + i] = (see & (1u << i)) != 0 ? v[32 * k + i] : -INFINITY;
            }
          }
        } else if (__any_sync(0xffffffffu, lim_lo > 0)) {
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] = (i < lim && i >= lim_lo) ? v[i] : -INFINITY;
        } else if (__any_sync(0xffffffffu, lim < kChunkTile)) {
#pragma unroll
          for (int i = 0; i < 128; ++i) v[i] = (i < lim) ? v[i] : -INFINITY;
        }
        float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
        for (int i = 0; i < 128; i += 8) {
          m0 = fmax3(m0, v[i], v[i + 1]);
          m1 = fmax3(m1, v[i + 2], v[i + 3]);
          m2 = fmax3(m2, v[i + 4], v[i + 5]);
          m3 = fmax3(m3, v[i + 6], v[i + 7]);
        }
        const float m_new = fmaxf(m_use, fmaxf(fmax3(m0, m1, m2), m3) * c2);
        float alpha = 1.f;
        bool rescale = false;
        if (j == 0) {
          m_use = m_new;
        } else if (m_new > m_use + 8.0f) {
          alpha = ex2(m_use - m_new);
          m_use = m_new;
          rescale = true;
        }
        // a row that has seen no key yet keeps m = -inf; subtracting 0 then
        // gives P = exp2(-inf) = 0 instead of NaN
        const float m_sub = m_use == -INFINITY ? 0.f : m_use;
        const float2 cc2 = make_float2(c2, c2), negm = make_float2(-m_sub, -m_sub);
        float2 ra = make_float2(0.f, 0.f), rb = make_float2(0.f, 0.f);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {  // P in two halves, written over S values that were consumed
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = hh * 64 + 2 * i;
            float2 t2 = ffma2(make_float2(v[e], v[e + 1]), cc2, negm);
            t2.x = ex2(t2.x);
            t2.y = ex2(t2.y);
            pk[i] = pack_bf16x2(t2.x, t2.y);
            if (i & 1) rb = fadd2(rb, t2); else ra = fadd2(ra, t2);
          }
          tmem_st32(tmem + lane_off + s_col + hh * 32, pk);
        }
        l = fmaf(l, alpha, (ra.x + ra.y) + (rb.x + rb.y));
        if (__any_sync(0xffffffffu, rescale)) {
          // S_j was issued after O += P_{j-1} V_{j-1} of this half, in MMA
          // issue order, so O is complete here.
#pragma unroll
          for (int d0 = 0; d0 < D; d0 += 32) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_off + o_col + d0, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st32(tmem + lane_off + o_col + d0, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sh.p_full[hf]);
      }
      if (!ok) break;
      // epilogue: the last O += P V of this half, then O / l and LSE, or the partial result
      const bool whole = x.whole();
      const int64_t orow = (int64_t)x.q0 + tok;
      const int32_t head = x.kh * p.group + row_head;
      float* part = parts.o + ((2 * (int64_t)blockIdx.x + (x.begins() ? 1 : 0)) * parts.rows + hf * 128 + row) * D;
      if (tiles > 0) {
        if (!mbar_wait_warp(&sh.pv_done[hf], (g + tiles - 1) & 1, abort)) break;
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: 0; NaN stays
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += 32) {
        uint32_t o[32];
        if (tiles > 0) {
          tmem_ld32(tmem + lane_off + o_col + d0, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (live && whole) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + orow * p.o_rs + (int64_t)head * p.o_hs + d0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
            if (in_span(p.out_span, dst + i, 16, p.err)) dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i)  // (a thread has a row of its own: whole sectors)
            if (in_span(parts.o_span, part + d0 + 8 * i, 32, p.err)) store_sector(part + d0 + 8 * i, &o[8 * i]);
        }
      }
      if (live && whole) {
        float* la = p.lse + (int64_t)head * p.total_q + orow;
        if (in_span(p.lse_span, la, 4, p.err))
          *la = l == 0.f ? -INFINITY : (m_use + __log2f(l)) * 0.69314718055994531f;
      } else if (live) {
        const int64_t r = (2 * (int64_t)blockIdx.x + (x.begins() ? 1 : 0)) * parts.rows + hf * 128 + row;
        if (in_span(parts.ml_span, parts.ml + 2 * r, 8, p.err))
          *reinterpret_cast<float2*>(parts.ml + 2 * r) = make_float2(m_use, l);
      }
      tc_fence_before();
      if (TREE) pieces.done(sh);
      g += tiles;
    }
  } else if constexpr (E4M3) {
    warpgroup_set_regs<C::REGS_CONVERT, C::REGS_LAUNCH>();
    // ------------------------------------------------------------ codes to bf16
    // A thread takes the 64 codes of one column chunk of a key (64 threads walk
    // down one chunk, so that eight lanes meet eight bank groups in reading and
    // in writing): the key's scale is looked up once for all of them.
    const int t = threadIdx.x - 384;  // 0..127
    const int cc = C::NC == 2 ? t >> 6 : 0, r0 = C::NC == 2 ? t & 63 : t;
    const int box_shift = min(p.pages.page_shift, 7);
    PieceReader<true> pieces;
    PagedPiece copy;
    uint32_t pos = 0;
    bool ok = true;
    while (ok && (TREE ? pieces.wait(sh, abort) : pieces.next(sh, copy, abort))) {
      const PagedPiece& x = TREE ? sh.piece[pieces.n % kPieces] : copy;  // (as the softmax)
      const int32_t tiles = min(x.j1, x.u.tiles);
      const int32_t unit_lo = TREE ? tree_unit_lo(p, x) : x.u.lo;
      for (int32_t j = x.j0; ok && j < tiles; ++j) {
        const int32_t key0 = (x.u.tile0 + j) * kChunkTile;
#pragma unroll 1
        for (int which = 0; which < 2; ++which, ++pos) {
          const uint32_t rs = pos % C::NRAW, s = pos % C::NSLOT;
          if (!mbar_wait_warp(&sh.raw_full[rs], (pos / C::NRAW) & 1, abort)) { ok = false; break; }
          if (!mbar_wait_warp(&sh.kv_empty[s], ((pos / C::NSLOT) & 1) ^ 1, abort)) { ok = false; break; }
          __syncwarp();
          const uint8_t* src = raw + rs * C::CHUNK;
          const uint8_t* sc = scales + rs * C::SCALES;
          uint8_t* dst = ring + s * C::TILE;
          // rows of V that no row of the unit sees may hold anything: cleared
          const int lo = which ? unit_lo - key0 : -1, hi = which ? x.u.hi - key0 : kChunkTile;
#pragma unroll
          for (int i = 0; i < C::NC; ++i) {
            const int r = r0 + i * 64;
            const float f = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(
                sc + ((r >> box_shift) << 7) + ((r & ((1 << box_shift) - 1)) << 1)));
            const bool keep = r >= lo && r < hi, large = keep && f > 0x1p7f;
            // 2^120 * scale, 0 for a row to clear (the codes' bits are finite in any case)
            const float f1 = keep ? (large ? 0x1p127f : f * 0x1p120f) : 0.f;
            const uint32_t ff = pack_bf16x2(f1, f1);
            const uint8_t* from = src + r * 128;
            uint8_t* to = dst + cc * C::CHUNK + r * 128;
            uint4 u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) u[k] = *reinterpret_cast<const uint4*>(from + (((cc * 4 + k) ^ (r & 7)) << 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // the upper and the lower bytes of four bf16, then two and two of them
                const uint32_t h = (w[e] & 0x80808080u) | ((w[e] >> 4) & 0x07070707u), l = (w[e] * 16u) & 0xf0f0f0f0u;
                y[2 * e] = mul_pair(__byte_perm(l, h, 0x5140), ff);
                y[2 * e + 1] = mul_pair(__byte_perm(l, h, 0x7362), ff);
              }
              *reinterpret_cast<uint4*>(to + (((2 * k) ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<uint4*>(to + (((2 * k + 1) ^ (r & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
            if (large) {  // 2^120 * scale does not fit into a bf16: times the rest of it
              const uint32_t gg = pack_bf16x2(f * 0x1p-7f, f * 0x1p-7f);
#pragma unroll 1
              for (int k = 0; k < 32; ++k) {
                uint32_t* y = reinterpret_cast<uint32_t*>(to) + k;
                *y = mul_pair(*y, gg);
              }
            }
          }
          if (TREE && which && key0 + kChunkTile > x.sk - x.n) {  // nor may new rows that no row of the unit sees
            uint32_t any[4];
            tree_unit_bits(p, x, unit_lo, key0, any);
#pragma unroll
            for (int i = 0; i < C::NC; ++i) {
              const int r = r0 + i * 64, w = r >> 5;
              const uint32_t lower = (w & 1) ? any[1] : any[0], upper = (w & 1) ? any[3] : any[2];
              if ((((w & 2) ? upper : lower) >> (r & 31)) & 1u) continue;
              uint4* to = reinterpret_cast<uint4*>(dst + cc * C::CHUNK + r * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) to[k] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&sh.kv_full[s]);
          mbar_arrive(&sh.raw_empty[rs]);
        }
      }
      if (TREE && ok) pieces.done(sh);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && sh.abort) record_error(p.err, kErrTimeout);
}

template <int D, bool E4M3, bool TREE>
cudaError_t launch_chunk_as(const PagedLaunch& L, int32_t take, cudaStream_t stream) {
  using C = ChunkCfg<D, E4M3>;
  auto kern = varlen_paged_chunk_kernel<D, E4M3, TREE>;
  // The register split assumes the compiled per-thread count; refuse to
  // launch a build that came out differently.
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != (int)C::REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(kern, (unsigned)L.sms, C::THREADS, C::SMEM, stream, L.chunk_q, L.chunk_k, L.chunk_v, L.chunk_ks,
                           L.chunk_vs, L.p, L.chunk, take);
}

template <int D, bool E4M3>
cudaError_t launch_chunk_d(const PagedLaunch& L, int32_t take, cudaStream_t stream) {
  return L.tree ? launch_chunk_as<D, E4M3, true>(L, take, stream) : launch_chunk_as<D, E4M3, false>(L, take, stream);
}

}  // namespace

cudaError_t launch_paged_chunk(const PagedLaunch& L, int32_t take, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return L.e4m3 ? launch_chunk_d<64, true>(L, take, stream) : launch_chunk_d<64, false>(L, take, stream);
    case 96: return L.e4m3 ? launch_chunk_d<96, true>(L, take, stream) : launch_chunk_d<96, false>(L, take, stream);
    case 128: return L.e4m3 ? launch_chunk_d<128, true>(L, take, stream) : launch_chunk_d<128, false>(L, take, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace varlen
