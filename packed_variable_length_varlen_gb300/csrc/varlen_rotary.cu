// varlen_rotary.cu -- rotary positions on packed rows, and the same on the way
// into the paged cache.
//
// Pair (x1, x2) of a head becomes scale (x1 cos t - x2 sin t, x2 cos t + x1 sin t)
// with t = position * f.  Bound: every element is read and written once and
// costs three operations; the angles are shared by all heads of a row.  So a lane
// keeps V pairs of a head (V = 8, or 4 where rotary_dim is no multiple of 16),
// and their sines and cosines, which the warp's lanes work out together for its row, and
// takes them through up to four heads, whose loads are all issued first (one, two, three,
// six, eight heads: 962, 688, 667, 660, 696 us where four take 629).  The lanes of a head lie next to one another:
// each reads V elements of the first half of the turned part and the V that stand
// half of it further on, 16 bytes a load, and lanes past the turned part take what
// lies behind it in the same two pieces.  Pairs (i, i + r/2) are then one element
// of each piece; interleaved pairs lie within a piece, and the same loads serve.
//
// The angle: t / 2 pi = position * turns * 2^-64 mod 1 is a 64-bit integer product
// whose overflow is the reduction, so far positions lose nothing; its top 32 bits
// give the quadrant and a remainder of at most an eighth of a turn, exact to 2^-32
// turn, on which the Taylor series of sine and cosine (to t^9 and t^10, remainders
// below 2^-29 and 2^-31) are good to fp32's last bit.
//
// Measured: 262144 rows of 40 heads of 128, 629 us, 7.2 TB/s (a plain copy moves 6.8);
// 29012 rows of 32 heads of 96, half of each turned, 58 us, 6.4 TB/s; 7493 rows of 32 heads,
// with 8 of K and of V into a bf16 cache, 32 us, 5.8 TB/s; 16 rows of those into an E4M3
// cache 2.4 us, the launch and two memory latencies; 60000 rows of 32 heads, with 8 of K and V,
// from cold 237 us into a bf16 cache, 6.2 TB/s, and 270 into an E4M3 one, 5.0 TB/s.  Few heads a row
// leave most of a warp's places empty: 65536 rows of 8 + 1 heads of 64 take 52 us, 2.9 TB/s, and
// 75 and 92 with the write, bf16 and E4M3; of 1 + 1 heads of 128 48, 1.4 TB/s, and 71 and 89.
// With angles worked out by every lane the first was 667.
#include <algorithm>

#include "sm103_ptx.cuh"
#include "varlen_e4m3.cuh"
#include "varlen_step.h"

namespace varlen {

namespace {

constexpr int kRotaryThreads = 128;
constexpr int kWarps = kRotaryThreads / 32;
constexpr int kPairs = 64;  // of a head, at most
// Lanes up to which each takes one head, for the sake of a short chain; one head and
// four, us: 16 rows of 40 heads of 128 2.2 and 2.6, 256 rows 2.7 and 2.9, 512 (163840 lanes)
// 3.3 and 3.1, 1024 5.2 and 4.3.  (Set by the rows' form; the write of 512 rows of 48 heads,
// 196608 lanes, takes 4.6 and 4.9, so that its border lies somewhat higher.)
constexpr int kFewLanes = 1 << 17;

// V bf16 elements.
template <int V>
struct Piece {
  uint32_t w[V / 2];
};

template <int V>
__device__ __forceinline__ Piece<V> load_piece(const Span& s, const __nv_bfloat16* a, unsigned int* err) {
  Piece<V> x;
  if constexpr (V == 8) {
    const uint4 u = in_span(s, a, 16, err) ? *reinterpret_cast<const uint4*>(a) : make_uint4(0, 0, 0, 0);
    x.w[0] = u.x;
    x.w[1] = u.y;
    x.w[2] = u.z;
    x.w[3] = u.w;
  } else {
    const uint2 u = in_span(s, a, 8, err) ? *reinterpret_cast<const uint2*>(a) : make_uint2(0, 0);
    x.w[0] = u.x;
    x.w[1] = u.y;
  }
  return x;
}

template <int V>
__device__ __forceinline__ void store_piece(const Span& s, void* a, const Piece<V>& x, unsigned int* err) {
  if constexpr (V == 8) {
    if (in_span(s, a, 16, err)) *reinterpret_cast<uint4*>(a) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
  } else {
    if (in_span(s, a, 8, err)) *reinterpret_cast<uint2*>(a) = make_uint2(x.w[0], x.w[1]);
  }
}

template <int V>
__device__ __forceinline__ void store_codes(const Span& s, uint8_t* a, const Piece<V>& x, float inv, bool zero,
                                            unsigned int* err) {
  uint32_t c[V / 4];
#pragma unroll
  for (int i = 0; i < V / 4; ++i) c[i] = zero ? 0u : codes2(x.w[2 * i], inv) | (codes2(x.w[2 * i + 1], inv) << 16);
  if constexpr (V == 8) {
    if (in_span(s, a, 8, err)) *reinterpret_cast<uint2*>(a) = make_uint2(c[0], c[1]);
  } else {
    if (in_span(s, a, 4, err)) *reinterpret_cast<uint32_t*>(a) = c[0];
  }
}

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sine and cosine of h * 2^-32 turns.
__device__ __forceinline__ void sincos_turn(uint32_t h, float& s, float& c) {
  const uint32_t q = (h + 0x20000000u) >> 30;
  const float t = (float)(int32_t)(h - (q << 30)) * 1.46291807926715968e-9f;  // 2 pi 2^-32
  const float u = t * t;
  float sn = fmaf(u, 2.75573192239858907e-6f, -1.98412698412698413e-4f);
  sn = fmaf(sn, u, 8.33333333333333333e-3f);
  sn = fmaf(sn, u, -1.66666666666666667e-1f);
  sn = fmaf(sn * u, t, t);
  float cs = fmaf(u, -2.75573192239858907e-7f, 2.48015873015873016e-5f);
  cs = fmaf(cs, u, -1.38888888888888889e-3f);
  cs = fmaf(cs, u, 4.16666666666666667e-2f);
  cs = fmaf(cs, u, -0.5f);
  cs = fmaf(cs, u, 1.f);
  const float a = (q & 1) ? cs : sn, b = (q & 1) ? sn : cs;
  s = (q & 2) ? -a : a;
  c = ((q + 1) & 2) ? -b : b;
}

// The top 32 bits of pos * f mod 2^64.
__device__ __forceinline__ uint32_t turns_of(int32_t pos, uint64_t f) {
  const uint32_t lo = (uint32_t)f, hi = (uint32_t)(f >> 32);
  return (uint32_t)pos * hi + __umulhi((uint32_t)pos, lo) - (pos < 0 ? lo : 0u);
}

// N floats from shared memory; a is aligned to N of them or to 4 (N = 2: to 2).
template <int N>
__device__ __forceinline__ void get_floats(float* x, const float* a) {
  if constexpr (N == 2) {
    const float2 u = *reinterpret_cast<const float2*>(a);
    x[0] = u.x;
    x[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(a + i);
      x[i] = u.x;
      x[i + 1] = u.y;
      x[i + 2] = u.z;
      x[i + 3] = u.w;
    }
  }
}

// (a, b) turned: c and s carry the scale.
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float y = fmaf(a, c, -b * s);
  b = fmaf(b, c, a * s);
  a = y;
}

// LG: lanes of a head (a power of two >= head_dim / 2 V); SWEEPS: heads that a lane takes.
template <int V, int LG, bool INTER, RotaryTo TO, int SWEEPS>
__global__ void __launch_bounds__(kRotaryThreads) varlen_rotary_kernel(const __grid_constant__ RotaryParams p) {
  __shared__ __align__(16) float table[kWarps][2][kPairs];  // cosines and sines of a warp's row
  dependency_wait();
  dependents_may_launch();
  constexpr int kSlots = 32 / LG, kBlock = kSlots * SWEEPS;  // heads of a warp at once, and in all
  float* cosines = table[threadIdx.x >> 5][0];
  float* sines = table[threadIdx.x >> 5][1];
  const int lane = threadIdx.x & 31, c = lane & (LG - 1), slot = lane / LG;
  const int32_t all = p.heads + (TO == kToRows ? 1 : 2) * p.kv_heads, blocks = (all + kBlock - 1) / kBlock;
  const int64_t units = (int64_t)p.total * blocks, step = (int64_t)gridDim.x * (kRotaryThreads / 32);
  const int turned = p.rot / (2 * V);  // lanes that turn; the next ones carry what lies behind rotary_dim
  const bool turns = c < turned, used = c < p.head_dim / (2 * V);
  const int at = turns ? c * V : p.rot + (c - turned) * V, apart = turns ? p.rot / 2 : (p.head_dim - p.rot) / 2;
  for (int64_t u = (int64_t)blockIdx.x * (kRotaryThreads / 32) + (threadIdx.x >> 5); u < units; u += step) {
    const int64_t row = u / blocks;
    const int32_t head0 = (int32_t)(u - row * blocks) * kBlock + slot;
    Piece<V> lo[SWEEPS], hi[SWEEPS];
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int32_t h = head0 + i * kSlots, hk = h - p.heads, hv = hk - p.kv_heads;
      const __nv_bfloat16* a = nullptr;
      Span s = p.q_span;
      if (h < p.heads) {
        if (turns || !p.q_same) a = p.q + row * p.q_rs + (int64_t)h * p.q_hs + at;
      } else if (hk < p.kv_heads) {
        if (turns || !p.k_same) a = p.k + row * p.k_rs + (int64_t)hk * p.k_hs + at;
        s = p.k_span;
      } else if (TO != kToRows && hv < p.kv_heads) {
        a = p.v + row * p.v_rs + (int64_t)hv * p.v_hs + at;
        s = p.v_span;
      }
      if (!used || a == nullptr) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) lo[i].w[j] = hi[i].w[j] = 0u;
      } else {
        lo[i] = load_piece<V>(s, a, p.err);
        hi[i] = load_piece<V>(s, a + apart, p.err);
      }
    }
    int32_t pos;
    bool here = true;
    if (p.positions != nullptr) {
      pos = p.positions[row];
    } else {
      const int32_t b = warp_find_segment(p.cu, p.batch, p.total, (int32_t)row);
      const int32_t first = clamp_row(p.cu[b], p.total);
      pos = (int32_t)row - first;
      here = row >= first && row < clamp_row(p.cu[b + 1], p.total);
    }
    if (!here) continue;  // warp-uniform
    // the warp's lanes share the row's angles out
#pragma unroll
    for (int j = 0; j < kPairs; j += 32) {
      const int i = j + lane;
      if (i < p.rot / 2) {
        float s, k;
        sincos_turn(turns_of(pos, p.turns[i]), s, k);
        cosines[i] = k * p.scale;
        sines[i] = s * (p.scale * p.sign);
      }
    }
    __syncwarp();
    float cs[V], sn[V];
    if (turns) {  // pairs of this lane: V in a row, or (interleaved) V / 2 of each piece
      constexpr int N = INTER ? V / 2 : V;
#pragma unroll
      for (int y = 0; y < V / N; ++y) {
        const int first = INTER ? (at >> 1) + y * (p.rot / 4) : at;
        get_floats<N>(&cs[y * N], cosines + first);
        get_floats<N>(&sn[y * N], sines + first);
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) cs[j] = sn[j] = 0.f;
    }
    __syncwarp();  // (the next row's angles take the same place)
    int32_t page = p.num_pages, in_page = 0;
    if (TO != kToRows) {
      const int64_t to = p.slots[row];
      if (to >= 0 && (to >> p.page_shift) < p.num_pages) {
        page = (int32_t)(to >> p.page_shift);
        in_page = (int32_t)(to & ((1 << p.page_shift) - 1));
      } else if (to >= 0 && lane == 0) {
        record_error(p.err, kErrBounds);
      }
    }
#pragma unroll
    for (int i = 0; i < SWEEPS; ++i) {
      const int32_t h = head0 + i * kSlots, hk = h - p.heads, hv = hk - p.kv_heads;
      if (turns && hk < p.kv_heads) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          float a0 = lo_of(lo[i].w[j]), a1 = hi_of(lo[i].w[j]), b0 = lo_of(hi[i].w[j]), b1 = hi_of(hi[i].w[j]);
          if (INTER) {
            turn(a0, a1, cs[j], sn[j]);
            turn(b0, b1, cs[V / 2 + j], sn[V / 2 + j]);
          } else {
            turn(a0, b0, cs[2 * j], sn[2 * j]);
            turn(a1, b1, cs[2 * j + 1], sn[2 * j + 1]);
          }
          lo[i].w[j] = pack_bf16x2(a0, a1);
          hi[i].w[j] = pack_bf16x2(b0, b1);
        }
      }
      if (h < p.heads) {
        if (used && (turns || !p.q_same)) {
          __nv_bfloat16* o = p.q_out + row * p.qo_rs + (int64_t)h * p.qo_hs + at;
          store_piece<V>(p.qo_span, o, lo[i], p.err);
          store_piece<V>(p.qo_span, o + apart, hi[i], p.err);
        }
      } else if (TO == kToRows) {
        if (hk < p.kv_heads && used && (turns || !p.k_same)) {
          __nv_bfloat16* o = p.k_out + row * p.ko_rs + (int64_t)hk * p.ko_hs + at;
          store_piece<V>(p.ko_span, o, lo[i], p.err);
          store_piece<V>(p.ko_span, o + apart, hi[i], p.err);
        }
      }
      if (TO != kToRows) {
        const bool is_k = hk < p.kv_heads, store = hk >= 0 && hv < p.kv_heads && page < p.num_pages;
        const int32_t hd = is_k ? hk : hv;
        uint8_t* o = is_k ? p.kp + (int64_t)page * p.k_page + (int64_t)in_page * p.k_row + (int64_t)hd * p.k_head
                          : p.vp + (int64_t)page * p.v_page + (int64_t)in_page * p.v_row + (int64_t)hd * p.v_head;
        const Span& s = is_k ? p.kp_span : p.vp_span;
        if constexpr (TO == kToCacheBf16) {
          if (store && used) {
            store_piece<V>(s, o + at * 2, lo[i], p.err);
            store_piece<V>(s, o + (at + apart) * 2, hi[i], p.err);
          }
        } else {
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < V / 2; ++j) m = __vmaxu2(m, __vmaxu2(lo[i].w[j] & 0x7fff7fffu, hi[i].w[j] & 0x7fff7fffu));
          m = max(m & 0xffffu, m >> 16);
#pragma unroll
          for (int w = 1; w < LG; w <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, w));
          float inv;
          const uint32_t bits = scale_bits(m, inv);
          if (store && used) {
            store_codes<V>(s, o + at, lo[i], inv, bits == 0x7fc0u, p.err);
            store_codes<V>(s, o + at + apart, hi[i], inv, bits == 0x7fc0u, p.err);
          }
          if (store && c == 0) {
            const int64_t j = (((int64_t)page * p.kv_heads + hd) << p.page_shift) + in_page;
            unsigned short* d = reinterpret_cast<unsigned short*>(is_k ? p.k_scale : p.v_scale) + j;
            if (in_span(is_k ? p.ks_span : p.vs_span, d, 2, p.err)) *d = (unsigned short)bits;
          }
        }
      }
    }
  }
}

template <int V, int LG, bool INTER, RotaryTo TO, int SWEEPS>
cudaError_t launch_rotary_sweeps(const RotaryLaunch& L, cudaStream_t stream) {
  constexpr int kBlock = 32 / LG * SWEEPS;
  const int64_t all = L.p.heads + (int64_t)(TO == kToRows ? 1 : 2) * L.p.kv_heads;
  const int64_t units = L.p.total * ((all + kBlock - 1) / kBlock);
  const unsigned grid = (unsigned)std::min<int64_t>((units + kWarps - 1) / kWarps, 1 << 30);
  return launch_overlapped(varlen_rotary_kernel<V, LG, INTER, TO, SWEEPS>, dim3(grid), kRotaryThreads, 0, stream, L.p);
}

template <int V, int LG, bool INTER, RotaryTo TO>
cudaError_t launch_rotary_to(const RotaryLaunch& L, cudaStream_t stream) {
  const int64_t heads = (int64_t)L.p.total * (L.p.heads + (int64_t)(TO == kToRows ? 1 : 2) * L.p.kv_heads);
  return heads * LG <= kFewLanes ? launch_rotary_sweeps<V, LG, INTER, TO, 1>(L, stream)
                                 : launch_rotary_sweeps<V, LG, INTER, TO, 4>(L, stream);
}

template <int V, int LG>
cudaError_t launch_rotary_lanes(const RotaryLaunch& L, cudaStream_t stream) {
  switch (L.to) {
    case kToRows:
      return L.interleaved ? launch_rotary_to<V, LG, true, kToRows>(L, stream)
                           : launch_rotary_to<V, LG, false, kToRows>(L, stream);
    case kToCacheBf16:
      return L.interleaved ? launch_rotary_to<V, LG, true, kToCacheBf16>(L, stream)
                           : launch_rotary_to<V, LG, false, kToCacheBf16>(L, stream);
    default:
      return L.interleaved ? launch_rotary_to<V, LG, true, kToCacheE4m3>(L, stream)
                           : launch_rotary_to<V, LG, false, kToCacheE4m3>(L, stream);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& L, cudaStream_t stream) {
  if (L.p.rot % 16 == 0)
    return L.p.head_dim == 64 ? launch_rotary_lanes<8, 4>(L, stream) : launch_rotary_lanes<8, 8>(L, stream);
  return L.p.head_dim == 64 ? launch_rotary_lanes<4, 8>(L, stream) : launch_rotary_lanes<4, 16>(L, stream);
}

}  // namespace varlen
