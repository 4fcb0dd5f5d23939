// varlen_cache.cu -- writing packed keys and values into a paged cache and
// reading them back, in bf16 and in E4M3 with a power-of-two scale for each
// (token, head).
//
// Both kernels move each row once and compute next to nothing: the floor is
// 2 rows H (2 D + row bytes) over the memory's copy rate.  Four lanes take
// one (row, head) of K and of V together: D/32 16-byte loads of each, spread
// so that a group's load covers 64 consecutive bytes, and the groups of
// consecutive heads follow one another in memory.  All loads of a thread are
// issued before the first is used (8 x 16 bytes at D = 128), while the row's
// segment and page are looked up.
// Measured: 64 prompts of 0..8192 rows, 32 heads of 128, to E4M3: 809 us, 7.27
// TB/s; two of 9001 and 20011 rows, 16 heads of 96, to bf16: 54 us, 6.75 TB/s; 8 x
// 17580 rows of 56 heads back from E4M3: 877 us, 6.93 TB/s.  A plain copy moves 6.8.
//
// E4M3: with a = max |x| of the vector, s = 2^e for the least e >= -127 with
// a <= 448 * 2^e.  Writing a = f * 2^X, 1 <= f < 2: 448 = 1.75 * 2^8, so e =
// X - 8, plus one when f > 1.75; both are read off the bf16 bits of a, whose
// order as integers is the order of |x| (a non-finite value is 0x7f80 or
// above).  x * 2^-e is exact in fp32, so the code's one rounding is the
// conversion's.
#include <cuda_fp8.h>

#include <algorithm>

#include "sm103_ptx.cuh"
#include "varlen_paged.h"

namespace varlen {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kLanes = 4;  // lanes of one (row, head)

// A packed row's place: page (num_pages: none) and row in it; found is false
// for rows outside every segment, pos < 0 for rows before the sequence.  A read
// takes a length past what the table can name for that many positions; a write
// does not, as the clamp would move its rows onto older ones: positions past
// the table have no page, which is recorded as an error.
struct Place {
  bool found;
  int32_t pos, page, row;
};

template <bool WRITE>
__device__ __forceinline__ Place place_of(const CacheParams& p, int32_t row, int32_t b) {
  Place x{false, -1, p.pages.num_pages, 0};
  // (heads of one warp may cover several rows: walk on from its first one)
  while (b + 1 < p.batch && clamp_row(__ldg(p.cu + b + 1), p.total) <= row) ++b;
  const int32_t lo = clamp_row(__ldg(p.cu + b), p.total), hi = clamp_row(__ldg(p.cu + b + 1), p.total);
  if (row < lo || row >= hi) return x;
  x.found = true;
  x.pos = (WRITE ? max(p.pages.seqlens[b], 0) : cache_len(p.pages, b)) - (hi - row);
  if (x.pos < 0) return x;
  if (WRITE && (x.pos >> p.pages.page_shift) >= p.pages.max_pages) {
    if (p.err != nullptr) atomicOr(p.err, (unsigned int)kErrBounds);
    return x;
  }
  x.page = page_at(p.pages, b, x.pos >> p.pages.page_shift, p.err);
  x.row = x.pos & (p.pages.page_size - 1);
  return x;
}

// The (row, head) of this thread's lane group in sweep `it` and its place.
// The whole warp calls it; rows past the end get found = false.
struct Slot {
  int64_t row;
  int32_t head;
  bool live;
};

__device__ __forceinline__ Slot slot_of(const CacheParams& p, int64_t g) {
  Slot s;
  s.live = g < (int64_t)p.total * p.heads;
  const int64_t gc = s.live ? g : (int64_t)p.total * p.heads - 1;
  s.row = gc / p.heads;
  s.head = (int32_t)(gc - s.row * p.heads);
  return s;
}

// |x| of eight bf16 values as two u16 maxima per word.
__device__ __forceinline__ uint32_t absmax_bits(uint32_t m, const uint4& u) {
  m = __vmaxu2(m, u.x & 0x7fff7fffu);
  m = __vmaxu2(m, u.y & 0x7fff7fffu);
  m = __vmaxu2(m, u.z & 0x7fff7fffu);
  return __vmaxu2(m, u.w & 0x7fff7fffu);
}

// bf16 bits of the scale for the largest |x| bits `a`, and 1 / scale.
__device__ __forceinline__ uint32_t scale_bits(uint32_t a, float& inv) {
  int e = (int)(a >> 7) - 8 + ((a & 0x7fu) > 0x60u ? 1 : 0);  // biased exponent
  e = max(e, 0);                                             // 2^-127: bf16's subnormal 0x0040
  if (a == 0) e = 127;
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
  if (a >= 0x7f80u) {
    inv = 0.f;
    return 0x7fc0u;
  }
  return e == 0 ? 0x0040u : (uint32_t)e << 7;
}

__device__ __forceinline__ uint32_t codes2(uint32_t w, float inv) {
  const float2 x = make_float2(__uint_as_float(w << 16) * inv, __uint_as_float(w & 0xffff0000u) * inv);
  return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint2 codes8(const uint4& u, float inv) {
  return make_uint2(codes2(u.x, inv) | (codes2(u.y, inv) << 16), codes2(u.z, inv) | (codes2(u.w, inv) << 16));
}

// Two codes (low 16 bits of w) times s, rounded to bf16.
__device__ __forceinline__ uint32_t values2(uint32_t w, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(x.x * s, x.y * s);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) varlen_cache_write_kernel(const CacheParams p) {
  constexpr int N = D / 32;  // 16-byte chunks of bf16 per lane
  const int64_t groups = (int64_t)p.total * p.heads;
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t step = (int64_t)gridDim.x * (kCacheThreads / kLanes);
  for (int64_t g0 = (int64_t)blockIdx.x * (kCacheThreads / kLanes) + (threadIdx.x >> 5) * (32 / kLanes); g0 < groups;
       g0 += step) {  // warp-uniform
    const Slot s = slot_of(p, g0 + ((threadIdx.x & 31) / kLanes));
    const __nv_bfloat16* ka = p.k_new + s.row * p.k_rs + (int64_t)s.head * p.k_hs + lane * 8;
    const __nv_bfloat16* va = p.v_new + s.row * p.v_rs + (int64_t)s.head * p.v_hs + lane * 8;
    uint4 k[N], v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] = in_span(p.k_span, ka + i * 32, 16, p.err) ? __ldg(reinterpret_cast<const uint4*>(ka + i * 32)) : make_uint4(0, 0, 0, 0);
      v[i] = in_span(p.v_span, va + i * 32, 16, p.err) ? __ldg(reinterpret_cast<const uint4*>(va + i * 32)) : make_uint4(0, 0, 0, 0);
    }
    const int32_t b = warp_find_segment(p.cu, p.batch, p.total, __shfl_sync(0xffffffffu, (int32_t)s.row, 0));
    const Place x = place_of<true>(p, (int32_t)s.row, b);
    const bool store = s.live && x.found && x.page < p.pages.num_pages;
    uint8_t* kd = p.k + (int64_t)x.page * p.k_page + (int64_t)x.row * p.k_row + (int64_t)s.head * p.k_head;
    uint8_t* vd = p.v + (int64_t)x.page * p.v_page + (int64_t)x.row * p.v_row + (int64_t)s.head * p.v_head;
    if constexpr (!E4M3) {
      if (!store) continue;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint8_t *ko = kd + lane * 16 + i * 64, *vo = vd + lane * 16 + i * 64;
        if (in_span(p.kp_span, ko, 16, p.err)) *reinterpret_cast<uint4*>(ko) = k[i];
        if (in_span(p.vp_span, vo, 16, p.err)) *reinterpret_cast<uint4*>(vo) = v[i];
      }
    } else {
      uint32_t mk = 0, mv = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        mk = absmax_bits(mk, k[i]);
        mv = absmax_bits(mv, v[i]);
      }
      mk = max(mk & 0xffffu, mk >> 16) | (max(mv & 0xffffu, mv >> 16) << 16);  // K low, V high
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) mk = __vmaxu2(mk, __shfl_xor_sync(0xffffffffu, mk, o));
      if (!store) continue;
      float ik, iv;
      const uint32_t sk = scale_bits(mk & 0xffffu, ik), sv = scale_bits(mk >> 16, iv);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        uint8_t *ko = kd + lane * 8 + i * 32, *vo = vd + lane * 8 + i * 32;
        const uint2 ck = sk == 0x7fc0u ? make_uint2(0, 0) : codes8(k[i], ik);
        const uint2 cv = sv == 0x7fc0u ? make_uint2(0, 0) : codes8(v[i], iv);
        if (in_span(p.kp_span, ko, 8, p.err)) *reinterpret_cast<uint2*>(ko) = ck;
        if (in_span(p.vp_span, vo, 8, p.err)) *reinterpret_cast<uint2*>(vo) = cv;
      }
      if (lane < 2) {
        const int64_t at = ((int64_t)x.page * p.heads + s.head) * p.pages.page_size + x.row;
        unsigned short* d = reinterpret_cast<unsigned short*>(lane == 0 ? p.k_scale : p.v_scale) + at;
        if (in_span(lane == 0 ? p.ks_span : p.vs_span, d, 2, p.err)) *d = (unsigned short)(lane == 0 ? sk : sv);
      }
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) varlen_cache_read_kernel(const CacheParams p) {
  constexpr int N = D / 32;  // 16-byte chunks of bf16 per lane
  const int64_t groups = (int64_t)p.total * p.heads;
  const int lane = threadIdx.x & (kLanes - 1);
  const int64_t step = (int64_t)gridDim.x * (kCacheThreads / kLanes);
  for (int64_t g0 = (int64_t)blockIdx.x * (kCacheThreads / kLanes) + (threadIdx.x >> 5) * (32 / kLanes); g0 < groups;
       g0 += step) {  // warp-uniform
    const Slot s = slot_of(p, g0 + ((threadIdx.x & 31) / kLanes));
    const int32_t b = warp_find_segment(p.cu, p.batch, p.total, __shfl_sync(0xffffffffu, (int32_t)s.row, 0));
    const Place x = place_of<false>(p, (int32_t)s.row, b);
    if (!s.live || !x.found) continue;
    const bool held = x.page < p.pages.num_pages;
    const uint8_t* kd = p.k + (int64_t)x.page * p.k_page + (int64_t)x.row * p.k_row + (int64_t)s.head * p.k_head;
    const uint8_t* vd = p.v + (int64_t)x.page * p.v_page + (int64_t)x.row * p.v_row + (int64_t)s.head * p.v_head;
    uint4 k[N], v[N];
    if constexpr (!E4M3) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint8_t *ka = kd + lane * 16 + i * 64, *va = vd + lane * 16 + i * 64;
        k[i] = held && in_span(p.kp_span, ka, 16, p.err) ? __ldg(reinterpret_cast<const uint4*>(ka)) : make_uint4(0, 0, 0, 0);
        v[i] = held && in_span(p.vp_span, va, 16, p.err) ? __ldg(reinterpret_cast<const uint4*>(va)) : make_uint4(0, 0, 0, 0);
      }
    } else {
      uint2 ck[N], cv[N];
      const int64_t at = ((int64_t)x.page * p.heads + s.head) * p.pages.page_size + x.row;
      const __nv_bfloat16 *ka = p.k_scale + at, *va = p.v_scale + at;
      const float sk = held && in_span(p.ks_span, ka, 2, p.err) ? __bfloat162float(*ka) : 0.f;
      const float sv = held && in_span(p.vs_span, va, 2, p.err) ? __bfloat162float(*va) : 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint8_t *kc = kd + lane * 8 + i * 32, *vc = vd + lane * 8 + i * 32;
        ck[i] = held && in_span(p.kp_span, kc, 8, p.err) ? __ldg(reinterpret_cast<const uint2*>(kc)) : make_uint2(0, 0);
        cv[i] = held && in_span(p.vp_span, vc, 8, p.err) ? __ldg(reinterpret_cast<const uint2*>(vc)) : make_uint2(0, 0);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        k[i] = make_uint4(values2(ck[i].x, sk), values2(ck[i].x >> 16, sk), values2(ck[i].y, sk), values2(ck[i].y >> 16, sk));
        v[i] = make_uint4(values2(cv[i].x, sv), values2(cv[i].x >> 16, sv), values2(cv[i].y, sv), values2(cv[i].y >> 16, sv));
      }
    }
    __nv_bfloat16* ko = p.k_out + s.row * p.k_rs + (int64_t)s.head * p.k_hs + lane * 8;
    __nv_bfloat16* vo = p.v_out + s.row * p.v_rs + (int64_t)s.head * p.v_hs + lane * 8;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (in_span(p.k_span, ko + i * 32, 16, p.err)) *reinterpret_cast<uint4*>(ko + i * 32) = k[i];
      if (in_span(p.v_span, vo + i * 32, 16, p.err)) *reinterpret_cast<uint4*>(vo + i * 32) = v[i];
    }
  }
}

template <int D, bool E4M3>
cudaError_t launch_cache_d(const CacheLaunch& L, cudaStream_t stream) {
  const int64_t groups = (int64_t)L.p.total * L.p.heads;
  const int64_t blocks = (groups + kCacheThreads / kLanes - 1) / (kCacheThreads / kLanes);
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, 1 << 30);
  if (L.write) varlen_cache_write_kernel<D, E4M3><<<grid, kCacheThreads, 0, stream>>>(L.p);
  else varlen_cache_read_kernel<D, E4M3><<<grid, kCacheThreads, 0, stream>>>(L.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache(const CacheLaunch& L, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return L.e4m3 ? launch_cache_d<64, true>(L, stream) : launch_cache_d<64, false>(L, stream);
    case 96: return L.e4m3 ? launch_cache_d<96, true>(L, stream) : launch_cache_d<96, false>(L, stream);
    case 128: return L.e4m3 ? launch_cache_d<128, true>(L, stream) : launch_cache_d<128, false>(L, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace varlen
