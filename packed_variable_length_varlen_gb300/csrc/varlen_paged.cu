// varlen_paged.cu -- attention over the paged cache, the plain kernel: one
// warp per (query row, head), the keys one after another with a running
// maximum m and sum l (o and l are scaled by exp2(m - m') when m grows).
#include <cuda_fp8.h>

#include <algorithm>

#include "sm103_ptx.cuh"
#include "varlen_paged.h"

namespace varlen {

namespace {

template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const uint8_t* base, Span span, const __nv_bfloat16* scale, Span sspan,
                                         int lane, unsigned int* err, float (&x)[D / 32]) {
  if constexpr (E4M3) {
    const float s = in_span(sspan, scale, 2, err) ? __bfloat162float(*scale) : 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint8_t* a = base + lane + i * 32;
      const __half_raw h = __nv_cvt_fp8_to_halfraw(in_span(span, a, 1, err) ? *a : 0, __NV_E4M3);
      x[i] = __half2float(*reinterpret_cast<const __half*>(&h)) * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const __nv_bfloat16* a = reinterpret_cast<const __nv_bfloat16*>(base) + lane + i * 32;
      x[i] = in_span(span, a, 2, err) ? __bfloat162float(*a) : 0.f;
    }
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(128) varlen_paged_kernel(const PagedParams p) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * 4;
  for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5); w < (int64_t)p.total_q * p.num_heads; w += warps) {
    const int32_t row = (int32_t)(w / p.num_heads), h = (int32_t)(w % p.num_heads), kh = h / p.group;
    const int32_t b = warp_find_segment(p.cu_q, p.batch, p.total_q, row);
    const int32_t r0 = clamp_row(__ldg(p.cu_q + b), p.total_q), r1 = clamp_row(__ldg(p.cu_q + b + 1), p.total_q);
    if (row < r0 || row >= r1) continue;
    const int32_t sk = cache_len(p.pages, b);
    int32_t lo, hi;
    band_keys(row - r0, row - r0, r1 - r0, sk, p.win_left, p.win_right, &lo, &hi);
    float q[N], o[N], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const __nv_bfloat16* a = p.q + (int64_t)row * p.q_rs + (int64_t)h * p.q_hs + lane + i * 32;
      q[i] = in_span(p.q_span, a, 2, p.err) ? __bfloat162float(*a) : 0.f;
      o[i] = 0.f;
    }
    for (int32_t j = lo; j < hi; ++j) {
      const int32_t page = page_at(p.pages, b, j >> p.pages.page_shift, p.err), r = j & (p.pages.page_size - 1);
      float k[N], v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) k[i] = v[i] = 0.f;
      if (page < p.pages.num_pages) {
        const int64_t at = ((int64_t)page * p.kv_heads + kh) * p.pages.page_size + r;
        load_row<D, E4M3>(p.k + (int64_t)page * p.k_page + (int64_t)r * p.k_row + (int64_t)kh * p.k_head, p.kp_span,
                          p.k_scale + at, p.ks_span, lane, p.err, k);
        load_row<D, E4M3>(p.v + (int64_t)page * p.v_page + (int64_t)r * p.v_row + (int64_t)kh * p.v_head, p.vp_span,
                          p.v_scale + at, p.vs_span, lane, p.err, v);
      }
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float mn = fmaxf(m, s), a = ex2(m - mn), w2 = ex2(s - mn);
      l = fmaf(l, a, w2);
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], a, w2 * v[i]);
      m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      __nv_bfloat16* a = p.out + (int64_t)row * p.o_rs + (int64_t)h * p.o_hs + lane + i * 32;
      if (in_span(p.out_span, a, 2, p.err)) *a = __float2bfloat16_rn(o[i] * inv);
    }
    float* la = p.lse + (int64_t)h * p.total_q + row;
    if (lane == 0 && in_span(p.lse_span, la, 4, p.err))
      *la = l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

template <int D, bool E4M3>
cudaError_t launch_paged_d(const PagedLaunch& L, cudaStream_t stream) {
  const int64_t warps = (int64_t)L.p.total_q * L.p.num_heads;
  varlen_paged_kernel<D, E4M3><<<(unsigned)std::min<int64_t>((warps + 3) / 4, 1 << 30), 128, 0, stream>>>(L.p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return L.e4m3 ? launch_paged_d<64, true>(L, stream) : launch_paged_d<64, false>(L, stream);
    case 96: return L.e4m3 ? launch_paged_d<96, true>(L, stream) : launch_paged_d<96, false>(L, stream);
    case 128: return L.e4m3 ? launch_paged_d<128, true>(L, stream) : launch_paged_d<128, false>(L, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace varlen
