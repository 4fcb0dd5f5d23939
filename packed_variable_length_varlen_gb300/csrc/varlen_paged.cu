// varlen_paged.cu -- joins the partial results that the attention kernels left
// in the workspace, and launches the kernels of one call.
#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

// One unit per CTA of the attention kernel that began but did not end one
// (blockIdx.x; most have none), its rows shared out over blockIdx.y.  With
// parts i in the order of the CTAs: m = max m_i, w_i = 2^(m_i - m), l = sum l_i
// w_i, O = sum w_i o_i / l.  The weights come first, so that the loads of o
// depend on nothing: a unit of 228 parts takes 5 us where a running maximum
// over them took 19.  The warps take every kJoinWarps-th part, and their sums
// are added in the order of the warps.
constexpr int kJoinWarps = 8, kJoinRows = 8;
constexpr int kMaxParts = few_ctas(true) * kMaxSms;

// The sum (or maximum) of v over the block, in a fixed order.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* tmp) {
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, v, w);
    v = MAX ? fmaxf(v, t) : v + t;
  }
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
  __syncthreads();
  v = tmp[0];
  for (int w = 1; w < kJoinWarps; ++w) v = MAX ? fmaxf(v, tmp[w]) : v + tmp[w];
  __syncthreads();
  return v;
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    varlen_paged_join_kernel(const PagedParams p, const PagedParts parts) {
  __shared__ float so[kJoinWarps][D], weight[kMaxParts], tmp[kJoinWarps];
  dependency_wait();
  const PagedJoin u = parts.join[blockIdx.x];
  dependents_may_launch();
  if (u.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t q0 = clamp_row(__ldg(p.cu_q + u.b), p.total_q), q1 = clamp_row(__ldg(p.cu_q + u.b + 1), p.total_q);
  const int64_t first = (int64_t)u.blk * parts.unit_rows;
  const int32_t rows = (int32_t)min((int64_t)(q1 - q0) * p.group - first, (int64_t)parts.unit_rows);
  for (int32_t row = blockIdx.y; row < rows; row += kJoinRows) {
    auto at = [&](int32_t k) { return (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * parts.rows + row; };
    float m = -INFINITY;
    for (int32_t k = threadIdx.x; k < u.parts; k += kJoinWarps * 32) {
      weight[k] = parts.ml[at(k) * 2];
      m = fmaxf(m, weight[k]);
    }
    m = block_reduce<true>(m, tmp);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    for (int32_t k = threadIdx.x; k < u.parts; k += kJoinWarps * 32) {
      weight[k] = ex2(weight[k] - ref);
      l += parts.ml[at(k) * 2 + 1] * weight[k];
    }
    l = block_reduce<false>(l, tmp);  // (and the weights are there)
    float o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 8
    for (int32_t k = warp; k < u.parts; k += kJoinWarps) {
      const float* oa = parts.o + at(k) * D + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(oa[i * 32], weight[k], o[i]);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) so[warp][i * 32 + lane] = o[i];
    __syncthreads();
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: 0; NaN stays
    const int64_t r = first + row;
    const int32_t tok = (int32_t)(r / p.group), hd = u.kh * p.group + (int32_t)(r - (int64_t)tok * p.group);
    if (threadIdx.x < D) {
      float x = 0.f;
      for (int w = 0; w < kJoinWarps; ++w) x += so[w][threadIdx.x];
      __nv_bfloat16* a = p.out + (int64_t)(q0 + tok) * p.o_rs + (int64_t)hd * p.o_hs + threadIdx.x;
      if (in_span(p.out_span, a, 2, p.err)) *a = __float2bfloat16_rn(x * inv);
    }
    if (threadIdx.x == 0) {
      float* la = p.lse + (int64_t)hd * p.total_q + q0 + tok;
      if (in_span(p.lse_span, la, 4, p.err)) *la = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

// The same for the kernel for many rows, whose units have 256 rows and mostly
// few parts: a warp takes a row.
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    varlen_paged_join_rows_kernel(const PagedParams p, const PagedParts parts) {
  __shared__ float weights[kJoinWarps][kMaxSms];
  dependency_wait();
  const PagedJoin u = parts.join[blockIdx.x];
  dependents_may_launch();
  if (u.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* weight = weights[warp];
  const int32_t q0 = clamp_row(__ldg(p.cu_q + u.b), p.total_q), q1 = clamp_row(__ldg(p.cu_q + u.b + 1), p.total_q);
  const int32_t half_tokens = kChunkRows / 2 / p.group;
  for (int32_t row = blockIdx.y * kJoinWarps + warp; row < kChunkRows; row += gridDim.y * kJoinWarps) {
    const int32_t half = row >> 7, in_half = row & 127, t = in_half / p.group;
    const int64_t tok = (int64_t)u.blk * 2 * half_tokens + half * half_tokens + t;
    if (t >= half_tokens || tok >= q1 - q0) continue;
    auto at = [&](int32_t k) { return (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * parts.rows + row; };
    float m = -INFINITY, l = 0.f;
    for (int32_t k = lane; k < u.parts; k += 32) {
      weight[k] = parts.ml[at(k) * 2];
      m = fmaxf(m, weight[k]);
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int32_t k = lane; k < u.parts; k += 32) {
      weight[k] = ex2(weight[k] - ref);
      l += parts.ml[at(k) * 2 + 1] * weight[k];
    }
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    __syncwarp();
    float o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int32_t k = 0; k < u.parts; ++k) {
      const float* oa = parts.o + at(k) * D + lane;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(oa[i * 32], weight[k], o[i]);
    }
    __syncwarp();
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int32_t hd = u.kh * p.group + in_half - t * p.group;
    __nv_bfloat16* a = p.out + (q0 + tok) * p.o_rs + (int64_t)hd * p.o_hs + lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      if (in_span(p.out_span, a + i * 32, 2, p.err)) a[i * 32] = __float2bfloat16_rn(o[i] * inv);
    float* la = p.lse + (int64_t)hd * p.total_q + q0 + tok;
    if (lane == 0 && in_span(p.lse_span, la, 4, p.err))
      *la = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
  }
}

template <int D>
cudaError_t launch_join_d(const PagedLaunch& L, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (L.few)
    e = launch_overlapped(varlen_paged_join_kernel<D>, dim3(L.sms * few_ctas(L.e4m3), kJoinRows), kJoinWarps * 32, 0,
                          stream, L.p, L.few_parts);
  if (e == cudaSuccess && L.many)
    e = launch_overlapped(varlen_paged_join_rows_kernel<D>, dim3(L.sms, 8), kJoinWarps * 32, 0, stream, L.p, L.chunk);
  return e;
}

}  // namespace

cudaError_t launch_paged_join(const PagedLaunch& L, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return launch_join_d<64>(L, stream);
    case 96: return launch_join_d<96>(L, stream);
    case 128: return launch_join_d<128>(L, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_paged(const PagedLaunch& L, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (L.many) e = launch_paged_chunk(L, L.few ? kTakeMany : kTakeAll, stream);
  if (e == cudaSuccess && L.few) e = launch_paged_few(L, L.many ? kTakeFew : kTakeAll, stream);
  return e == cudaSuccess ? launch_paged_join(L, stream) : e;
}

}  // namespace varlen
