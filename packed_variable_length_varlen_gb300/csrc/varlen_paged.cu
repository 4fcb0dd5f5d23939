// varlen_paged.cu -- joins the partial results that the attention kernels left
// in the workspace, and launches the kernels of one call.
#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

// One unit per CTA of the attention kernel that began but did not end one
// (blockIdx.x; most have none), its rows shared out over blockIdx.y.  With
// parts i in the order of the CTAs: m = max m_i, l = sum l_i 2^(m_i - m),
// O = sum o_i 2^(m_i - m) / l.  The warps of a block take every kJoinWarps-th
// part, and their sums are added in the order of the warps.
constexpr int kJoinWarps = 8, kJoinRows = 8;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    varlen_paged_join_kernel(const PagedParams p, const PagedParts parts) {
  __shared__ float so[kJoinWarps][D], sm[kJoinWarps], sl[kJoinWarps];
  dependency_wait();
  const PagedJoin u = parts.join[blockIdx.x];
  dependents_may_launch();
  if (u.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t q0 = clamp_row(__ldg(p.cu_q + u.b), p.total_q), q1 = clamp_row(__ldg(p.cu_q + u.b + 1), p.total_q);
  const int64_t first = (int64_t)u.blk * kFewRows;
  const int32_t rows = (int32_t)min((int64_t)(q1 - q0) * p.group - first, (int64_t)kFewRows);
  for (int32_t row = blockIdx.y; row < rows; row += kJoinRows) {
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 4
    for (int32_t k = warp; k < u.parts; k += kJoinWarps) {
      const int64_t at = (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * parts.rows + row;
      const float2 ml = __ldg(reinterpret_cast<const float2*>(parts.ml + at * 2));
      const float mn = fmaxf(m, ml.x);
      const float a0 = mn == -INFINITY ? 1.f : ex2(m - mn), a1 = mn == -INFINITY ? 1.f : ex2(ml.x - mn);
      m = mn;
      l = l * a0 + ml.y * a1;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = o[i] * a0 + __ldg(parts.o + at * D + i * 32 + lane) * a1;
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) so[warp][i * 32 + lane] = o[i];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    float mm = -INFINITY, ll = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) mm = fmaxf(mm, sm[w]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    for (int w = 0; w < kJoinWarps; ++w) ll += sl[w] * ex2(sm[w] - ref);
    const float inv = ll > 0.f ? 1.f / ll : (ll == 0.f ? 0.f : ll);
    const int64_t r = first + row;
    const int32_t tok = (int32_t)(r / p.group), hd = u.kh * p.group + (int32_t)(r - (int64_t)tok * p.group);
    if (threadIdx.x < D) {
      float x = 0.f;
      for (int w = 0; w < kJoinWarps; ++w) x += so[w][threadIdx.x] * ex2(sm[w] - ref);
      __nv_bfloat16* a = p.out + (int64_t)(q0 + tok) * p.o_rs + (int64_t)hd * p.o_hs + threadIdx.x;
      if (in_span(p.out_span, a, 2, p.err)) *a = __float2bfloat16_rn(x * inv);
    }
    if (threadIdx.x == 0) {
      float* la = p.lse + (int64_t)hd * p.total_q + q0 + tok;
      if (in_span(p.lse_span, la, 4, p.err)) *la = ll == 0.f ? -INFINITY : (mm + __log2f(ll)) * 0.69314718055994531f;
    }
    __syncthreads();
  }
}

template <int D>
cudaError_t launch_join_d(const PagedLaunch& L, cudaStream_t stream) {
  return launch_overlapped(varlen_paged_join_kernel<D>, dim3(L.sms * kFewCtasPerSm, kJoinRows), kJoinWarps * 32,
                           0, stream, L.p, L.few);
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
  const cudaError_t e = launch_paged_few(L, kTakeAll, stream);
  if (e != cudaSuccess) return e;
  return launch_paged_join(L, stream);
}

}  // namespace varlen
