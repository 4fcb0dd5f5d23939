// varlen_paged.cu -- joins the partial results that the attention kernels left
// in the workspace, and launches the kernels of one call.
//
// The joins read what the attention kernels wrote just before (out of L2,
// mostly) and are bound by latency: four dependent loads and a launch, 4 to 6 us
// for few rows; for many rows up to 40 MB at D = 128, 11 to 17 us.
#include "sm103_ptx.cuh"
#include "varlen_paged.h"
#include "varlen_paged_walk.cuh"

namespace varlen {

namespace {

// A block for each CTA of the attention kernel joins the unit that the CTA began
// but did not end (most have none).  With parts i in the order of the CTAs: m =
// max m_i, w_i = 2^(m_i - m), l = sum l_i w_i, O = sum w_i o_i / l.  The weights
// come first, so that the loads of o depend on nothing.  A warp takes a row.
// Where a unit has more than kWarpParts parts, the blocks of the CTAs that
// hold it take a row each, its parts shared out over the warps, whose sums are
// added in order: one sequence of 185619 keys, two units of 228 parts and 8 rows,
// takes 33 us in all (43 with a running maximum over the parts in one block).
constexpr int kJoinWarps = 16, kWarpParts = 16;
constexpr int kMaxParts = few_ctas(true) * kMaxSms;

struct JoinRow {
  int64_t q;      // packed query row
  int32_t head;
};

__device__ __forceinline__ void join_lse(const PagedParams& p, const JoinRow& r, float m, float l) {
  float* la = p.lse + (int64_t)r.head * p.total_q + r.q;
  if (in_span(p.lse_span, la, 4, p.err)) *la = l == 0.f ? -INFINITY : (m + __log2f(l)) * 0.69314718055994531f;
}
__device__ __forceinline__ float join_inv(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }  // no key: 0; NaN stays

// (m, l) of slot row i, and an element of its output, as a part left them.
__device__ __forceinline__ float2 part_ml(const PagedParams& p, const PagedParts& parts, int64_t i) {
  const float* a = parts.ml + 2 * i;
  return in_span(parts.ml_span, a, 8, p.err) ? *reinterpret_cast<const float2*>(a) : make_float2(-INFINITY, 0.f);
}
__device__ __forceinline__ float part_o(const PagedParams& p, const PagedParts& parts, const float* a) {
  return in_span(parts.o_span, a, 4, p.err) ? *a : 0.f;
}

// One warp joins slot row `row` of unit u.
template <int D>
__device__ __forceinline__ void join_by_warp(const PagedParams& p, const PagedParts& parts, const PagedJoin& u,
                                             int32_t row, const JoinRow& r, float* weight) {
  const int lane = threadIdx.x & 31;
  auto at = [&](int32_t k) { return (2 * (int64_t)(u.first + k) + (k == 0 ? 1 : 0)) * parts.rows + row; };
  float m = -INFINITY, l = 0.f;
  for (int32_t k = lane; k < u.parts; k += 32) {
    const float2 ml = part_ml(p, parts, at(k));
    weight[2 * k] = ml.x;
    weight[2 * k + 1] = ml.y;
    m = fmaxf(m, ml.x);
  }
#pragma unroll
  for (int w = 16; w >= 1; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float ref = m == -INFINITY ? 0.f : m;
  for (int32_t k = lane; k < u.parts; k += 32) {
    weight[2 * k] = ex2(weight[2 * k] - ref);
    l += weight[2 * k + 1] * weight[2 * k];
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
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(part_o(p, parts, oa + i * 32), weight[2 * k], o[i]);
  }
  const float inv = join_inv(l);
  __nv_bfloat16* a = p.out + r.q * p.o_rs + (int64_t)r.head * p.o_hs + lane;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    if (in_span(p.out_span, a + i * 32, 2, p.err)) a[i * 32] = __float2bfloat16_rn(o[i] * inv);
  if (lane == 0) join_lse(p, r, m, l);
  __syncwarp();  // a warp's next row writes the weights that all its lanes read here
}

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

// The whole block joins row `row` of unit u.
template <int D>
__device__ __forceinline__ void join_by_block(const PagedParams& p, const PagedParts& parts, const PagedJoin& u,
                                              int32_t row, const JoinRow& r, float* weight, float (*so)[D], float* tmp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto at = [&](int32_t k) { return (2 * (int64_t)(u.first + k) + (k == 0 ? 1 : 0)) * parts.rows + row; };
  float m = -INFINITY;
  for (int32_t k = threadIdx.x; k < u.parts; k += kJoinWarps * 32) {
    const float2 ml = part_ml(p, parts, at(k));
    weight[2 * k] = ml.x;
    weight[2 * k + 1] = ml.y;
    m = fmaxf(m, ml.x);
  }
  m = block_reduce<true>(m, tmp);
  const float ref = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int32_t k = threadIdx.x; k < u.parts; k += kJoinWarps * 32) {
    weight[2 * k] = ex2(weight[2 * k] - ref);
    l += weight[2 * k + 1] * weight[2 * k];
  }
  l = block_reduce<false>(l, tmp);  // (and the weights are there)
  float o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
#pragma unroll 8
  for (int32_t k = warp; k < u.parts; k += kJoinWarps) {
    const float* oa = parts.o + at(k) * D + lane;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(part_o(p, parts, oa + i * 32), weight[2 * k], o[i]);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) so[warp][i * 32 + lane] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) x += so[w][threadIdx.x];
    __nv_bfloat16* a = p.out + r.q * p.o_rs + (int64_t)r.head * p.o_hs + threadIdx.x;
    if (in_span(p.out_span, a, 2, p.err)) *a = __float2bfloat16_rn(x * join_inv(l));
  }
  if (threadIdx.x == 0) join_lse(p, r, m, l);
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32)
    varlen_paged_join_kernel(const PagedParams p, const PagedParts parts) {
  __shared__ float so[kJoinWarps][D], weight[2 * kMaxParts], tmp[kJoinWarps];
  dependency_wait();
  const PagedJoin units[2] = {get_join(p, parts, 2 * blockIdx.x), get_join(p, parts, 2 * blockIdx.x + 1)};
  dependents_may_launch();
  const int warp = threadIdx.x >> 5;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const PagedJoin u = units[which];
    if (u.parts == 0 || (which == 0 && u.parts <= kWarpParts)) continue;  // block-uniform
    const int32_t q0 = clamp_row(p.cu_q[u.b], p.total_q), q1 = clamp_row(p.cu_q[u.b + 1], p.total_q);
    const int32_t first = u.blk * kFewRows, rows = min((q1 - q0) * p.group - first, kFewRows);
    auto row_of = [&](int32_t row) {
      const int32_t tok = (first + row) / p.group;
      return JoinRow{(int64_t)q0 + tok, u.kh * p.group + first + row - tok * p.group};
    };
    if (u.parts <= kWarpParts) {
      for (int32_t row = warp; row < rows; row += kJoinWarps)
        join_by_warp<D>(p, parts, u, row, row_of(row), weight + warp * 2 * kWarpParts);
    } else {
      const int32_t blocks = min(u.parts, rows);  // that share the rows
      for (int32_t row = blockIdx.x - u.first; row < rows && (int32_t)blockIdx.x - u.first < blocks; row += blocks)
        join_by_block<D>(p, parts, u, row, row_of(row), weight, so, tmp);
    }
    __syncthreads();
  }
}

// The same for the kernel for many rows, whose units have 256 rows: a row a
// warp, kChunkRows / kRowsWarps blocks a unit.
constexpr int kRowsWarps = 8;

template <int D>
__global__ void __launch_bounds__(kRowsWarps * 32)
    varlen_paged_join_rows_kernel(const PagedParams p, const PagedParts parts) {
  __shared__ float weight[kRowsWarps][2 * kMaxSms];
  dependency_wait();
  const PagedJoin u = get_join(p, parts, 2 * blockIdx.x + 1);
  dependents_may_launch();
  if (u.parts != 0) {
    const int32_t warp = threadIdx.x >> 5, row = blockIdx.y * kRowsWarps + warp;
    const int32_t q0 = clamp_row(p.cu_q[u.b], p.total_q), q1 = clamp_row(p.cu_q[u.b + 1], p.total_q);
    const int32_t half_tokens = kChunkRows / 2 / p.group;
    const int32_t half = row >> 7, in_half = row & 127, t = in_half / p.group;
    const int64_t tok = (int64_t)u.blk * 2 * half_tokens + half * half_tokens + t;
    if (t < half_tokens && tok < q1 - q0)
      join_by_warp<D>(p, parts, u, row, JoinRow{q0 + tok, u.kh * p.group + in_half - t * p.group}, weight[warp]);
  }
}

template <int D>
cudaError_t launch_join_d(const PagedLaunch& L, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (L.few)
    e = launch_overlapped(varlen_paged_join_kernel<D>,
                          dim3(L.sms * few_ctas(L.e4m3)), kJoinWarps * 32, 0, stream, L.p, L.few_parts);
  if (e == cudaSuccess && L.many)
    e = launch_overlapped(varlen_paged_join_rows_kernel<D>, dim3(L.sms, kChunkRows / kRowsWarps), kRowsWarps * 32, 0, stream, L.p, L.chunk);
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
