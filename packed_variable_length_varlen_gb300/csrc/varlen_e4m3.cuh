// varlen_e4m3.cuh -- a vector of bf16 as E4M3 codes and a power-of-two scale:
// what the cache's writers share.
//
// With a = max |x| of the vector, s = 2^e for the least e >= -127 with
// a <= 448 * 2^e.  Writing a = f * 2^X, 1 <= f < 2: 448 = 1.75 * 2^8, so e =
// X - 8, plus one when f > 1.75; both are read off the bf16 bits of a, whose
// order as integers is the order of |x| (a non-finite value is 0x7f80 or
// above).  x * 2^-e is exact in fp32, so the code's one rounding is the
// conversion's.
#pragma once

#include <cuda_fp8.h>

#include "varlen_internal.h"

namespace varlen {

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

}  // namespace varlen
