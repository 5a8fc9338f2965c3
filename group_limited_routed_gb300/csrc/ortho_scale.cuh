// Scaling of the orthogonalised update, shared by its kernels: element
// access, the power-of-two range of the F16 copy, norms over any range of
// magnitudes, and the scales of the intermediates.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pair_product.cuh"

namespace beam {

// F16 scales of the three intermediates (powers of two): singular values stay
// near or below one, so elements stay below these and the small ones keep
// their bits.
constexpr float kScaleX = 1024.f, kScaleGram = 1024.f, kScalePoly = 256.f;

template <bool F16>
__device__ __forceinline__ float from16(uint32_t bits) {
  return F16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(bits)))
             : __uint_as_float(bits << 16);
}

template <int TYPE>
__device__ __forceinline__ float element(const void* src, int64_t at) {
  if constexpr (TYPE == kF32)
    return static_cast<const float*>(src)[at];
  else
    return from16<TYPE == kF16>(static_cast<const uint16_t*>(src)[at]);
}

// The power of two that brings the largest magnitude into [2^13, 2^14): F16
// then keeps every bit of a 16-bit update down to 2^-27 of its largest
// element, and no product or norm over- or underflows.  Zero, infinite and
// NaN maxima take 1 (and then give zeros, or NaN throughout).
__device__ __forceinline__ float range_scale(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 23);
  if (amax_bits == 0 || e == 255) return 1.f;
  const int k = min(13 + 127 - e, 120);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// Sum of squares over any range of magnitudes: sum * 2^(2 exp), where exp is
// the exponent of the largest element met so far (its bits' exponent field).
struct ScaledSum {
  int exp = 0;
  float sum = 0.f;

  static __device__ __forceinline__ float pow2(int k) {  // 2^k, 0 below the normal range
    return k < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
  }
  __device__ __forceinline__ void add(int e, float s) {
    if (e > exp) {
      sum *= pow2(max(2 * (exp - e), -200));
      exp = e;
    }
    sum = fmaf(s, pow2(max(2 * (e - exp), -200)), sum);
  }
  // Eight elements; `top` keeps the bits of the largest magnitude.
  __device__ __forceinline__ void add8(const float (&v)[8], uint32_t& top) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      // as integers, so that a NaN is larger than every number
      m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    top = max(top, m);
    if (m == 0 || m >= 0x7f800000u) return;  // not finite: the maximum tells
    // squares of the elements times 2^(127 - e), which brings the largest
    // near 1 (subnormals count from the smallest normal exponent; the largest
    // exponent's power of two would be subnormal)
    const int e = min(max(static_cast<int>(m >> 23), 1), 253);
    const float k1 = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) sq = fmaf(v[k] * k1, v[k] * k1, sq);
    add(e, sq);
  }
};

// s of X = s * (copy scaled by k): 1 / (norm + eps), both in the copy's
// scale; the sum is in units of 2^(2 (exp - 127)).  An all-zero matrix with
// eps = 0 stays 0 / 0; one that is not finite becomes NaN.
__device__ __forceinline__ float inverse_norm(uint32_t amax, const ScaledSum& s, float k,
                                              float eps) {
  const float norm = sqrtf(s.sum) * (__uint_as_float(static_cast<uint32_t>(s.exp) << 23) * k);
  return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : 1.f / (norm + eps * k);
}

}  // namespace beam
