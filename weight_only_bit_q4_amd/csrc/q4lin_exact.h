// q4lin_exact.h -- a weight's values and an output's sum from their
// definitions in binary64, for the rare outputs whose binary32 partial sums
// left the range.  Internal header: not part of the C ABI.
#pragma once

#include "q4lin_device.h"
#include "q4lin_kernels.h"

namespace q4lin {

// E4M3 (bias 7, subnormals) -> binary32, by its fields
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
  const uint32_t e = (b >> 3) & 0xFu, m = b & 7u;
  const float mag = e != 0u ? __builtin_bit_cast(float, ((e + 120u) << 23) | (m << 20)) : (float)m * 0x1p-9f;
  return (b & 0x80u) ? -mag : mag;
}

// Weight W[n][k] of format F in binary64, exact (the plain definition, for
// the repair below).
template <int F>
__device__ double weight_exact(const uint8_t* __restrict__ lo, const uint8_t* __restrict__ hi,
                               const uint8_t* __restrict__ sc, int K, int n, int k) {
  const size_t r = (size_t)n;
  if constexpr (F == FMT_BF16) {
    return (double)bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(lo)[r * K + k]);
  } else if constexpr (F == FMT_W8) {
    const int c = (int)(int8_t)lo[r * K + k];
    return (double)c * (double)f16_bits_to_f32(reinterpret_cast<const uint16_t*>(sc)[r * (K / 32) + k / 32]);
  } else {
    const uint32_t b = lo[r * (K / 2) + k / 2];
    const int nib = (int)((k & 1) ? (b >> 4) : (b & 15u));
    if constexpr (F == FMT_NVFP4) {
      const int e = (nib >> 1) & 3, m = nib & 1;
      double v = e == 0 ? 0.5 * m : __builtin_ldexp(1.0 + 0.5 * m, e - 1);
      if (nib & 8) v = -v;
      return v * (double)e4m3_to_f32(sc[r * (K / 16) + k / 16]);
    } else {
      const double s = (double)f16_bits_to_f32(reinterpret_cast<const uint16_t*>(sc)[r * (K / 64) + k / 64]);
      if constexpr (F == FMT_Q4) {
        return (double)(nib - 8) * s;
      } else if constexpr (F == FMT_Q5) {
        const int q = nib | ((int)((hi[r * (K / 8) + k / 8] >> (k & 7)) & 1u) << 4);
        return (double)(q - 16) * s;
      } else {
        const int q = nib | ((int)((hi[r * (K / 4) + k / 4] >> (2 * (k & 3))) & 3u) << 4);
        return (double)(q - 32) * s;
      }
    }
  }
}

// sum_k W[n][k] x[t][k] in binary64 (each product exact)
template <int F>
__device__ __forceinline__ double exact_sum(const uint16_t* __restrict__ x, const uint8_t* __restrict__ lo,
                                            const uint8_t* __restrict__ hi, const uint8_t* __restrict__ sc, int K,
                                            int n, int t) {
  double acc = 0.0;
  for (int k = 0; k < K; ++k)
    acc += weight_exact<F>(lo, hi, sc, K, n, k) * (double)bf16_bits_to_f32(x[(size_t)t * K + k]);
  return acc;
}
// ... as a call, for kernels that rarely take it
template <int F>
__device__ __attribute__((noinline)) double exact_sum_call(const uint16_t* __restrict__ x,
                                                           const uint8_t* __restrict__ lo,
                                                           const uint8_t* __restrict__ hi,
                                                           const uint8_t* __restrict__ sc, int K, int n, int t) {
  return exact_sum<F>(x, lo, hi, sc, K, n, t);
}

}  // namespace q4lin
