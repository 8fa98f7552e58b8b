// q4lin_lora_tail.h -- the low-rank adapters' term as the last step of a
// base product's kernel: a few tokens' rank values u are small enough that
// every output row fetches its own row of B.  Internal header: not part of
// the C ABI.
#pragma once

#include "q4lin_device.h"
#include "q4lin_kernels.h"

namespace q4lin {

// s_a sum over this lane's share of the ranks of B_a[n][r] u[t][r] (pieces of
// eight ranks lane, lane + lanes, ...), binary32; 0 for a token without an
// adapter
__device__ __forceinline__ float lora_share(const LoraTail& l, int N, int n, int t, int lane, int lanes) {
  const int id = l.ids[t];
  if ((uint32_t)id >= (uint32_t)l.adapters) return 0.0f;
  const u32x4_t* b = reinterpret_cast<const u32x4_t*>(l.b + ((size_t)id * N + n) * l.rank);
  const f32x4_t* u = reinterpret_cast<const f32x4_t*>(l.u + (size_t)t * l.rank);
  float v = 0.0f;
  for (int p = lane; p < l.rank >> 3; p += lanes) {
    const u32x4_t w = b[p];
    const f32x4_t u0 = u[2 * p], u1 = u[2 * p + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t ui = i < 2 ? u0 : u1;
      v = __builtin_fmaf(bf16_bits_to_f32(w[i] & 0xFFFFu), ui[2 * (i & 1)], v);
      v = __builtin_fmaf(__builtin_bit_cast(float, w[i] & 0xFFFF0000u), ui[2 * (i & 1) + 1], v);
    }
  }
  return l.scale != nullptr ? l.scale[id] * v : v;
}

}  // namespace q4lin
