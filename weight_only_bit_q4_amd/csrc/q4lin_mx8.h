// q4lin_mx8.h -- MXFP8 activations as the kernels see them (OCP Microscaling
// Formats: E4M3 values in blocks of 32 that share an E8M0 power of two), and
// the matrix-core product that takes them.  Internal header: not part of the
// C ABI.
//
// The product of a 4-bit code and an activation needs no conversion of the
// code: the byte q in 0..15 read as E4M3 is q 2^-9 (the subnormals 0..7 and
// the first binade 8..15 continue each other), and the operand's own block
// scale 2^9 makes it q.  The offset is the accumulator's start: one product
// of the activations with a constant operand of -8 (0x88) gives
// sum -8 x for every row at once.
//
// v_mfma_scale_f32_32x32x64_f8f6f4, as measured lane by lane: lane l = 32 h + i
// holds row i of A (column i of B) in eight registers; registers 0..3 are k =
// 16 h .. 16 h + 15 of the first block of 32, registers 4..7 the same of the
// second; the scale byte of lane l is row i's for block h.  D: column i, rows
// 8 (r / 4) + 4 h + r % 4.
#pragma once

#include "q4lin_device.h"

namespace q4lin {
namespace mx8 {

typedef int v8i_t __attribute__((ext_vector_type(8)));

constexpr int kScaleQ = 127 + 9;  // E8M0 of 2^9: a code byte counts as its number

// 32 codes of a lane's half of a group (16 bytes as they lie in memory: eight
// bytes of each block) as an operand: per dword the low nibbles (even k),
// then the high ones (odd k).
__device__ __forceinline__ v8i_t code_operand(u32x2_t b0, u32x2_t b1) {
  v8i_t v;
  const uint32_t c[4] = {b0.x, b0.y, b1.x, b1.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (int)(c[j] & 0x0F0F0F0Fu);
    v[2 * j + 1] = (int)((c[j] >> 4) & 0x0F0F0F0Fu);
  }
  return v;
}

// 16 values of each block in the codes' order: of every eight, those of even
// k, then those of odd k.
__device__ __forceinline__ v8i_t value_operand(u32x4_t b0, u32x4_t b1) {
  v8i_t v;
  const uint32_t c[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (int)__builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x06040200u);
    v[2 * j + 1] = (int)__builtin_amdgcn_perm(c[2 * j + 1], c[2 * j], 0x07050301u);
  }
  return v;
}

// D = X Q^T + C: x with the scale byte of its lane in byte SEL of xs, q codes
template <int SEL>
__device__ __forceinline__ f32x16_t product(v8i_t x, v8i_t q, f32x16_t c, uint32_t xs) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, q, c, 0, 0, SEL, (int)xs, 0, kScaleQ);
}

// sum -8 x over the group, in every column
template <int SEL>
__device__ __forceinline__ f32x16_t offset_sums(v8i_t x, uint32_t xs) {
  constexpr int m8 = (int)0x88888888u;
  const v8i_t minus8 = {m8, m8, m8, m8, m8, m8, m8, m8};
  const f32x16_t zero = {};
  return product<SEL>(x, minus8, zero, xs);
}

}  // namespace mx8
}  // namespace q4lin
