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
#include "q4lin_mfma16.h"

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

// E8M0 as binary32: 0 is the subnormal 2^-127, 255 NaN
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __builtin_bit_cast(float, e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}
// Four E4M3 values (a dword) in their block's scale as two bf16 pairs: exact
// (four significant bits and a power of two) up to bf16's range; NaN from
// either.  (Checked for every value and scale.)
__device__ __forceinline__ u32x2_t to_bf16x4(uint32_t w, float scale) {
  return u32x2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
}
// 32 of them, in memory order
__device__ __forceinline__ void to_bf16(const u32x4_t (&m)[2], uint32_t e, u32x4_t (&out)[4]) {
  const float scale = scale_value(e);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const u32x2_t a = to_bf16x4(m[d >> 1][2 * (d & 1)], scale), b = to_bf16x4(m[d >> 1][2 * (d & 1) + 1], scale);
    out[d] = u32x4_t{a.x, a.y, b.x, b.y};
  }
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

// The two kinds of activations a kernel is written for.  A lane's operands of
// a group from LDS: `x` a token's run of groups, `c` a row's, J the group's
// number in it, 16-byte pieces permuted by `key`.

// MXFP8: 64 bytes and two scale bytes of a token per group.
struct OpMx8 {
  static constexpr int XB = 64;
  static constexpr bool kScaled = true;
  typedef v8i_t X;
  typedef v8i_t Q;
  template <int J>
  static __device__ __forceinline__ X load_x(const uint8_t* x, int key, int lh) {
    return value_operand(*reinterpret_cast<const u32x4_t*>(x + 16 * ((4 * J + lh) ^ key)),
                         *reinterpret_cast<const u32x4_t*>(x + 16 * ((4 * J + 2 + lh) ^ key)));
  }
  template <int J>
  static __device__ __forceinline__ Q load_q(const uint8_t* c, int key, int lh) {
    return code_operand(*reinterpret_cast<const u32x2_t*>(c + 8 * lh + 16 * ((2 * J) ^ key)),
                        *reinterpret_cast<const u32x2_t*>(c + 8 * lh + 16 * ((2 * J + 1) ^ key)));
  }
  template <int SEL>
  static __device__ __forceinline__ f32x16_t offset(const X& x, uint32_t e) {
    return offset_sums<SEL>(x, e);
  }
  template <int SEL>
  static __device__ __forceinline__ f32x16_t product(const X& x, const Q& q, const f32x16_t& off, uint32_t e) {
    return mx8::product<SEL>(x, q, off, e);
  }
};

// bf16 in the codes' order (of every eight: k0 k4 k1 k5 k2 k6 k3 k7), codes as
// the exact bf16 128 + q; the offsets of the codes come with the activations.
// Exact products, binary32 sums (of terms some 30 times those of q - 8: the
// offset, -136 times the activations' sum, takes most of them away).  Lane half h takes k = 32 h + 8 m .. + 7 in
// instruction m.
struct OpBf16 {
  static constexpr int XB = 128;
  static constexpr bool kScaled = false;
  struct X {
    u32x4_t v[4];
  };
  typedef u32x4_t Q;
  typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
  template <int J>
  static __device__ __forceinline__ X load_x(const uint8_t* x, int key, int lh) {
    X r;
#pragma unroll
    for (int m = 0; m < 4; ++m) r.v[m] = *reinterpret_cast<const u32x4_t*>(x + 16 * ((8 * J + 4 * lh + m) ^ key));
    return r;
  }
  template <int J>
  static __device__ __forceinline__ Q load_q(const uint8_t* c, int key, int lh) {
    return *reinterpret_cast<const u32x4_t*>(c + 16 * ((2 * J + lh) ^ key));
  }
  template <int SEL>
  static __device__ __forceinline__ f32x16_t product(const X& x, const Q& c, const f32x16_t& off, uint32_t) {
    f32x16_t d = off;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      u32x4_t q;
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = mfma16::and_or(c[m] >> (4 * i), 0x000F000Fu, 0x43004300u);
      d = mfma(x.v[m], q, d);
    }
    return d;
  }
};

}  // namespace mx8
}  // namespace q4lin
