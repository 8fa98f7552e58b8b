// q4lin_mfma16.h -- building blocks of the kernels in which each token picks
// its own weights (low-rank adapters, experts): 16 x 16 x 32 matrix-core
// products of bf16 operands, bounded buffer loads, the two-part bf16 form of
// a binary32 value.  Internal header: not part of the C ABI.
#pragma once

#include "q4lin_device.h"

namespace q4lin {
namespace mfma16 {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Buffer loads: offsets at or past the resource's byte count return zeros
// without a memory access, so a load past the end needs no branch.
using rsrc_t = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
constexpr uint32_t kNowhere = 0x80000000u;  // a buffer offset past every range

// 16 bytes per lane from memory straight into LDS, lane l to lds_base + 16 l
// (lds_base wave-uniform; HINT: kOnce for what is not read again)
constexpr int kOnce = 2;  // non-temporal
template <int HINT = 0>
__device__ __forceinline__ void dma16(rsrc_t r, uint32_t voffset, uint32_t soffset, void* lds_base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds_base, 16, voffset,
                                           soffset, 0, HINT);
}

// waits until at most N of the wave's loads are outstanding (gfx9 encoding:
// vmcnt bits 3:0 and 15:14, expcnt 6:4 and lgkmcnt 11:8 left at "no wait");
// until its LDS operations are done
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N <= 63, "vmcnt holds 0..63");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (((N >> 4) & 3) << 14) | (7 << 4) | (15 << 8));
}
__device__ __forceinline__ void wait_lgkm0() { __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (7 << 4)); }

// the value of the lane at byte address src4 (four times its number)
__device__ __forceinline__ u32x4_t lane_piece(u32x4_t v, int src4) {
  return u32x4_t{(uint32_t)__builtin_amdgcn_ds_bpermute(src4, (int)v.x),
                 (uint32_t)__builtin_amdgcn_ds_bpermute(src4, (int)v.y),
                 (uint32_t)__builtin_amdgcn_ds_bpermute(src4, (int)v.z),
                 (uint32_t)__builtin_amdgcn_ds_bpermute(src4, (int)v.w)};
}

// D = A B + C on one wave, K = 32.  Lane l = 16 q + i holds row i of A and
// column i of B, both at k = 8 q .. 8 q + 7; D: column i, rows 4 q .. 4 q + 3.
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}

// (a & m) | c in one instruction (three-input bitwise operation)
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t m, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, m, c, 0xEA);
}

// v = hi + lo with hi = bf16(v), lo = bf16(v - hi): 16 significant bits, so
// that a product of the two parts on the matrix cores loses no more than
// 2^-17 of v (one bf16 alone would lose 2^-9, as much as the final store).
__device__ __forceinline__ void split_bf16(float v, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_bf16_rne(v);
  const float rest = v - bf16_bits_to_f32(hi);
  // an infinite or NaN value is carried by hi alone (inf - inf is NaN)
  lo = (hi & 0x7F80u) == 0x7F80u ? 0u : f32_to_bf16_rne(rest);
}

}  // namespace mfma16
}  // namespace q4lin
