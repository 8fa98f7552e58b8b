// q4lin_quant.hip -- activations in 8 bits: the root-mean-square norm (with
// the residual's addition) and the gated quantization, both writing MXFP8.
//
//   v = x + r           (r: the residual stream, optional; h = bf16(v))
//   y = v w / sqrt(mean(v^2) + eps)              (rmsnorm_mx8)
//   y = x or silu(gate) x                        (quantize_mx8)
//   per block of 32: e the least integer >= -127 with max |y| <= 448 2^e,
//   values E4M3(y 2^-e) (nearest, ties to even; nothing saturates), scale
//   byte e + 127; a block with an infinity or NaN is NaN (scale 255).
//
// Bound: bytes.  One pass: a row stays in its workgroup's registers between
// the sum of squares and the store (longer rows than kMaxPieces a thread are
// read a second time, then from the caches).  v is binary32 and is not
// rounded to bf16 on its way into the norm: h's rounding is the residual
// stream's alone.  Squares and their sum are binary64, which the bytes hide.
//
// Measured: 4096 rows of 5120 with the residual 28 to 30 us (147 MB: the rate
// of a large copy), 2048 rows of 6144 quantized 7.9 (38 MB), one row 2.8.
#include "q4lin_kernels.h"
#include "q4lin_device.h"
#include "q4lin_mx8.h"

namespace q4lin {
namespace {

constexpr int kMaxPieces = 4;  // 16-byte pieces (8 values) of a row that a thread keeps

struct Eight {
  float v[8];
};

__device__ __forceinline__ Eight unpack8(u32x4_t b) {
  Eight e;
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e.v[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
    e.v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
  }
  return e;
}

__device__ __forceinline__ u32x4_t pack8(const Eight& e) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = (uint32_t)f32_to_bf16_rne(e.v[2 * j]) | ((uint32_t)f32_to_bf16_rne(e.v[2 * j + 1]) << 16);
  return u32x4_t{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ u32x4_t load16(const uint16_t* p) { return *reinterpret_cast<const u32x4_t*>(p); }

// The block's scale from the eight values of each of its four lanes (lanes 4 b
// .. 4 b + 3), and the values in it.  Magnitudes compare as integers, which
// puts NaN above every number.
__device__ __forceinline__ uint32_t to_mx8(const Eight& y, u32x2_t& out) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __builtin_bit_cast(uint32_t, y.v[i]) & 0x7FFFFFFFu;
    most = b > most ? b : most;
  }
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)most, 0xB1, 0xF, 0xF, false);
  most = o > most ? o : most;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)most, 0x4E, 0xF, 0xF, false);
  most = o > most ? o : most;
  // 448 = 1.75 2^8
  const int ex = (int)(most >> 23);
  int byte = ex - 8 + ((most & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  byte = byte < 0 ? 0 : byte;
  if (ex == 255) byte = 255;
  const float inverse = __builtin_bit_cast(float, byte == 255 ? 0x7FC00000u : (uint32_t)(254 - byte) << 23);
  int w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = __builtin_amdgcn_cvt_pk_fp8_f32(y.v[4 * j] * inverse, y.v[4 * j + 1] * inverse, 0, false);
    w[j] = __builtin_amdgcn_cvt_pk_fp8_f32(y.v[4 * j + 2] * inverse, y.v[4 * j + 3] * inverse, w[j], true);
  }
  out = u32x2_t{(uint32_t)w[0], (uint32_t)w[1]};
  return (uint32_t)byte;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* r;  // nullptr: no residual, h is not written
  const uint16_t* w;  // nullptr: ones
  uint16_t* h;
  uint8_t* values;
  uint8_t* scales;
  int K;
  float eps;
};

__device__ __forceinline__ Eight summed(const NormArgs& a, size_t at) {
  Eight v = unpack8(load16(a.x + at));
  if (a.r != nullptr) {
    const Eight r = unpack8(load16(a.r + at));
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] += r.v[i];
  }
  return v;
}

// The row's factor 1 / sqrt(mean + eps) as rstd and a power of two.  That is one
// but for factors near the ends of binary32 or past them: rows of bf16's
// subnormals have up to 2^133 sqrt(K), rows near its largest number 2^-128.
// (4096 rows of 5120 with the residual 29.4 us, 29.3 without the power.)
struct RowFactor {
  float shift, rstd;
};
__device__ __forceinline__ RowFactor row_factor(double mean_eps) {
  const double r = 1.0 / sqrt(mean_eps);
  if (r > 0x1p100) return {0x1p64f, (float)(r * 0x1p-64)};
  if (r < 0x1p-100) return {0x1p-64f, (float)(r * 0x1p64)};
  return {1.f, (float)r};
}

__device__ __forceinline__ void norm_store(const NormArgs& a, size_t row, int p, const Eight& v, RowFactor f) {
  const size_t at = row * (size_t)a.K + 8 * (size_t)p;
  if (a.r != nullptr) *reinterpret_cast<u32x4_t*>(a.h + at) = pack8(v);
  Eight y;
  if (a.w != nullptr) {
    const Eight w = unpack8(load16(a.w + 8 * (size_t)p));
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] = v.v[i] * f.shift * f.rstd * w.v[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y.v[i] = v.v[i] * f.shift * f.rstd;
  }
  u32x2_t out;
  const uint32_t scale = to_mx8(y, out);
  *reinterpret_cast<u32x2_t*>(a.values + at) = out;
  if ((p & 3) == 0) a.scales[row * (size_t)(a.K >> 5) + (p >> 2)] = (uint8_t)scale;
}

// One workgroup per row.  K is a multiple of 64 and a wave's pieces are 64 in
// a row, so the four lanes of a block of 32 are all inside the row or all
// past it.  KEEP: the pieces of a thread, kept in registers (0: any number,
// read twice).
template <int KEEP>
__global__ void __launch_bounds__(1024)
rmsnorm_mx8_kernel(NormArgs a) {
  __shared__ double part[16];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int pieces = a.K >> 3;
  const size_t row = blockIdx.x, at = row * (size_t)a.K;
  Eight kept[KEEP ? KEEP : 1];
  double sum = 0.0;  // (squares of values past 2^63 leave binary32)
  if constexpr (KEEP > 0) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int p = tid + j * threads;
      if (p < pieces) kept[j] = summed(a, at + 8 * (size_t)p);
    }
#pragma unroll
    for (int j = 0; j < KEEP; ++j)
      if (tid + j * threads < pieces)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)kept[j].v[i], (double)kept[j].v[i], sum);
  } else {
    for (int p = tid; p < pieces; p += threads) {
      const Eight v = summed(a, at + 8 * (size_t)p);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = __builtin_fma((double)v.v[i], (double)v.v[i], sum);
    }
  }
  double total = sum64_lanes(sum);
  if ((tid & 63) == 0) part[tid >> 6] = total;
  __syncthreads();
  total = 0.0;
  for (int w = 0; w < threads >> 6; ++w) total += part[w];
  const RowFactor f = row_factor(total / a.K + (double)a.eps);
  if constexpr (KEEP > 0) {
#pragma unroll
    for (int j = 0; j < KEEP; ++j) {
      const int p = tid + j * threads;
      if (p < pieces) norm_store(a, row, p, kept[j], f);
    }
  } else {
    for (int p = tid; p < pieces; p += threads) norm_store(a, row, p, summed(a, at + 8 * (size_t)p), f);
  }
}

// silu(gate) x.  Below kLowGate e^-gate leaves binary32 where the product need
// not (x up to 2^128): there silu is gate e^gate to 2^-126 of itself, taken as
// four factors e^(gate/4), x among them, so that nothing passes an end of
// binary32 before the product itself does.
constexpr float kLowGate = -88.f;
__device__ __forceinline__ float gated(float g, float x) {
  if (!(g < kLowGate)) return x * (g / (1.f + __expf(-g)));
  const float q = __expf(0.25f * g);
  return g * q * x * q * q * q;
}

// A thread takes eight values of a row.
__global__ void __launch_bounds__(256)
quantize_mx8_kernel(const uint16_t* x, const uint16_t* gate, uint8_t* values, uint8_t* scales, int64_t K,
                    int64_t x_stride, int64_t gate_stride, int64_t T) {
  const int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (8 * p >= K) return;  // (whole blocks of 32: K is a multiple of 64)
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    Eight y = unpack8(load16(x + t * x_stride + 8 * p));
    if (gate != nullptr) {
      const Eight g = unpack8(load16(gate + t * gate_stride + 8 * p));
      float least = g.v[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) least = fminf(least, g.v[i]);
      if (least >= kLowGate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] *= g.v[i] / (1.f + __expf(-g.v[i]));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y.v[i] = gated(g.v[i], y.v[i]);
      }
    }
    u32x2_t out;
    const uint32_t scale = to_mx8(y, out);
    *reinterpret_cast<u32x2_t*>(values + t * K + 8 * p) = out;
    if ((p & 3) == 0) scales[t * (K >> 5) + (p >> 2)] = (uint8_t)scale;
  }
}

// Eight bf16 in the paired order: k0 k4 k1 k5 k2 k6 k3 k7.
__device__ __forceinline__ u32x4_t paired8(u32x4_t v) {
  return u32x4_t{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                 __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

// The activations of the exact products: bf16 in that order, and of each group
// the offset of its codes, -136 times the sum (binary64, rounded once).  A
// thread takes eight values, eight threads a group; MX: from E4M3 values and
// their scales, exact (four significant bits and a power of two) up to bf16's
// range.
template <bool MX>
__global__ void __launch_bounds__(256)
paired_kernel(const void* x, const uint8_t* scales, uint16_t* out, float* offsets, int64_t pieces) {
  // (whole groups: pieces is a multiple of eight, and so is the grid's step)
  for (int64_t p = (int64_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += (int64_t)gridDim.x * 256) {
    u32x4_t v;
    if constexpr (MX) {
      const u32x2_t m = *reinterpret_cast<const u32x2_t*>(static_cast<const uint8_t*>(x) + 8 * p);
      const float scale = mx8::scale_value(scales[p >> 2]);
      const u32x2_t a = mx8::to_bf16x4(m.x, scale), b = mx8::to_bf16x4(m.y, scale);
      v = u32x4_t{a.x, a.y, b.x, b.y};
    } else {
      v = load16(static_cast<const uint16_t*>(x) + 8 * p);
    }
    const Eight e = unpack8(v);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += (double)e.v[i];
    sum = sum8_lanes(sum);
    *reinterpret_cast<u32x4_t*>(out + 8 * p) = paired8(v);
    if ((p & 7) == 0) offsets[p >> 3] = (float)(-136.0 * sum);
  }
}

}  // namespace

hipError_t launch_rmsnorm_mx8(const void* x, const void* residual, const void* weight, void* h, void* values,
                              void* scales, int64_t k, int64_t t, float eps, hipStream_t stream) {
  const NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(residual),
                   static_cast<const uint16_t*>(weight), static_cast<uint16_t*>(h), static_cast<uint8_t*>(values),
                   static_cast<uint8_t*>(scales), (int)k, eps};
  const int pieces = (int)(k / 8);
  // few rows: a thread per piece, so that the row's loads are all in flight
  // at once; many rows fill the chip with 256 threads each
  int threads = t >= 512 ? 256 : 1024;
  while (threads < 1024 && pieces > threads * kMaxPieces) threads *= 2;
  const int need = (pieces + 63) / 64 * 64;
  threads = need < threads ? need : threads;
  const int keep = (pieces + threads - 1) / threads;
  const dim3 grid((unsigned)t), block((unsigned)threads);
  if (keep == 1) rmsnorm_mx8_kernel<1><<<grid, block, 0, stream>>>(a);
  else if (keep == 2) rmsnorm_mx8_kernel<2><<<grid, block, 0, stream>>>(a);
  else if (keep == 3) rmsnorm_mx8_kernel<3><<<grid, block, 0, stream>>>(a);
  else if (keep == 4) rmsnorm_mx8_kernel<4><<<grid, block, 0, stream>>>(a);
  else rmsnorm_mx8_kernel<0><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_mx8(const void* x, const void* gate, void* values, void* scales, int64_t k, int64_t t,
                               int64_t x_stride, int64_t gate_stride, hipStream_t stream) {
  const int64_t cols = (k / 8 + 255) / 256;
  const dim3 grid((unsigned)cols, (unsigned)(t < 32768 ? t : 32768));
  quantize_mx8_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(gate),
                                                static_cast<uint8_t*>(values), static_cast<uint8_t*>(scales), k,
                                                x_stride, gate_stride, t);
  return hipGetLastError();
}

hipError_t launch_paired(const void* x, const void* scales, void* out, float* offsets, int64_t k, int64_t t,
                         hipStream_t stream) {
  const int64_t pieces = t * k / 8, blocks = (pieces + 255) / 256;
  // (a grid whose threads pass 2^32 in one dimension is cut without an error)
  constexpr int64_t kMost = 1 << 20;
  const dim3 grid((unsigned)(blocks < kMost ? blocks : kMost));
  uint16_t* const o = static_cast<uint16_t*>(out);
  if (scales != nullptr)
    paired_kernel<true><<<grid, 256, 0, stream>>>(x, static_cast<const uint8_t*>(scales), o, offsets, pieces);
  else
    paired_kernel<false><<<grid, 256, 0, stream>>>(x, nullptr, o, offsets, pieces);
  return hipGetLastError();
}

}  // namespace q4lin
