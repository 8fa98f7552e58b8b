// q4lin_lora.hip -- low-rank adapters of many requests beside a shared
// projection:
//
//     y[t][n] = bf16( S[t][n] + s_a sum_r B_a[n][r] u[t][r] ),
//     u[t][r] = sum_k A_a[r][k] x[t][k],           a = ids[t]
//
// with S = W X the base product in binary32 (made by the weight's own route)
// and no second term where ids[t] names no adapter.  Two launches beside the
// base product:
//
//   shrink   u, in binary32.  A workgroup takes 16 tokens, one of the
//            distinct adapters among them (slot) and 16 ranks; its eight
//            waves and KS workgroups split K.  Bound: reading A_a once per
//            16 tokens that share it; the K split is there because one
//            workgroup streams a whole 16 x K slab of A no faster than about
//            50 GB/s.
//   finish   sums the KS parts of u, scales, multiplies with B_a and adds S:
//            one read of S and B_a, one write of y, one rounding.  A wave
//            takes 16 tokens and 16 NB rows and goes through the distinct
//            adapters of its tokens: one pass over B for a run of tokens of
//            one adapter, 16 for 16 tokens of 16.
//
// u is binary32 from end to end; the matrix cores take s_a u as two bf16
// parts (split_bf16), so the adapters' term is as exact as the base sum.
#include "q4lin_kernels.h"
#include "q4lin_mfma16.h"

namespace q4lin {
namespace {

using namespace mfma16;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// The adapter of token t0 + i in lane 16 q + i (-1: none), and in `first` a
// bit for each lane 0..15 whose adapter no lower lane has.
__device__ __forceinline__ int tile_adapters(const int* __restrict__ ids, int t0, int T, int L, int li,
                                             uint32_t& first) {
  int id = t0 + li < T ? ids[t0 + li] : -1;
  if ((uint32_t)id >= (uint32_t)L) id = -1;
  bool dup = id < 0;
#pragma unroll
  for (int j = 0; j < 15; ++j) dup |= j < li && __builtin_amdgcn_readlane(id, j) == id;
  first = (uint32_t)__builtin_amdgcn_ballot_w64(!dup) & 0xFFFFu;
  return id;
}

// u parts [KS][T][R].  grid: (rank tiles of 16 RT) * KS, slots, token tiles.
template <int RT>
__global__ void __launch_bounds__(kThreads)
lora_shrink_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int* __restrict__ ids,
                   float* __restrict__ u, int K, int T, int R, int L, int KS) {
  __shared__ float red[kWaves][RT][16][20];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int t0 = blockIdx.z * 16;
  uint32_t first;
  const int id = tile_adapters(ids, t0, T, L, li, first);
  if ((int)blockIdx.y >= __builtin_popcount(first)) return;
  for (uint32_t s = blockIdx.y; s > 0; --s) first &= first - 1;
  const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(first));
  const int ks = blockIdx.x % KS, r0 = (blockIdx.x / KS) * (16 * RT);

  // this wave's run of 32-k steps
  const int steps = K >> 5, parts = KS * kWaves, part = ks * kWaves + wave;
  const int sb = (int)((int64_t)steps * part / parts), se = (int)((int64_t)steps * (part + 1) / parts);
  const uint16_t* xp = x + (size_t)min(t0 + li, T - 1) * K + 8 * lq;  // rows past the last repeat it
  const uint16_t* ap[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) ap[r] = a + ((size_t)ad * R + min(r0 + 16 * r + li, R - 1)) * K + 8 * lq;
  f32x4_t acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  int s = sb;
  for (; s + 4 <= se; s += 4) {  // four steps' loads in flight
    u32x4_t xv[4], av[RT][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      xv[j] = *reinterpret_cast<const u32x4_t*>(xp + 32 * (size_t)(s + j));
#pragma unroll
      for (int r = 0; r < RT; ++r) av[r][j] = *reinterpret_cast<const u32x4_t*>(ap[r] + 32 * (size_t)(s + j));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = mfma(xv[j], av[r][j], acc[r]);
  }
  for (; s < se; ++s) {
    const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(xp + 32 * (size_t)s);
#pragma unroll
    for (int r = 0; r < RT; ++r)
      acc[r] = mfma(xv, *reinterpret_cast<const u32x4_t*>(ap[r] + 32 * (size_t)s), acc[r]);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][r][4 * lq + i][li] = acc[r][i];
  __syncthreads();
  for (int o = threadIdx.x; o < RT * 256; o += kThreads) {
    const int r = o >> 8, t = (o >> 4) & 15, c = o & 15;
    const int rank = r0 + 16 * r + c;
    if (t0 + t >= T || rank >= R || ids[t0 + t] != ad) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += red[w][r][t][c];
    u[((size_t)ks * T + t0 + t) * R + rank] = v;
  }
}

// grid: row blocks of 4 waves * 16 NB rows, token tiles.  RS: 32-rank steps
// that cover R.
template <int RS, int NB>
__global__ void __launch_bounds__(256)
lora_finish_kernel(const uint16_t* __restrict__ b, const float* __restrict__ scale, const int* __restrict__ ids,
                   const float* __restrict__ u, SumSource base, uint16_t* __restrict__ y, int N, int T, int R, int L,
                   int KS, int vec) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int li = lane & 15, lq = lane >> 4;
  const int t0 = blockIdx.y * 16;
  const int n0 = (blockIdx.x * 4 + wave) * (16 * NB);
  if (n0 >= N) return;
  const int t = t0 + li;
  uint32_t todo;
  const int id = tile_adapters(ids, t0, T, L, li, todo);

  // token li's s_a u as two bf16 parts, ranks 32 s + 8 lq .. + 7 of step s
  u32x4_t uh[RS], ul[RS];
  const float sc = id >= 0 && scale != nullptr ? scale[id] : 1.0f;
#pragma unroll
  for (int s = 0; s < RS; ++s) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (id >= 0 && 32 * s + 8 * lq < R) {
      for (int k = 0; k < KS; ++k) {  // parts in order
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(u + ((size_t)k * T + t) * R + 32 * s + 8 * lq);
        const f32x4_t p0 = p[0], p1 = p[1];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] += p0[j];
          v[4 + j] += p1[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h0, l0, h1, l1;
      split_bf16(sc * v[2 * j], h0, l0);
      split_bf16(sc * v[2 * j + 1], h1, l1);
      uh[s][j] = h0 | (h1 << 16);
      ul[s][j] = l0 | (l1 << 16);
    }
  }

  f32x4_t acc[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  while (todo != 0) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    todo &= todo - 1;
    const uint16_t* bp = b + ((size_t)ad * N + n0) * R + 8 * lq;
    f32x4_t d[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) d[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const bool in = 32 * s + 8 * lq < R;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        u32x4_t bv = {0u, 0u, 0u, 0u};
        const int row = min(16 * c + li, N - 1 - n0);  // rows past the last repeat it and are not stored
        if (in) bv = *reinterpret_cast<const u32x4_t*>(bp + (size_t)row * R + 32 * s);
        d[c] = mfma(bv, uh[s], d[c]);
        d[c] = mfma(bv, ul[s], d[c]);
      }
    }
    // (a token keeps its own adapter's products only: taken, not added, so
    // that an infinity in one request's adapter stays in its own rows)
    const bool mine = id == ad;
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[c][i] = mine ? d[c][i] : acc[c][i];
  }
  if (t >= T) return;

  // the base sum, the one rounding, the store: rows n0 + 16 c + 4 lq .. + 3 of token t
  const int te = base.texp != nullptr ? base.texp[t] : 0;
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int n = n0 + 16 * c + 4 * lq;
    const size_t o = (size_t)t * N + n;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int k = 0; k < base.ks; ++k) {  // slices in order
      const float* p = base.part + (size_t)k * base.stride + o;
      if (vec) {
        if (n < N) v += *reinterpret_cast<const f32x4_t*>(p);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) v[i] += p[i];
      }
    }
    uint16_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f = v[i];
      // the many-token route's sums carry a power of two per token and row
      if (base.texp != nullptr && n + i < N) f = __builtin_ldexpf(f, te - base.rexp[n + i]);
      h[i] = f32_to_bf16_rne(f + acc[c][i]);
    }
    if (vec) {
      if (n < N)
        *reinterpret_cast<u32x2_t*>(y + o) = u32x2_t{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) y[o + i] = h[i];
    }
  }
}

// Workgroups that share K (so that at least about one per CU runs): each
// still has 32 k steps for most of its waves.
int shrink_split(int64_t k, int64_t t, int64_t r, int64_t adapters, int rt) {
  const int64_t tiles = (t + 15) / 16 * ((r + 16 * rt - 1) / (16 * rt));
  const int64_t slots = t < adapters ? t : adapters;  // an upper bound of the distinct adapters
  const int64_t groups = tiles * (slots < 16 ? slots : 16);
  int64_t ks = 256 / groups;
  if (ks > 8) ks = 8;
  if (ks > k / (32 * kWaves)) ks = k / (32 * kWaves);
  return ks < 1 ? 1 : (int)ks;
}

// rank tiles per workgroup: where there are many tokens, as many as share
// the activations' loads; else one, for more workgroups
int shrink_tiles(int64_t t, int64_t r) { return t < 256 || r <= 16 ? 1 : r <= 32 ? 2 : 4; }

template <int RS>
hipError_t launch_finish(const LoraArgs& a, const float* u, const SumSource& base, int ks, hipStream_t s) {
  const int64_t tiles = (a.t + 15) / 16;
  const int vec = (a.n & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
  // four 16-row tiles per wave share the token operand; one where that would
  // leave CUs idle
  const bool wide = tiles * ((a.n + 255) / 256) >= 256;
  const int nb = wide ? 4 : 1;
  const dim3 grid((unsigned)((a.n + 64 * nb - 1) / (64 * nb)), (unsigned)tiles);
  auto go = [&](auto kern) {
    kern<<<grid, dim3(256), 0, s>>>(static_cast<const uint16_t*>(a.b), static_cast<const float*>(a.scale),
                                    static_cast<const int*>(a.ids), u, base, static_cast<uint16_t*>(a.y), (int)a.n,
                                    (int)a.t, (int)a.rank, (int)a.adapters, ks, vec);
  };
  if (wide) go(lora_finish_kernel<RS, 4>);
  else go(lora_finish_kernel<RS, 1>);
  return hipGetLastError();
}

}  // namespace

size_t lora_u_bytes(int64_t k, int64_t t, int64_t rank, int64_t adapters) {
  const int ks = shrink_split(k, t, rank, adapters, shrink_tiles(t, rank));
  return ((size_t)ks * (size_t)t * (size_t)rank * 4 + 255) & ~(size_t)255;
}

hipError_t launch_lora_shrink(const LoraArgs& a, float* u, hipStream_t s) {
  const int rt = shrink_tiles(a.t, a.rank), ks = shrink_split(a.k, a.t, a.rank, a.adapters, rt);
  const int64_t slots = a.t < a.adapters ? a.t : a.adapters;
  const dim3 grid((unsigned)((a.rank + 16 * rt - 1) / (16 * rt) * ks), (unsigned)(slots < 16 ? slots : 16),
                  (unsigned)((a.t + 15) / 16));
  auto go = [&](auto kern) {
    kern<<<grid, dim3(kThreads), 0, s>>>(static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.a),
                                         static_cast<const int*>(a.ids), u, (int)a.k, (int)a.t, (int)a.rank,
                                         (int)a.adapters, ks);
  };
  if (rt == 1) go(lora_shrink_kernel<1>);
  else if (rt == 2) go(lora_shrink_kernel<2>);
  else go(lora_shrink_kernel<4>);
  return hipGetLastError();
}

hipError_t launch_lora_finish(const LoraArgs& a, const float* u, const SumSource& base, hipStream_t s) {
  const int ks = shrink_split(a.k, a.t, a.rank, a.adapters, shrink_tiles(a.t, a.rank));
  if (a.rank <= 32) return launch_finish<1>(a, u, base, ks, s);
  if (a.rank <= 64) return launch_finish<2>(a, u, base, ks, s);
  if (a.rank <= 128) return launch_finish<4>(a, u, base, ks, s);
  return launch_finish<8>(a, u, base, ks, s);
}

}  // namespace q4lin
