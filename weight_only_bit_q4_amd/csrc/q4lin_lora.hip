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
//   shrink   u, in binary32.  A workgroup takes 16 tokens, the distinct
//            adapters among them one after the other (few tiles: each in a
//            workgroup of its own) and 16 or 32 ranks; its eight waves and KS
//            workgroups split K.  Bound: reading x once and A_a once per 16
//            tokens that share it.  1024 tokens of runs, rank 32, K = 5120
//            (13 MB): 8.2 us.
//   finish   sums the KS parts of u, scales, multiplies with B_a and adds S:
//            one read of S and B_a, one write of y, one rounding.  A wave
//            takes 16 tokens and 16 NB rows of a block and goes through the
//            distinct adapters of its tokens.  Up to 4096 tokens it takes
//            them by adapter, in an order that the shrink's launch makes, so
//            that B is read about once whatever their order in x (1024 tokens
//            on 6144 rows, 38 MB: 13.8 us; mixed tokens of 8 adapters 13.8
//            against 22 in their own order, 280 of 24 on 7703 rows 17 / 41).
//
// Up to 4096 rank values (T R) each token's own products make them
// (lora_dots_kernel), and up to 32 tokens the base product's kernel adds the
// adapters' term as its last step (LoraTail): two launches in all.
//
// u is binary32 from end to end; the matrix cores take s_a u as two bf16
// parts (split_bf16), so the adapters' term is as exact as the base sum.
// Outputs that come out non-finite are formed again from binary64 base sums
// and a binary32 term.
#include "q4lin_exact.h"
#include "q4lin_kernels.h"
#include "q4lin_mfma16.h"

namespace q4lin {

// up to this many rank values the tokens' own products make them
bool lora_few(int64_t t, int64_t rank) { return t * rank <= 4096; }

namespace {

using namespace mfma16;

constexpr int kWaves = 8;
constexpr int kMaxSplit = 4;  // of the shrink's K
constexpr int kThreads = 64 * kWaves;

// The adapter of the tile's token i in lane 16 q + i, given its id (-1:
// none), and in `first` a bit for each lane 0..15 whose adapter no lower lane
// has.
__device__ __forceinline__ int tile_adapters(int id, int L, int li, uint32_t& first) {
  if ((uint32_t)id >= (uint32_t)L) id = -1;
  bool dup = id < 0;
#pragma unroll
  for (int j = 0; j < 15; ++j) dup |= j < li && __builtin_amdgcn_readlane(id, j) == id;
  first = (uint32_t)__builtin_amdgcn_ballot_w64(!dup) & 0xFFFFu;
  return id;
}

// u parts [KS][T][R].  grid: rank tiles of 16 RT times KS, slots, token tiles; a
// workgroup takes every gridDim.y-th of its tile's distinct adapters.
template <int RT>
__global__ void __launch_bounds__(kThreads)
lora_shrink_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int* __restrict__ ids,
                   float* __restrict__ u, int* __restrict__ order, int K, int T, int R, int L, int KS) {
  __shared__ float red[kWaves][RT][16][20];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int ks = blockIdx.x % KS, t0 = blockIdx.z * 16, r0 = blockIdx.x / KS * (16 * RT);
  // order: the tokens by adapter, then by number (those without one last), in
  // workgroups of their own behind the others.  A token's place is the count
  // of tokens before it: 32 lanes a token, 16 tokens a workgroup.
  const int tiles = (T + 15) >> 4;
  if ((int)blockIdx.z >= tiles) {
    const int tile = ((blockIdx.z - tiles) * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
    if (tile >= tiles) return;
    const int t = min(16 * tile + (int)(threadIdx.x >> 5), T - 1);
    const uint32_t own = (uint32_t)ids[t];
    int before = 0;
#pragma unroll 8
    for (int o = threadIdx.x & 31; o < T; o += 32) {
      const uint32_t other = (uint32_t)ids[o];
      before += other < own || (other == own && o < t);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) before += __shfl_xor(before, m);
    order[before] = t;  // (tokens past the last repeat it)
    return;
  }

  uint32_t todo;
  const int id = tile_adapters(t0 + li < T ? ids[t0 + li] : -1, L, li, todo);

  // this wave's run of 32-k steps
  const int steps = K >> 5, parts = KS * kWaves, part = ks * kWaves + wave;
  const int sb = (int)((int64_t)steps * part / parts), se = (int)((int64_t)steps * (part + 1) / parts);
  // four lanes load 64 bytes of one row (neighbouring lanes on different rows
  // occupy the address unit several times as long); a lane exchange hands
  // lane (li, lq) its piece.  Rows past the last repeat it.
  const int lr = lane >> 2, lp = 8 * (lane & 3), src4 = (4 * li + lq) * 4;
  const uint16_t* xp = x + (size_t)min(t0 + lr, T - 1) * K + lp;
  for (int slot = 0; todo != 0; ++slot) {
    const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
    todo &= todo - 1;
    if (slot % gridDim.y != blockIdx.y) continue;
    const uint16_t* ap[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) ap[r] = a + ((size_t)ad * R + min(r0 + 16 * r + lr, R - 1)) * K + lp;
    f32x4_t acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s = sb; s < se; s += 4) {
      // four steps' loads in flight (steps past the run repeat the last and
      // are not used)
      u32x4_t xv[4], av[RT][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const size_t k = 32 * (size_t)min(s + j, se - 1);
        xv[j] = *reinterpret_cast<const u32x4_t*>(xp + k);
#pragma unroll
        for (int r = 0; r < RT; ++r) av[r][j] = *reinterpret_cast<const u32x4_t*>(ap[r] + k);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (s + j >= se) break;
        const u32x4_t xo = lane_piece(xv[j], src4);
#pragma unroll
        for (int r = 0; r < RT; ++r) acc[r] = mfma(xo, lane_piece(av[r][j], src4), acc[r]);
      }
    }
    __syncthreads();  // (the adapter before is summed)
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
}

// The same for few tokens: a workgroup makes RPW rank values of one token with
// its own adapter (no tile, so tokens that share one read it again, from the
// caches), its four waves sharing K: 2.6 us where the tiles take 4 at one
// token and rank 16.  u: float [T][R].  grid: R / RPW, T.
template <int RPW>
__global__ void __launch_bounds__(256)
lora_dots_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const int* __restrict__ ids,
                 float* __restrict__ u, int K, int R, int L) {
  __shared__ float part[4][RPW];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.y, r0 = blockIdx.x * RPW;
  const int id = ids[t];
  if ((uint32_t)id >= (uint32_t)L) return;
  const uint16_t* xr = x + (size_t)t * K;
  const uint16_t* ar = a + ((size_t)id * R + r0) * K;
  float sum[RPW];
#pragma unroll
  for (int i = 0; i < RPW; ++i) sum[i] = 0.f;
#pragma unroll 4
  for (int k = 8 * (64 * wave + lane); k < K; k += 2048) {
    const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(xr + k);
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const u32x4_t av = *reinterpret_cast<const u32x4_t*>(ar + (size_t)i * K + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t aw = av[j], xw = xv[j];
        sum[i] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, aw), __builtin_bit_cast(bf16x2_t, xw), sum[i], false);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RPW; ++i) {
    const float v = (float)sum64_lanes((double)sum[i]);
    if (lane == 0) part[wave][i] = v;
  }
  __syncthreads();
  if ((int)threadIdx.x < RPW) {
    const int i = threadIdx.x;
    u[(size_t)t * R + r0 + i] = (part[0][i] + part[1][i]) + (part[2][i] + part[3][i]);
  }
}

// The base product's weight and activations, for sums that left the range.
struct BaseWeight {
  const uint16_t* x;
  const uint8_t* lo;
  const uint8_t* hi;
  const uint8_t* sc;
  int fmt, K;
};
__device__ double exact_base(const BaseWeight& w, int n, int t) {
  switch (w.fmt) {
    case FMT_Q4: return exact_sum_call<FMT_Q4>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
    case FMT_Q5: return exact_sum_call<FMT_Q5>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
    case FMT_Q6: return exact_sum_call<FMT_Q6>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
    case FMT_W8: return exact_sum_call<FMT_W8>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
    case FMT_NVFP4: return exact_sum_call<FMT_NVFP4>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
    default: return exact_sum_call<FMT_BF16>(w.x, w.lo, w.hi, w.sc, w.K, n, t);
  }
}

// s sum_r B[r] u[r] in binary32 (b: one row of an adapter, u: a token's first
// part of KS, `part` floats apart)
__device__ float adapter_term(const uint16_t* b, const float* u, size_t part, int R, int KS, float scale) {
  float v = 0.f;
  for (int r = 0; r < R; ++r) {
    float ur = u[r];
    for (int k = 1; k < KS; ++k) ur += u[k * part + r];
    v = __builtin_fmaf(bf16_bits_to_f32(b[r]), ur, v);
  }
  return scale * v;
}

// A workgroup takes 16 tokens and every gridDim.x-th block of 64 NB rows; a
// wave 16 NB of a block's rows.  RS: 32-rank steps that cover R.  The base
// sums come in, and y goes out, in runs of 256 NB bytes of a token's row (a
// wave takes four tokens), the next block's sums asked for before the
// current one is written; the adapters' term crosses over to that order
// through LDS (two buffers, a barrier per block).  Where a tile's tokens have
// several adapters, the next adapter's rows are on their way while one's are
// used, as far as registers go (179 mixed tokens of 24 adapters of rank 32 in
// their own order, 6443 rows: 13 us against 17).
template <int RS, int NB>
__global__ void __launch_bounds__(256)
lora_finish_kernel(const uint16_t* __restrict__ b, const float* __restrict__ scale, const int* __restrict__ ids,
                   const float* __restrict__ u, const int* __restrict__ order, SumSource base,
                   uint16_t* __restrict__ y, int N, int T, int R, int L,
                   int KS, int vec, BaseWeight w) {
  constexpr int ROWS = 64 * NB;  // of a block
  constexpr int D = RS * NB <= 2 ? 4 : RS * NB <= 8 ? 2 : 1;  // adapters whose rows are in registers
  __shared__ __attribute__((aligned(16))) float term[2][16][ROWS + 4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int t0 = blockIdx.y * 16;
  // this lane's token and those of the wave's rows (tokens past the last repeat it)
  const int tl = order != nullptr ? order[min(t0 + li, T - 1)] : min(t0 + li, T - 1);
  int tw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) tw[i] = __builtin_amdgcn_readlane(tl, 4 * wave + i);

  // This lane's base sums of a block: tokens tw[i], rows nl .. nl + NB - 1
  typedef float fv_t __attribute__((ext_vector_type(NB)));
  struct Sums {
    fv_t v[4];
  };
  auto load_sums = [&](int nb0) __device__ {
    Sums s;
    const int nl = nb0 + NB * lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* p = base.part + (size_t)tw[i] * N + nl;
      s.v[i] = fv_t{};
      if (vec) {
        if (nl < N) s.v[i] = *reinterpret_cast<const fv_t*>(p);
      } else {
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (nl + j < N) s.v[i][j] = p[j];
      }
    }
    for (int k = 1; k < base.ks; ++k) {  // the other slices of a K split, in order
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* p = base.part + (size_t)k * base.stride + (size_t)tw[i] * N + nl;
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (nl + j < N) s.v[i][j] += p[j];
      }
    }
    return s;
  };
  Sums cur = load_sums(blockIdx.x * ROWS);

  uint32_t first;
  const int id = tile_adapters(t0 + li < T ? ids[tl] : -1, L, li, first);
  // token li's s_a u as two bf16 parts, ranks 32 s + 8 lq .. + 7 of step s
  u32x4_t uh[RS], ul[RS];
  const float sc = id >= 0 && scale != nullptr ? scale[id] : 1.0f;
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    f32x4_t v0 = {0.f, 0.f, 0.f, 0.f}, v1 = v0;
    if (id >= 0 && 32 * r + 8 * lq < R) {
      const f32x4_t* p = reinterpret_cast<const f32x4_t*>(u + (size_t)tl * R + 32 * r + 8 * lq);
      v0 = p[0];
      v1 = p[1];
      if (KS > 1) {
        f32x4_t p0[kMaxSplit], p1[kMaxSplit];  // (all parts in flight; past the last, the last again)
#pragma unroll
        for (int k = 1; k < kMaxSplit; ++k) {
          const f32x4_t* q = p + (size_t)min(k, KS - 1) * T * (R >> 2);
          p0[k] = q[0];
          p1[k] = q[1];
        }
#pragma unroll
        for (int k = 1; k < kMaxSplit; ++k)
          if (k < KS) {
            v0 += p0[k];
            v1 += p1[k];
          }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h0, l0, h1, l1;
      const f32x4_t v = j < 2 ? v0 : v1;
      split_bf16(sc * v[2 * (j & 1)], h0, l0);
      split_bf16(sc * v[2 * (j & 1) + 1], h1, l1);
      uh[r][j] = h0 | (h1 << 16);
      ul[r][j] = l0 | (l1 << 16);
    }
  }
  int te[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) te[i] = base.texp != nullptr ? base.texp[tw[i]] : 0;

  int buf = 0;
  float left = 0.f;  // NaN when one of this lane's outputs is not finite (infinity and NaN times zero)
  for (int nb0 = blockIdx.x * ROWS; nb0 < N; nb0 += gridDim.x * ROWS, buf ^= 1) {
    const int n0 = nb0 + wave * (16 * NB), nl = nb0 + NB * lane;
    int re[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) re[j] = base.texp != nullptr && nl + j < N ? base.rexp[nl + j] : 0;
    f32x4_t acc[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int last = max(N - 1 - n0, 0);  // rows past the last repeat it and are not stored
    // adapter by adapter, the rows of the next D - 1 asked for ahead
    uint32_t todo = n0 < N ? first : 0u, ask = todo;
    u32x4_t bv[D][RS][NB];
    auto load_rows = [&](u32x4_t (&v)[RS][NB]) __device__ {
      if (ask == 0) return;
      const int ad = __builtin_amdgcn_readlane(id, __builtin_ctz(ask));
      ask &= ask - 1;
      const uint16_t* bp = b + ((size_t)ad * N + n0) * R + 8 * lq;
#pragma unroll
      for (int r = 0; r < RS; ++r)
#pragma unroll
        for (int c = 0; c < NB; ++c) {
          v[r][c] = u32x4_t{0u, 0u, 0u, 0u};
          if (32 * r + 8 * lq < R)
            v[r][c] = *reinterpret_cast<const u32x4_t*>(bp + (size_t)min(16 * c + li, last) * R + 32 * r);
        }
    };
#pragma unroll
    for (int j = 0; j < D - 1; ++j) load_rows(bv[j]);
    while (todo != 0) {
#pragma unroll
      for (int j = 0; j < D; ++j) {
        if (todo == 0) break;
        load_rows(bv[(j + D - 1) % D]);
        f32x4_t d[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) d[c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            d[c] = mfma(bv[j][r][c], uh[r], d[c]);
            d[c] = mfma(bv[j][r][c], ul[r], d[c]);
          }
        // (a token keeps its own adapter's products only: taken, not added, so
        // that an infinity in one request's adapter stays in its own rows)
        const bool mine = id == __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        todo &= todo - 1;
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][i] = mine ? d[c][i] : acc[c][i];
      }
    }
    // rows 16 NB wave + 16 c + 4 lq .. + 3 of token li
#pragma unroll
    for (int c = 0; c < NB; ++c)
      *reinterpret_cast<f32x4_t*>(&term[buf][li][16 * NB * wave + 16 * c + 4 * lq]) = acc[c];
    Sums next = cur;
    if (nb0 + gridDim.x * ROWS < N) next = load_sums(nb0 + gridDim.x * ROWS);
    // (not __syncthreads, which would wait for those loads)
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    // the base sum, the one rounding, the store
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t0 + 4 * wave + i >= T) break;
      uint16_t h[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        // (the many-token route's sums carry a power of two per token and row)
        const float f = __builtin_ldexpf(cur.v[i][j], te[i] - re[j]);
        const float v = f + term[buf][4 * wave + i][NB * lane + j];
        left = __builtin_fmaf(v, 0.f, left);
        h[j] = f32_to_bf16_rne(v);
      }
      uint16_t* o = y + (size_t)tw[i] * N + nl;
      if (vec && NB == 4) {
        if (nl < N)
          *reinterpret_cast<u32x2_t*>(o) =
              u32x2_t{h[0] | ((uint32_t)h[1 % NB] << 16), h[2 % NB] | ((uint32_t)h[3 % NB] << 16)};
      } else {
#pragma unroll
        for (int j = 0; j < NB; ++j)
          if (nl + j < N) o[j] = h[j];
      }
    }
    cur = next;
  }
  if (__builtin_amdgcn_ballot_w64(left != left) == 0) return;

  // Rare: an output that is not finite is formed again, by the lane that
  // stored it: a base sum that is not finite exactly, as the base product's own
  // kernels do, the term in binary32 as the rank values are (an infinity of B
  // times their two parts is NaN where the second part is zero or of the other
  // sign).
  for (int nb0 = blockIdx.x * ROWS; nb0 < N; nb0 += gridDim.x * ROWS) {
#pragma unroll 1
    for (int o = 0; o < 4 * NB; ++o) {
      const int i = o / NB, n = nb0 + NB * lane + o % NB;
      const int t = __builtin_amdgcn_readlane(tl, 4 * wave + i);
      if (t0 + 4 * wave + i >= T) break;
      if (n >= N || (y[(size_t)t * N + n] & 0x7F80u) != 0x7F80u) continue;
      float v = base.part[(size_t)t * N + n];
      for (int k = 1; k < base.ks; ++k) v += base.part[(size_t)k * base.stride + (size_t)t * N + n];
      if (base.texp != nullptr) v = __builtin_ldexpf(v, base.texp[t] - base.rexp[n]);
      if (!__builtin_isfinite(v)) v = (float)exact_base(w, n, t);
      const uint32_t own = (uint32_t)ids[t];
      if (own < (uint32_t)L)
        v += adapter_term(b + ((size_t)own * N + n) * R, u + (size_t)t * R, (size_t)T * R, R, KS,
                          scale != nullptr ? scale[own] : 1.0f);
      y[(size_t)t * N + n] = f32_to_bf16_rne(v);
    }
  }
}

// The shrink's rank tiles per workgroup (two share the activations' loads) and
// the workgroups that share K: about one per CU where the tokens of a tile
// have one adapter.  (1024 tokens of rank 32 at K = 5120: 14 us without the
// split, when 64 workgroups each read 480 KB.)
struct ShrinkPlan {
  int rt, ks;
};
ShrinkPlan shrink_plan(int64_t k, int64_t t, int64_t r) {
  if (lora_few(t, r)) return ShrinkPlan{1, 1};
  const int rt = r <= 16 ? 1 : 2;
  int64_t ks = 256 / ((t + 15) / 16 * ((r + 16 * rt - 1) / (16 * rt)));
  if (ks > kMaxSplit) ks = kMaxSplit;
  if (ks > k / (32 * kWaves)) ks = k / (32 * kWaves);
  return ShrinkPlan{rt, ks < 1 ? 1 : (int)ks};
}

// Whether the finish takes the tokens by adapter (the shrink makes the order,
// T / 32 comparisons a lane).
constexpr int64_t kOrderT = 4096;
bool lora_ordered(int64_t t, int64_t rank, int64_t adapters) {
  return t > 16 && t <= kOrderT && adapters > 1 && !lora_few(t, rank);
}
// the order, behind the rank values
int* lora_order(const LoraArgs& a, const float* u) {
  if (!lora_ordered(a.t, a.rank, a.adapters)) return nullptr;
  const size_t bytes = lora_u_bytes(a.k, a.t, a.rank, a.adapters) - (((size_t)a.t * 4 + 255) & ~(size_t)255);
  return reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(const_cast<float*>(u)) + bytes);
}

template <int RS>
hipError_t launch_finish(const LoraArgs& a, const float* u, const SumSource& base, hipStream_t s) {
  const int ks = shrink_plan(a.k, a.t, a.rank).ks;
  const int64_t tiles = (a.t + 15) / 16;
  const int vec = (a.n & 3) == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
  // four 16-row tiles per wave share the token operand; one where that would
  // leave CUs idle.  About three workgroups per CU.
  const bool wide = tiles * ((a.n + 255) / 256) >= 256;
  const int64_t blocks = (a.n + (wide ? 255 : 63)) / (wide ? 256 : 64);
  const int64_t most = 768 / tiles > 1 ? 768 / tiles : 1;
  const dim3 grid((unsigned)(blocks < most ? blocks : most), (unsigned)tiles);
  const BaseWeight w{static_cast<const uint16_t*>(a.x), static_cast<const uint8_t*>(a.w),
                     static_cast<const uint8_t*>(a.w_hi), static_cast<const uint8_t*>(a.w_sc), a.fmt, (int)a.k};
  auto go = [&](auto kern) {
    kern<<<grid, dim3(256), 0, s>>>(static_cast<const uint16_t*>(a.b), static_cast<const float*>(a.scale),
                                    static_cast<const int*>(a.ids), u, lora_order(a, u), base, static_cast<uint16_t*>(a.y), (int)a.n,
                                    (int)a.t, (int)a.rank, (int)a.adapters, ks, vec, w);
  };
  if (wide) go(lora_finish_kernel<RS, 4>);
  else go(lora_finish_kernel<RS, 1>);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_dots(const LoraArgs& a, float* u, hipStream_t s) {
  // one rank value a workgroup while there are few
  const int rpw = a.t * a.rank <= 256 ? 1 : 4;
  auto go = [&](auto kern) {
    kern<<<dim3((unsigned)(a.rank / rpw), (unsigned)a.t), dim3(256), 0, s>>>(
        static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.a), static_cast<const int*>(a.ids), u,
        (int)a.k, (int)a.rank, (int)a.adapters);
  };
  if (rpw == 1) go(lora_dots_kernel<1>);
  else go(lora_dots_kernel<4>);
  return hipGetLastError();
}

size_t lora_u_bytes(int64_t k, int64_t t, int64_t rank, int64_t adapters) {
  const size_t u = ((size_t)shrink_plan(k, t, rank).ks * (size_t)t * (size_t)rank * 4 + 255) & ~(size_t)255;
  return lora_ordered(t, rank, adapters) ? u + (((size_t)t * 4 + 255) & ~(size_t)255) : u;
}

hipError_t launch_lora_shrink(const LoraArgs& a, float* u, hipStream_t s) {
  if (lora_few(a.t, a.rank)) return launch_lora_dots(a, u, s);
  const auto [rt, ks] = shrink_plan(a.k, a.t, a.rank);
  const int64_t tiles = (a.t + 15) / 16;
  // A tile's adapters in workgroups of their own while there are few tiles (a
  // workgroup without one costs its launch)
  int64_t slots = a.t < a.adapters ? a.t : a.adapters;
  if (slots > 16) slots = 16;
  while (slots > 1 && slots * tiles > 64) slots >>= 1;
  const int64_t ranks = (a.rank + 16 * rt - 1) / (16 * rt) * ks;
  const int64_t extra = lora_order(a, u) != nullptr ? (tiles + ranks * slots - 1) / (ranks * slots) : 0;
  const dim3 grid((unsigned)ranks, (unsigned)slots, (unsigned)(tiles + extra));
  auto go = [&, ks = ks](auto kern) {
    kern<<<grid, dim3(kThreads), 0, s>>>(static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.a),
                                         static_cast<const int*>(a.ids), u, lora_order(a, u), (int)a.k, (int)a.t,
                                         (int)a.rank, (int)a.adapters, ks);
  };
  if (rt == 1) go(lora_shrink_kernel<1>);
  else go(lora_shrink_kernel<2>);
  return hipGetLastError();
}

hipError_t launch_lora_finish(const LoraArgs& a, const float* u, const SumSource& base, hipStream_t s) {
  if (a.rank <= 32) return launch_finish<1>(a, u, base, s);
  if (a.rank <= 64) return launch_finish<2>(a, u, base, s);
  if (a.rank <= 128) return launch_finish<4>(a, u, base, s);
  return launch_finish<8>(a, u, base, s);
}

}  // namespace q4lin
