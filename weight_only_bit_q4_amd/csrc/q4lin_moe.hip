// q4lin_moe.hip -- a mixture-of-experts layer for few tokens, experts in
// Q4_G64_FP16:
//
//     l[t][e] = sum_k router[e][k] x[t][k],  p = softmax over e,
//     the top_k largest l of a token (equals: the lowest e) with weights p,
//     h_j = silu(Wg_e x) * (Wu_e x),         e = ids[t][j],
//     y[t] = bf16( sum_j weights[t][j] Wd_e h_j ).
//
// A choice (t, j) is a "pair" p = t top_k + j.  Launches: the
// logits and the choice (one kernel for small routers), the gate and up
// products with the gate applied, the down products of every pair, and their
// weighted sum per token; for a few tokens the choice is made inside the gate
// and up kernel and the sum inside the down kernel.  A pair
// whose id is outside 0..E-1 takes part in nothing.
//
// Expert products.  Their floor is the weight stream: 34 bytes per 64 weights
// of each expert that some token chose.  Three kernels share the arithmetic
// and differ in what a wave holds (the figures stand at the choices):
//   gated:    gate and up rows of up to 16 activation rows a pass; the four
//             waves of a workgroup share K, each with an LDS ring of its own;
//   down_few: down products of a few tokens, sixteen waves over K, y written
//             at once: every token reads its experts' rows for itself;
//   wide:     down products of several tokens, and the gate and up products
//             where an expert has many pairs: eight waves share the staged
//             activations, up to 32 activation rows a pass.
// The arithmetic is that of the library's other matrix-core routes: exact
// bf16 values 128 + q, products of a constant all-8 operand through the same
// instructions subtracted, the group's scale applied in binary32; the waves'
// partials are summed in a fixed order, so that a call repeats to the bit.
// h is kept as two bf16 parts (16 significant bits), as two activation rows
// per pair: one bf16 would cost as much precision as the store of y.  The sums
// of 128 + q leave binary32 where |x| or |h| reaches 2^114: such a token's row
// is not finite (it is not formed again).
#include "q4lin_kernels.h"
#include "q4lin_mfma16.h"

namespace q4lin {
namespace {

using namespace mfma16;

// ---------------------------------------------------------------------------
// Routing
// ---------------------------------------------------------------------------
constexpr int kRouteThreads = 1024;
constexpr int kMaxExperts = 1024;

__device__ __forceinline__ float dot8(u32x4_t a, u32x4_t b) {
  float d = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, (uint32_t)a[i]),
                                        __builtin_bit_cast(bf16x2_t, (uint32_t)b[i]), d, false);
  return d;
}

// Products of EPW rows of the router with TPW tokens over the k of one wave
// (pieces of 8 from 8 (64 part + lane), 512 parts apart): exact bf16
// products, eight at a time summed in binary32 and those in binary64, so
// that the order of two experts is that of their exact logits but for
// differences near 2^-24 of the terms.
template <int EPW, int TPW>
__device__ __forceinline__ void logit_sums(const uint16_t* const (&r)[EPW], const uint16_t* const (&x)[TPW], int K,
                                           int part, int parts, int lane, double (&sum)[TPW][EPW]) {
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int i = 0; i < EPW; ++i) sum[t][i] = 0.0;
#pragma unroll 4
  for (int k = 8 * (64 * part + lane); k < K; k += 512 * parts) {
    u32x4_t rv[EPW], xv[TPW];
#pragma unroll
    for (int i = 0; i < EPW; ++i) rv[i] = *reinterpret_cast<const u32x4_t*>(r[i] + k);
#pragma unroll
    for (int t = 0; t < TPW; ++t) xv[t] = *reinterpret_cast<const u32x4_t*>(x[t] + k);
#pragma unroll
    for (int t = 0; t < TPW; ++t)
#pragma unroll
      for (int i = 0; i < EPW; ++i) sum[t][i] += (double)dot8(rv[i], xv[t]);
  }
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int i = 0; i < EPW; ++i) sum[t][i] = sum64_lanes(sum[t][i]);
}

// A token's choice by a single wave.  An expert's key is its logit's bits in
// an order-preserving form, the lowest eleven bits of the fraction giving way
// to the expert's number (equals: the lowest first; a NaN lowest).
__device__ __forceinline__ uint64_t max64_lanes(uint64_t v) {
  auto step = [&](uint64_t o) __device__ { v = o > v ? o : v; };
  auto dpp = [&](auto c) __device__ {
    constexpr int C = decltype(c)::value;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, C, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), C, 0xF, 0xF, false);
    return ((uint64_t)hi << 32) | lo;
  };
  step(dpp(Slot<0xB1>{}));
  step(dpp(Slot<0x4E>{}));
  step(dpp(Slot<0x141>{}));
  step(dpp(Slot<0x140>{}));
  auto rows = [&](const auto& l, const auto& h) __device__ {
    const uint64_t a = ((uint64_t)h[0] << 32) | l[0], b = ((uint64_t)h[1] << 32) | l[1];
    v = a > b ? a : b;
  };
  rows(__builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false),
       __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false));
  rows(__builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false),
       __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false));
  return v;
}
__device__ __forceinline__ uint64_t route_key(double l, int e) {
  const uint64_t u = __builtin_bit_cast(uint64_t, l);
  const uint64_t o = l != l ? 0 : (u >> 63) ? ~u : u | 0x8000000000000000ull;
  return (o & ~2047ull) | (uint64_t)(kMaxExperts - e);
}
// the expert of rank n - 1 by its key (keys of experts lane, lane + 64, ...);
// with `chosen`, all n
template <int B>
__device__ __forceinline__ int choose_rank(uint64_t (&key)[B], int n, int lane, int* chosen) {
  int e = 0;
  for (int j = 0; j < n; ++j) {
    uint64_t best = key[0];
#pragma unroll
    for (int b = 1; b < B; ++b) best = key[b] > best ? key[b] : best;
    best = max64_lanes(best);
    e = kMaxExperts - (int)((uint32_t)best & 2047u);
#pragma unroll
    for (int b = 0; b < B; ++b) key[b] = key[b] == best ? 0 : key[b];
    if (chosen != nullptr && lane == 0) chosen[j] = e;
  }
  return e;
}
// a token's choice of n experts, from its E <= 64 B logits; chosen: n numbers of LDS
template <int B>
__device__ __forceinline__ void choose_one(const double* lg, int E, int n, int lane, int renorm, int* chosen,
                                           int* __restrict__ ids, float* __restrict__ weights) {
  uint64_t key[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int i = 64 * b + lane;
    const uint64_t k = route_key(lg[min(i, E - 1)], i);
    key[b] = i < E ? k : 0;
  }
  choose_rank<B>(key, n, lane, chosen);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  // the softmax runs over the chosen experts, or over all; lane j: ranks j, j + 64, ...
  const double l0 = lg[chosen[min(lane, n - 1)]];
  const uint64_t tb = __builtin_bit_cast(uint64_t, l0);
  const double top = __builtin_bit_cast(
      double, (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)tb) |
                  ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(tb >> 32)) << 32));
  const double p0 = exp(l0 - top);
  double sum = renorm && lane < n ? p0 : 0.0;
  for (int i = renorm ? lane + 64 : lane; i < (renorm ? n : E); i += 64) sum += exp(lg[renorm ? chosen[i] : i] - top);
  sum = sum64_lanes(sum);
  for (int j = lane; j < n; j += 64) {
    ids[j] = chosen[j];
    weights[j] = (float)((j < 64 ? p0 : exp(lg[chosen[j]] - top)) / sum);
  }
}

// Small routers: one workgroup per token makes the logits and the choice
__global__ void __launch_bounds__(kRouteThreads)
moe_route_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ router, int* __restrict__ ids,
                 float* __restrict__ weights, int K, int E, int top_k, int renorm) {
  constexpr int kRouteWaves = kRouteThreads / 64;
  __shared__ double lg[kMaxExperts];
  __shared__ int chosen[kMaxExperts];
  __shared__ double part[kRouteWaves][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t t = blockIdx.x;
  const uint16_t* xr[1] = {x + t * K};
  // four experts a wave, the waves left over sharing their k
  const int quads = (E + 3) / 4, parts = quads < kRouteWaves ? kRouteWaves / quads : 1;
  for (int q = wave / parts; q < quads; q += kRouteWaves / parts) {
    const uint16_t* r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = router + (size_t)min(4 * q + i, E - 1) * K;
    double sum[1][4];
    logit_sums<4, 1>(r, xr, K, wave % parts, parts, lane, sum);
    if (lane < 4) {
      const double v = lane == 0 ? sum[0][0] : lane == 1 ? sum[0][1] : lane == 2 ? sum[0][2] : sum[0][3];
      if (parts > 1) part[wave][lane] = v;
      else if (4 * q + lane < E) lg[4 * q + lane] = v;
    }
  }
  if (parts > 1) {
    __syncthreads();
    const int e = threadIdx.x;
    if (e < E) {
      double v = 0.0;
      for (int p = 0; p < parts; ++p) v += part[(e >> 2) * parts + p][e & 3];
      lg[e] = v;
    }
  }
  __syncthreads();
  if (wave != 0) return;
  if (E <= 256) choose_one<4>(lg, E, top_k, lane, renorm, chosen, ids + t * top_k, weights + t * top_k);
  else choose_one<kMaxExperts / 64>(lg, E, top_k, lane, renorm, chosen, ids + t * top_k, weights + t * top_k);
}

// Larger ones: the logits by waves over the whole chip, then the choices.
// A wave takes EPW experts and TPW tokens; or (one_logit) a workgroup takes
// one expert and one token, its four waves sharing K.
__global__ void __launch_bounds__(256)
moe_one_logit_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ router, double* __restrict__ lg,
                     int K, int E) {
  __shared__ double part[4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint16_t *r[1] = {router + (size_t)blockIdx.x * K}, *xr[1] = {x + (size_t)blockIdx.y * K};
  double sum[1][1];
  logit_sums<1, 1>(r, xr, K, wave, 4, lane, sum);
  if (lane == 0) part[wave] = sum[0][0];
  __syncthreads();
  if (threadIdx.x == 0) lg[(size_t)blockIdx.y * E + blockIdx.x] = (part[0] + part[1]) + (part[2] + part[3]);
}
template <int EPW, int TPW>
__global__ void __launch_bounds__(256)
moe_logits_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ router, double* __restrict__ lg, int K,
                  int E, int T) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int e0 = (blockIdx.y * 4 + wave) * EPW, t0 = blockIdx.x * TPW;
  if (e0 >= E) return;
  const uint16_t *r[EPW], *xr[TPW];
#pragma unroll
  for (int i = 0; i < EPW; ++i) r[i] = router + (size_t)min(e0 + i, E - 1) * K;
#pragma unroll
  for (int t = 0; t < TPW; ++t) xr[t] = x + (size_t)min(t0 + t, T - 1) * K;
  double sum[TPW][EPW];
  logit_sums<EPW, TPW>(r, xr, K, 0, 1, lane, sum);
#pragma unroll
  for (int t = 0; t < TPW; ++t)
#pragma unroll
    for (int i = 0; i < EPW; ++i)
      if (lane == 0 && t0 + t < T && e0 + i < E) lg[(size_t)(t0 + t) * E + e0 + i] = sum[t][i];
}
// one wave per token
template <int B>
__global__ void __launch_bounds__(64)
moe_choose_kernel(const double* __restrict__ lg, int* __restrict__ ids, float* __restrict__ weights, int E, int top_k,
                  int renorm) {
  __shared__ int chosen[64 * B];
  const size_t t = blockIdx.x;
  choose_one<B>(lg + t * E, E, top_k, threadIdx.x, renorm, chosen, ids + t * top_k, weights + t * top_k);
}

// ---------------------------------------------------------------------------
// Expert products
// ---------------------------------------------------------------------------
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPairGrid = 64;

// Code dword w (k0..k7) -> exact bf16 128 + q in natural order: byte b gives
// its low nibble and, through w >> 4, its high nibble
__device__ __forceinline__ u32x4_t q4_natural(uint32_t w) {
  const uint32_t u = w >> 4;
  u32x4_t r;
  r.x = and_or(__builtin_amdgcn_perm(u, w, 0x04040000u), 0x000F000Fu, 0x43004300u);
  r.y = and_or(__builtin_amdgcn_perm(u, w, 0x05050101u), 0x000F000Fu, 0x43004300u);
  r.z = and_or(__builtin_amdgcn_perm(u, w, 0x06060202u), 0x000F000Fu, 0x43004300u);
  r.w = and_or(__builtin_amdgcn_perm(u, w, 0x07070303u), 0x000F000Fu, 0x43004300u);
  return r;
}
// the same in the order k0 k4 k1 k5 k2 k6 k3 k7 (two instructions fewer):
// for activations that were written in that order
__device__ __forceinline__ u32x4_t q4_paired(uint32_t w) {
  return u32x4_t{and_or(w, 0x000F000Fu, 0x43004300u), and_or(w >> 4, 0x000F000Fu, 0x43004300u),
                 and_or(w >> 8, 0x000F000Fu, 0x43004300u), and_or(w >> 12, 0x000F000Fu, 0x43004300u)};
}
// place of value k (0..7) in that order
__device__ __forceinline__ int paired_place(int k) { return k < 4 ? 2 * k : 2 * k - 7; }

// Loads before it are issued before loads after it, so that a wait for one
// stage's loads need not wait for those of the stage behind it
__device__ __forceinline__ void in_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// bf16 values k0..k7 into the paired order
__device__ __forceinline__ u32x4_t to_paired(u32x4_t v) {
  return u32x4_t{__builtin_amdgcn_perm(v.z, v.x, 0x05040100u), __builtin_amdgcn_perm(v.z, v.x, 0x07060302u),
                 __builtin_amdgcn_perm(v.w, v.y, 0x05040100u), __builtin_amdgcn_perm(v.w, v.y, 0x07060302u)};
}

// The K loop works in stages of 256 k (four scale groups), two in flight.
// What a wave holds of a stage: the codes of its R row tiles (16 weight rows
// each) in its LDS ring, the activations of its activation tiles and the
// rows' scales in registers.
//   * Codes: eight lanes copy 128 bytes of one row (a load in which
//     neighbouring lanes take different rows occupies the address unit
//     several times as long); piece p of row i lies at 16-byte position
//     8 i + (p ^ (i & 7)), so that the sixteen rows of an operand read
//     spread over the banks.
//   * Scales: every second stage lane r loads the eight of the wave's row r,
//     16 bytes from the dword that holds the first, and the dword behind
//     them where rows of an odd number of groups start in the middle of one.
//   * Activations, GP = 1 (up to 16 activation rows): four lanes load from
//     one row; a lane exchange hands them over.
//   * Activations, GP = 2 or 4 (at most 8 or 4 activation rows): a tile's 16
//     rows are those rows times GP scale groups, zero but for the products
//     of the own group.  A product of GP groups' codes with such operands
//     keeps the groups' sums apart in different rows of one accumulator, so
//     that the scales (lane l: row l % 16, the group of its accumulator
//     rows) cost one multiplication for GP groups.
constexpr int kTileStage = 16 * 128;  // code bytes of a row tile in a stage

// where this lane copies codes from (rows lane / 8 of a tile's upper or lower
// half), and where it reads its 8 code bytes of group g in a slot: row li,
// byte 32 g + 8 lq
__device__ __forceinline__ uint32_t code_offset(uint32_t crow, int lane) {
  return (uint32_t)(lane >> 3) * crow + 16u * ((lane & 7) ^ (lane >> 3));
}
__device__ __forceinline__ int code_read(int li, int lq, int g) {
  return li * 128 + 16 * ((2 * g + (lq >> 1)) ^ (li & 7)) + 8 * (lq & 1);
}

template <int GP>
struct Acts {
  u32x4_t v[8 / GP];
};

// The scales of a wave's rows: 16 RT rows of one plane (and, gate and up, of
// a second one).  first: index of the first row's first scale in its plane.
template <int R, bool DOWN>
struct RowScales {
  static constexpr int PL = DOWN ? 1 : 2, RT = R / PL;
  static constexpr int LOADS = 2 * PL;
  struct Regs {
    u32x4_t v[PL];
    uint32_t next[PL];
  };
  rsrc_t r[PL];
  uint32_t off[PL], shift;
  int G;
  bool skewed;
  __device__ __forceinline__ RowScales(const uint16_t* scales0, const uint16_t* scales1, size_t first, int rows,
                                       int groups, int lane)
      : G(groups) {
    const uint32_t srow = (uint32_t)G * 2;
    skewed = (G & 1) != 0;
    shift = 0;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const uintptr_t a = reinterpret_cast<uintptr_t>((p ? scales1 : scales0) + first);
      const uint32_t skew = (uint32_t)(a & 2);  // the dword that holds the first scale starts 2 bytes before it
      r[p] = make_rsrc(reinterpret_cast<const void*>(a - skew), rows > 0 ? (skew + (uint32_t)rows * srow + 3u) & ~3u : 0u);
      const int row = lane - 16 * RT * p;
      const bool mine = row >= 0 && row < rows && row < 16 * RT;
      const uint32_t o = skew + (uint32_t)row * srow;
      off[p] = mine ? o & ~3u : kNowhere;
      shift = mine ? (o & 2) * 8 : shift;
      skewed |= skew != 0;
    }
  }
  // the scales of stages s and s + 1 (offsets past every range read as zeros)
  __device__ __forceinline__ void load(Regs& L, int s, int se) const {
    const uint32_t away = s < se ? 0u : kNowhere, away_next = s < se && skewed ? 0u : kNowhere;
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const uint32_t o = off[p] + 8u * (uint32_t)s;
      L.v[p] = __builtin_amdgcn_raw_buffer_load_b128(r[p], o | away, 0, 0);
      L.next[p] = __builtin_amdgcn_raw_buffer_load_b32(r[p], (o + 16) | away_next, 0, 0);
    }
    in_order();
  }
  // those of row `lane`, two groups a dword, zero past K
  __device__ __forceinline__ void rows(const Regs& L, int s, uint32_t (&d)[4]) const {
    u32x4_t v = L.v[0];
    uint32_t n = L.next[0];
    if constexpr (PL > 1) {
      v = v | L.v[1];
      n |= L.next[1];
    }
    if (skewed)
      v = u32x4_t{__builtin_amdgcn_alignbit(v.y, v.x, shift), __builtin_amdgcn_alignbit(v.z, v.y, shift),
                  __builtin_amdgcn_alignbit(v.w, v.z, shift), __builtin_amdgcn_alignbit(n, v.w, shift)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = G - 4 * s - 2 * i;
      d[i] = v[i] & (left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u);
    }
  }
};

// The pairs b0 .. b0 + BT - 1 that chose expert e, in order, into the wave's
// list; returns how many there are in all.
template <int BT>
__device__ __forceinline__ int list_pairs(const int* __restrict__ ids, int P, int e, int b0, int lane, int* list) {
  int m = 0;
  for (int p0 = 0; p0 < P; p0 += 512) {
    int v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = ids[min(p0 + 64 * j + lane, P - 1)];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = p0 + 64 * j + lane < P ? v[j] : -1;
      const uint64_t bm = __builtin_amdgcn_ballot_w64(v[j] == e);
      const int r = m + __builtin_popcountll(bm & ((1ull << lane) - 1)) - b0;
      if (v[j] == e && r >= 0 && r < BT) list[r] = p0 + 64 * j + lane;
      m += __builtin_popcountll(bm);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return m;
}

// The expert of this workgroup (its blockIdx.y), or -1: nothing to do.  Up to
// kPairGrid pairs, and fewer pairs than experts, the grid has a row of
// workgroups per pair (that of an expert's first pair works), else one per
// expert.
__device__ __forceinline__ int block_expert(const int* __restrict__ ids, int P, int E, int lane) {
  if (P > kPairGrid || P >= E) return blockIdx.y;
  const int id = lane < P ? ids[lane] : -1;
  const int e = __builtin_amdgcn_readlane(id, blockIdx.y);
  if ((uint32_t)e >= (uint32_t)E) return -1;
  const uint64_t mask = __builtin_amdgcn_ballot_w64(id == e);
  return (mask & ((1ull << blockIdx.y) - 1)) != 0 ? -1 : e;
}

// h = silu(g) u of pair p and row n in two bf16 parts
__device__ __forceinline__ void store_gated(float g, float u, uint16_t* h, int p, int rows, int n) {
  uint32_t hi, lo;
  split_bf16(g / (1.0f + expf(-g)) * u, hi, lo);
  uint16_t* o = h + (size_t)p * 2 * rows + (n & ~7) + paired_place(n & 7);
  o[0] = (uint16_t)hi;
  o[rows] = (uint16_t)lo;
}

// The activations of a pass: offset of the row that this lane loads from
// (kNowhere: none), for GP = 1 of tile 0 row lane / 4, else row li % MT
template <int GP>
__device__ __forceinline__ uint32_t act_offset(uint32_t row, int K, int lane) {
  const int li = lane & 15, lq = lane >> 4;
  return row * (uint32_t)K * 2u + (GP == 1 ? 32u * (lane & 3) : 32u * lq + 128u * (li / (16 / GP)));
}

// acc[r][i] = the sums over stages sb .. se - 1 of activation row 4 lq + i
// (GP > 1: of group (4 lq + i) / MT of row (4 lq + i) % MT) and weight row li
// of row tile r.  rc: the row tiles' codes, slot0 and slot1: the wave's ring.
template <int GP, int R, bool DOWN, int HINT>
__device__ __forceinline__ void stream_sums(const rsrc_t (&rc)[R], const RowScales<R, DOWN>& rs, rsrc_t rx,
                                            uint32_t x_off, uint8_t* slot0, uint8_t* slot1, int K, int sb,
                                            int se, int lane, f32x4_t (&acc)[R]) {
  constexpr int MT = 16 / GP;            // activation rows of a tile
  constexpr int LOADS = 2 * R + 8 / GP;  // of one stage, the scales not counted
  const int li = lane & 15, lq = lane >> 4, G = K >> 6;
  const uint32_t crow = (uint32_t)K >> 1;
  const uint32_t c_off = code_offset(crow, lane);
  int rd[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) rd[g] = code_read(li, lq, g);
  const int xsrc4 = (4 * li + lq) * 4;  // the lane holding this lane's activations after an exchange (byte address)
#pragma unroll
  for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // (a stage past the wave's share and groups past K: offsets past every
  // range, which read as zeros)
  auto load = [&](Acts<GP>& L, uint8_t* ring, int s) __device__ {
    const uint32_t away = s < se ? 0u : kNowhere;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        dma16<HINT>(rc[r], (c_off + 8u * h * crow + 128u * (uint32_t)s) | away, 0,
              ring + (2 * r + h) * (kTileStage / 2));
    in_order();
#pragma unroll
    for (int g = 0; g < 4 / GP; ++g) {
      const uint32_t away_g = s < se && 4 * s + GP * g + (GP == 1 ? 0 : li / MT) < G ? 0u : kNowhere;
      const uint32_t o = (x_off + 512u * (uint32_t)s) | away_g;
      L.v[2 * g] = __builtin_amdgcn_raw_buffer_load_b128(rx, o + 128 * GP * g, 0, 0);
      L.v[2 * g + 1] = __builtin_amdgcn_raw_buffer_load_b128(rx, o + 128 * GP * g + 16, 0, 0);
    }
    in_order();
  };
  auto compute = [&](const Acts<GP>& L, const uint8_t* ring, uint32_t d0, uint32_t d1, int s) __device__ {
    const u32x4_t eights = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
    uint32_t sc[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sc[r][0] = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * r + li) * 4, (int)d0);
      sc[r][1] = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * r + li) * 4, (int)d1);
    }
    auto codes = [&](int r, int g, u32x4_t (&w)[2]) __device__ {
      const u32x2_t cw = *reinterpret_cast<const u32x2_t*>(ring + rd[g] + r * kTileStage);
      w[0] = q4_paired(cw.x);
      w[1] = q4_paired(cw.y);
    };
    if constexpr (GP == 1) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (g > 0 && 4 * s + g >= G) break;
        u32x4_t x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[h] = lane_piece(L.v[2 * g + h], xsrc4);
          if constexpr (!DOWN) x[h] = to_paired(x[h]);
        }
        f32x4_t cr = mfma(x[0], eights, zero);
        cr = mfma(x[1], eights, cr);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          u32x4_t w[2];
          codes(r, g, w);
          const uint32_t sb16 = (g & 1) ? sc[r][g >> 1] >> 16 : sc[r][g >> 1] & 0xFFFFu;
          const float sv = f16_bits_to_f32((uint16_t)sb16);
          f32x4_t p = mfma(x[0], w[0], zero);
          p = mfma(x[1], w[1], p);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] = __builtin_fmaf(sv, p[i] - cr[i], acc[r][i]);
        }
      }
    } else {
#pragma unroll
      for (int g = 0; g < 4 / GP; ++g) {
        u32x4_t x[GP][2];
        f32x4_t cr = zero;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t v = DOWN ? L.v[2 * g + h] : to_paired(L.v[2 * g + h]);
#pragma unroll
          for (int j = 0; j < GP; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][h][i] = li / MT == j ? v[i] : 0u;
        }
#pragma unroll
        for (int j = 0; j < GP; ++j) {
          cr = mfma(x[j][0], eights, cr);
          cr = mfma(x[j][1], eights, cr);
        }
        const int own = GP * g + 4 * lq / MT;  // the group of this lane's accumulator rows
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const uint32_t sd = GP == 4 ? (lq >> 1 ? sc[r][1] : sc[r][0]) : sc[r][g];
          const float sv = f16_bits_to_f32((uint16_t)((own & 1) ? sd >> 16 : sd));
          f32x4_t p = zero;
#pragma unroll
          for (int j = 0; j < GP; ++j) {
            u32x4_t w[2];
            codes(r, GP * g + j, w);
            p = mfma(x[j][0], w[0], p);
            p = mfma(x[j][1], w[1], p);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] = __builtin_fmaf(sv, p[i] - cr[i], acc[r][i]);
        }
      }
    }
  };
  Acts<GP> L[2];
  typename RowScales<R, DOWN>::Regs S;
  rs.load(S, sb, se);
  load(L[0], slot0, sb);
  load(L[1], slot1, sb + 1);
  // the stage's copies have landed when only the next stage's loads are
  // outstanding; a slot's reads are done before it is written again
  for (int s = sb; s < se; s += 2) {
    wait_vm<LOADS>();
    in_order();
    uint32_t d[4];
    rs.rows(S, s, d);
    compute(L[0], slot0, d[0], d[1], s);
    wait_lgkm0();
    in_order();
    rs.load(S, s + 2, se);
    load(L[0], slot0, s + 2);
    wait_vm<LOADS>();
    in_order();
    if (s + 1 < se) compute(L[1], slot1, d[2], d[3], s + 1);
    wait_lgkm0();
    in_order();
    load(L[1], slot1, s + 3);
  }
  wait_vm<0>();  // (nothing lands in the ring any more)
  in_order();
}

// A few tokens' choice, made where it is used: the logits [T][E], and where
// the choice goes
constexpr int kFewTokens = 8;         // at most,
constexpr int kFewExperts = 256;      // of so many experts,
struct Choice {
  const double* lg;
  int* ids;
  float* weights;
  int T, renorm;
};

// The expert e of this workgroup (rows of workgroups as for block_expert: the
// choice of pair blockIdx.y, or blockIdx.y itself) and the pairs that chose
// it, in order, into the wave's list; returns how many, 0 if there are none
// or an earlier token chose it (whose workgroups serve it).  E <= 64 B.
template <int FT, int B>
__device__ __forceinline__ int choose_pairs(const Choice& c, int E, int top_k, int lane, int* list, int& e) {
  uint64_t key[FT][B];  // (every token's loads in flight; tokens past T repeat the last)
#pragma unroll
  for (int t = 0; t < FT; ++t)
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int i = 64 * b + lane;
      const uint64_t k = route_key(c.lg[(size_t)min(t, c.T - 1) * E + min(i, E - 1)], i);
      key[t][b] = i < E ? k : 0;
    }
  const bool by_expert = c.T * top_k >= E;
  const int mine = by_expert ? 0 : blockIdx.y / top_k;
  if (by_expert) {
    e = blockIdx.y;
  } else {
    uint64_t own[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      own[b] = key[0][b];
#pragma unroll
      for (int t = 1; t < FT; ++t) own[b] = t == mine ? key[t][b] : own[b];
    }
    e = choose_rank<B>(own, blockIdx.y - mine * top_k + 1, lane, nullptr);
  }
  int m = 0;
  bool served = false;
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    uint64_t mk = key[t][0];
#pragma unroll
    for (int b = 1; b < B; ++b) mk = e >> 6 == b ? key[t][b] : mk;
    const uint64_t ke = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mk, e & 63) |
                        ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(mk >> 32), e & 63) << 32);
    int rank = 0;
#pragma unroll
    for (int b = 0; b < B; ++b) rank += __builtin_popcountll(__builtin_amdgcn_ballot_w64(key[t][b] > ke));
    if (t < c.T && rank < top_k) {
      served |= t < mine;
      if (lane == 0) list[m] = t * top_k + rank;
      ++m;
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return served ? 0 : m;
}

// The gate and up products of experts with few rows each, and the gate: h in
// two parts, [pair][part][rows] in the paired order.  K: of the products,
// rows: of h, wk: waves that share K (the other kWaves / wk share the
// workgroup's rows).  CHOOSE: tokens whose choice is made here, at most (0:
// ids hold it).
template <int R, int CHOOSE, int HINT, int B>
__global__ void __launch_bounds__(kThreads, 2)
moe_gated_kernel(const uint16_t* x, const uint8_t* codes0, const uint16_t* scales0, const uint8_t* codes1,
                 const uint16_t* scales1, const int* __restrict__ ids, uint16_t* h, int K, int rows, int E, int P,
                 int top_k, uint32_t x_bytes, int wk, Choice choice) {
  constexpr int BT = 16;                // pairs per pass, at most
  constexpr int RT = R / 2;             // row tiles of h per wave
  constexpr int SLOT = R * kTileStage;  // bytes of one stage's codes
  typedef float Red[R][16][20];
  static_assert(sizeof(Red) <= (size_t)SLOT, "the waves' sums reuse a ring slot");
  // the rings' two slots (two objects, so that a read of one is known not to
  // depend on a copy in flight into the other)
  __shared__ __attribute__((aligned(16))) uint8_t ring0[kWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[kWaves * SLOT];
  __shared__ int list[kWaves][BT];
  __shared__ int chosen[CHOOSE ? kWaves : 1][CHOOSE ? kPairGrid : 1];
  static_assert(CHOOSE <= BT, "one pass");
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wr = kWaves / wk, kp = wave % wk, rp = wave / wk;

  int e, m = 1;
  if constexpr (CHOOSE > 0) {
    if (blockIdx.y == gridDim.y - 1) {  // (a workgroup of its own writes the choice)
      if (blockIdx.x > 0) return;
      for (int t = wave; t < choice.T; t += kWaves)
        choose_one<B>(choice.lg + (size_t)t * E, E, top_k, lane, choice.renorm, chosen[wave],
                                     choice.ids + (size_t)t * top_k, choice.weights + (size_t)t * top_k);
      return;
    }
    m = choose_pairs<CHOOSE, B>(choice, E, top_k, lane, list[wave], e);
    if (m == 0) return;
  } else {
    e = block_expert(ids, P, E, lane);
    if (e < 0) return;
  }

  const int n0 = (blockIdx.x * wr + rp) * (16 * RT);  // this wave's first output row
  const int G = K >> 6, stages = (G + 3) >> 2;
  const int sb = stages * kp / wk, se = stages * (kp + 1) / wk;
  const uint32_t crow = (uint32_t)K >> 1;
  rsrc_t rc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t0 = n0 + 16 * (r % RT);
    // (rows are multiples of 16: a tile is whole or absent)
    rc[r] = make_rsrc((r < RT ? codes0 : codes1) + ((size_t)e * rows + t0) * crow, t0 < rows ? 16u * crow : 0u);
  }
  const rsrc_t rx = make_rsrc(x, x_bytes);
  RowScales<R, false> rs(scales0, scales1, ((size_t)e * rows + n0) * G, min(16 * RT, rows - n0), G, lane);

  // One pass over the wave's share of K for the mr activation rows of the
  // list, then the workgroup's sums
  auto pass = [&](auto gpc, int mr) __device__ {
    constexpr int GP = decltype(gpc)::value, MT = 16 / GP;
    const int a = GP == 1 ? lane >> 2 : li % MT;
    // (rows past the last read as zeros)
    const uint32_t x_off = a < mr ? act_offset<GP>((uint32_t)(list[wave][min(a, mr - 1)] / top_k), K, lane) : kNowhere;
    f32x4_t acc[R];
    stream_sums<GP, R, false, HINT>(rc, rs, rx, x_off, ring0 + wave * SLOT, ring1 + wave * SLOT, K, sb, se, lane, acc);

    // the sums of the waves that share K and of a tile's groups
    Red& red = *reinterpret_cast<Red*>(ring0 + wave * SLOT);
    if (4 * lq % MT < mr)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[r][4 * lq + i][li] = acc[r][i];
    __syncthreads();
    const int tiles = wr * RT;
    for (int o = tid; o < 16 * tiles * mr; o += kThreads) {
      const int c = o & 15, tile = (o >> 4) % tiles, t = (o >> 4) / tiles;
      const int w0 = tile / RT * wk, r = tile % RT, n = (blockIdx.x * tiles + tile) * 16 + c;
      if (n >= rows) continue;
      auto sum = [&](int rr) __device__ {
        double v = 0.0;
        for (int w = 0; w < wk; ++w)
#pragma unroll
          for (int j = 0; j < GP; ++j)
            v += (double)(*reinterpret_cast<const Red*>(ring0 + (w0 + w) * SLOT))[rr][MT * j + t][c];
        return v;
      };
      store_gated((float)sum(r), (float)sum(RT + r), h, list[wave][t], rows, n);
    }
  };

  for (int b0 = 0; b0 < m; b0 += BT) {
    if constexpr (CHOOSE == 0) {
      m = list_pairs<BT>(ids, P, e, b0, lane, list[wave]);
      if (m == 0) return;
    }
    const int mr = min(BT, m - b0);
    // the smallest tiles that hold the rows
    if (mr <= 4) pass(Slot<4>{}, mr);
    else if (mr <= 8) pass(Slot<2>{}, mr);
    else pass(Slot<1>{}, mr);
    __syncthreads();
  }
}

// The down products of a few pairs and their weighted sums in one launch: a
// workgroup of 16 waves takes 16 R rows of y; its waves share the pairs and,
// where there are fewer than waves, each pair's K.  (An expert that several
// tokens chose is read again for each, by the same workgroup.)
constexpr int kFewWaves = 16;
template <int R>
__global__ void __launch_bounds__(64 * kFewWaves)
moe_down_few_kernel(const uint16_t* h, const uint8_t* codes, const uint16_t* scales, const int* __restrict__ ids,
                    const float* __restrict__ weights, uint16_t* y, int K, int rows, int E, int T, int top_k,
                    uint32_t h_bytes) {
  constexpr int SLOT = R * kTileStage;
  __shared__ __attribute__((aligned(16))) uint8_t ring0[kFewWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[kFewWaves * SLOT];
  __shared__ float sums[kFewWaves][kFewTokens][16 * R];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int n0 = blockIdx.x * (16 * R), P = T * top_k;
  const int G = K >> 6, stages = (G + 3) >> 2;
  const int wpp = P < kFewWaves ? kFewWaves / P : 1;  // waves per pair
  const uint32_t crow = (uint32_t)K >> 1;
  const rsrc_t rx = make_rsrc(h, h_bytes);
  for (int i = lane; i < kFewTokens * 16 * R; i += 64) (&sums[wave][0][0])[i] = 0.f;
  const int part = wave % wpp, sb = stages * part / wpp, se = stages * (part + 1) / wpp;
  for (int p = wave / wpp; p < P; p += kFewWaves / wpp) {
    const int e = __builtin_amdgcn_readfirstlane(ids[p]);
    if ((uint32_t)e >= (uint32_t)E || sb >= se) continue;
    const float wp = weights[p];
    rsrc_t rc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int t0 = n0 + 16 * r;
      rc[r] = make_rsrc(codes + ((size_t)e * rows + t0) * crow, t0 < rows ? 16u * crow : 0u);
    }
    const RowScales<R, true> rs(scales, scales, ((size_t)e * rows + n0) * G, min(16 * R, rows - n0), G, lane);
    const int a = li % 4;  // the pair's two parts
    const uint32_t x_off = a < 2 ? act_offset<4>(2u * p + a, K, lane) : kNowhere;
    f32x4_t acc[R];
    stream_sums<4, R, true, 0>(rc, rs, rx, x_off, ring0 + wave * SLOT, ring1 + wave * SLOT, K, sb, se, lane, acc);
    // this lane: row li, group lq of every stage
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float v = acc[r][0] + acc[r][1];
      v += __shfl_xor(v, 16);
      v += __shfl_xor(v, 32);
      if (lq == 0) sums[wave][p / top_k][16 * r + li] = __builtin_fmaf(wp, v, sums[wave][p / top_k][16 * r + li]);
    }
  }
  __syncthreads();
  for (int i = tid; i < T * 16 * R; i += 64 * kFewWaves) {
    const int t = i / (16 * R), r = i % (16 * R);
    if (n0 + r >= rows) continue;
    double v = 0.0;
    for (int w = 0; w < kFewWaves; ++w) v += (double)sums[w][t][r];
    y[(size_t)t * rows + n0 + r] = f32_to_bf16_rne((float)v);
  }
}

// ---------------------------------------------------------------------------
// The same for workgroups whose eight waves take different rows of the weight
// over the same K and share the activations of up to BT pairs a pass, in
// stages of 128 k.  Codes go through a ring of each wave (two slots),
// activations through one of the workgroup (three slots, a barrier per
// stage); both are asked for two stages before their use.  The two parts of h
// are two rows of a tile for up to eight pairs (PARTS = 1: three products a
// tile of codes), two products into the same sums for more (PARTS = 2: every
// sum and conversion serves both, half the scaling of twice the rows).
// Registers and LDS for four waves per SIMD, as far as the conversion of the
// codes and the scaling of the sums, not the weight stream, bound it: from
// about 16 rows.
// (96 tokens on eight experts of 14336 x 5120: vector and matrix instructions
// take 60 + 31 % of the SIMDs' cycles in the gate and up products, 55 + 56 %
// in the down products; both halves of a 128-byte line asked for together,
// with or without a place in the caches, move 5 to 20 % fewer bytes and take
// as long or longer.)
// blockIdx.z shares K (down: parts of the sums, added by the combine) or the
// passes (gate and up).
// ---------------------------------------------------------------------------
constexpr int kWideWaves = 8;
constexpr int kWideQuad = 4;  // stages of a share come in quads, as the scales do
template <int R, bool DOWN, int BT>
__global__ void __launch_bounds__(64 * kWideWaves, 4)
moe_wide_kernel(const uint16_t* act, const uint8_t* codes0, const uint16_t* scales0, const uint8_t* codes1,
                const uint16_t* scales1, const int* __restrict__ ids, void* out, int K, int rows, int E, int P,
                int top_k, uint32_t act_bytes) {
  constexpr int RP = DOWN ? 2 : 1;      // activation rows per pair
  constexpr int RT = DOWN ? R : R / 2;  // row tiles of the output per wave
  constexpr int XROW = 256;             // bytes of an activation row in a stage (128 k here)
  constexpr int TILE = 16 * 64;         // code bytes of a row tile in a stage
  constexpr int SLOT = R * TILE;
  __shared__ __attribute__((aligned(16))) uint8_t ring0[kWideWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[kWideWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t xs0[BT * RP * XROW];
  __shared__ __attribute__((aligned(16))) uint8_t xs1[BT * RP * XROW];
  __shared__ __attribute__((aligned(16))) uint8_t xs2[BT * RP * XROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int e = block_expert(ids, P, E, lane);
  if (e < 0) return;
  const int n0 = (blockIdx.x * kWideWaves + wave) * (16 * RT);  // this wave's first output row
  const int G = K >> 6, stages = (G + 1) >> 1;
  const int quads = (stages + kWideQuad - 1) / kWideQuad;
  const int part = DOWN ? blockIdx.z : 0, parts = DOWN ? gridDim.z : 1;
  const int sb = kWideQuad * (quads * part / parts), se = min(kWideQuad * (quads * (part + 1) / parts), stages);
  const uint32_t crow = (uint32_t)K >> 1;
  rsrc_t rc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t0 = n0 + 16 * (r % RT);
    rc[r] = make_rsrc((r < RT ? codes0 : codes1) + ((size_t)e * rows + t0) * crow, t0 < rows ? 16u * crow : 0u);
  }
  const rsrc_t rx = make_rsrc(act, act_bytes);
  // four lanes copy 64 bytes of a row; piece p of row i lies at position 4 i + (p ^ (i / 2 & 3))
  const uint32_t c_off = (uint32_t)(lane >> 2) * crow + 16u * ((lane & 3) ^ ((lane >> 3) & 3));
  const RowScales<R, DOWN> rs(scales0, scales1, ((size_t)e * rows + n0) * G, min(16 * RT, rows - n0), G, lane);
  // operand reads: codes as in stream_sums; activations of group g: pieces
  // 8 g + 2 lq + h of row li
  int rd[2], xd[4];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    rd[g] = wave * SLOT + li * 64 + 16 * ((2 * g + (lq >> 1)) ^ ((li >> 1) & 3)) + 8 * (lq & 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) xd[2 * g + h] = li * XROW + 16 * ((8 * g + 2 * lq + h) ^ li);
  }

  int m = INT32_MAX;
  for (int b0 = DOWN ? 0 : BT * blockIdx.z; b0 < m; b0 += DOWN ? BT : BT * gridDim.z) {
    // (the list goes by way of the wave's own slot into a register: lane i holds pair i)
    int* const list = reinterpret_cast<int*>(ring0 + wave * SLOT);
    m = list_pairs<BT>(ids, P, e, b0, lane, list);
    if (m <= b0) return;
    const int mine = list[lane & (BT - 1)];
    wait_lgkm0();
    in_order();
    const int c = min(BT, m - b0);  // pairs of this pass
    auto pass = [&](auto ntc, auto partsc) __device__ {
      constexpr int NT = decltype(ntc)::value, PARTS = decltype(partsc)::value;
      constexpr int AR = RP / PARTS;  // activation rows of a tile per pair
      const int mr = c * AR;
      // code order of the products (x is permuted into the paired one for a single tile)
      constexpr bool PAIRED = DOWN || NT == 1;
      constexpr int DMAS = NT * PARTS == 4 ? 2 : 1;  // a wave's copies of activations per stage
      constexpr int LOADS = R + DMAS;  // of a stage, the scales not counted
      // activation rows: a wave copies four rows, lane l the piece of
      // 16 bytes that lies at position l % 16 of row l / 16; piece p of row a
      // at position p ^ (a % 16), so that sixteen rows' reads of one piece
      // spread over the banks
      // (two parts of 16 rows: waves 0 to 3 the one, 4 to 7 the other; of 32 rows: every wave both)
      const int xrow = 4 * wave + (lane >> 4);
      uint32_t x_off;
      {
        constexpr bool HALVES = NT == 1 && PARTS == 2;
        const int a = HALVES ? xrow & 15 : xrow;
        const int p = __shfl(mine, min(a, mr - 1) / AR);
        const uint32_t row = DOWN ? 2u * p + (AR == 2 ? a & 1 : HALVES ? xrow >> 4 : 0) : (uint32_t)(p / top_k);
        x_off = a < mr ? row * (uint32_t)K * 2u + 16u * ((lane & 15) ^ (xrow & 15)) : kNowhere;
      }
      f32x4_t acc[NT][R];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[nt][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

      auto load_x = [&](uint8_t* xs, int s) __device__ {
        // (groups past K and rows past the last land as zeros)
        const bool in = ((lane & 15) ^ (xrow & 15)) < (s < se ? 8 * (G - 2 * s) : 0);
#pragma unroll
        for (int q = 0; q < DMAS; ++q)
          dma16(rx, in ? x_off + 256u * (uint32_t)s : kNowhere, q * 2u * (uint32_t)K, xs + (32 * q + 4 * wave) * XROW);
        in_order();
      };
      auto load_c = [&](uint8_t* ring, int s) __device__ {
        const uint32_t o = (c_off + 64u * (uint32_t)s) | (s < se ? 0u : kNowhere);
#pragma unroll
        for (int r = 0; r < R; ++r) dma16(rc[r], o, 0, ring + wave * SLOT + r * TILE);
        in_order();
      };
      auto compute = [&](const uint8_t* ring, const uint8_t* xs, uint32_t d0) __device__ {
        const u32x4_t eights = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        uint32_t sc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) sc[r] = (uint32_t)__builtin_amdgcn_ds_bpermute((16 * r + li) * 4, (int)d0);
        // Half by half (h of part q of group g): both parts of a pair add
        // up in the same sums, and a tile's converted codes serve both;
        // the LDS reads of a half are issued a half ahead
        u32x4_t x[2][NT], w[R][2];
        u32x2_t cw[R];
        f32x4_t cr[NT], p[R][NT];
        auto fetch = [&](auto uc) __device__ {
          constexpr int u = decltype(uc)::value, g = u / (2 * PARTS), q = u / 2 % PARTS, h = u & 1;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            x[u & 1][nt] = *reinterpret_cast<const u32x4_t*>(xs + xd[2 * g + h] + 16 * (NT * q + nt) * XROW);
          if constexpr (q + h == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) cw[r] = *reinterpret_cast<const u32x2_t*>(ring + rd[g] + r * TILE);
        };
        fetch(Slot<0>{});
        static_for<4 * PARTS>([&](auto uc) __device__ {
          constexpr int u = decltype(uc)::value, g = u / (2 * PARTS), q = u / 2 % PARTS, h = u & 1;
          if constexpr (q + h == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              w[r][0] = PAIRED ? q4_paired(cw[r].x) : q4_natural(cw[r].x);
              w[r][1] = PAIRED ? q4_paired(cw[r].y) : q4_natural(cw[r].y);
            }
          if constexpr (u + 1 < 4 * PARTS) fetch(Slot<u + 1>{});
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (PAIRED && !DOWN) x[u & 1][nt] = to_paired(x[u & 1][nt]);
            cr[nt] = mfma(x[u & 1][nt], eights, q + h ? cr[nt] : zero);
#pragma unroll
            for (int r = 0; r < R; ++r) p[r][nt] = mfma(x[u & 1][nt], w[r][h], q + h ? p[r][nt] : zero);
          }
          if constexpr (q == PARTS - 1 && h == 1)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float sv = f16_bits_to_f32((uint16_t)(g ? sc[r] >> 16 : sc[r] & 0xFFFFu));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][r][i] = __builtin_fmaf(sv, p[r][nt][i] - cr[nt][i], acc[nt][r][i]);
            }
        });
      };
      typename RowScales<R, DOWN>::Regs S;
      uint32_t d[4];
      rs.load(S, sb >> 1, (se + 1) >> 1);
      load_x(xs0, sb);
      load_c(ring0, sb);
      load_x(xs1, sb + 1);
      load_c(ring1, sb + 1);
      // Per stage: it has landed when only loads issued after its codes are
      // outstanding; behind the barrier every wave's part of its activations
      // has, and every wave has left the slot of the stage before, which
      // takes the activations of the stage after the next
      for (int s0 = sb; s0 < se; s0 += 12) {
        static_for<12>([&](auto ic) __device__ {
          constexpr int i = decltype(ic)::value;
          const int s = s0 + i;
          if (s < se) {  // (the same for all waves)
            wait_vm<LOADS + (i % 4 == 1 ? RowScales<R, DOWN>::LOADS : 0)>();
            in_order();
            __builtin_amdgcn_s_barrier();
            in_order();
            if constexpr (i % 4 == 0) {
              rs.rows(S, s >> 1, d);
              rs.load(S, (s >> 1) + 2, (se + 1) >> 1);
            }
            load_x((i + 2) % 3 == 0 ? xs0 : (i + 2) % 3 == 1 ? xs1 : xs2, s + 2);
            compute((i & 1) ? ring1 : ring0, i % 3 == 0 ? xs0 : i % 3 == 1 ? xs1 : xs2, d[i % 4]);
            in_order();
            wait_lgkm0();
            in_order();
            load_c((i & 1) ? ring1 : ring0, s + 2);
          }
        });
      }
      wait_vm<0>();  // (nothing lands in the slots any more)
      in_order();

#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; i += AR) {
          const int a = 16 * nt + 4 * lq + i;
          const int p = __shfl(mine, a / AR);
          if (a >= mr) continue;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int n = n0 + 16 * r + li;
            if (n >= rows) continue;
            if constexpr (DOWN) {
              static_cast<float*>(out)[((size_t)blockIdx.z * P + p) * rows + n] =
                  AR == 2 ? acc[nt][r][i] + acc[nt][r][(i + 1) & 3] : acc[nt][r][i];
            } else {
              store_gated(acc[nt][r][i], acc[nt][RT + r][i], static_cast<uint16_t*>(out), p, rows, n);
            }
          }
        }
    };
    if constexpr (!DOWN) {
      if (c <= 16) pass(Slot<1>{}, Slot<1>{});
      else pass(Slot<2>{}, Slot<1>{});
    } else if constexpr (BT == 16) {
      if (c <= 8) pass(Slot<1>{}, Slot<1>{});
      else pass(Slot<1>{}, Slot<2>{});
    } else {
      if (c <= 16) pass(Slot<1>{}, Slot<2>{});
      else pass(Slot<2>{}, Slot<2>{});
    }
    __syncthreads();
  }
}

// y[t][n .. n + 3] = bf16( sum_j weights[t][j] sum_k parts[k][t top_k + j][n .. n + 3] ), in order
template <int J>
__global__ void __launch_bounds__(256)
moe_combine_kernel(const float* __restrict__ parts, const int* __restrict__ ids, const float* __restrict__ weights,
                   uint16_t* __restrict__ y, int rows, int E, int top_k, int T, int ks, int vec) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = rows >> 2;
  if (i >= (int64_t)T * per) return;
  const int t = (int)(i / per), n = 4 * (int)(i - (int64_t)t * per);
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < top_k; j0 += J) {
    // (the loads of J pairs in flight; pairs past the last repeat it)
    int e[J];
    float w[J];
    f32x4_t d[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int p = t * top_k + min(j0 + j, top_k - 1);
      e[j] = ids[p];
      w[j] = weights[p];
      d[j] = *reinterpret_cast<const f32x4_t*>(parts + (size_t)p * rows + n);
    }
    for (int k0 = 1; k0 < ks; k0 += 3) {
      // (three parts' loads in flight; parts past the last repeat it: seven parts
      // of six pairs on 640 outputs 5 us, one after the other 12.5)
      f32x4_t more[3][J];
#pragma unroll
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int j = 0; j < J; ++j)
          more[k][j] = *reinterpret_cast<const f32x4_t*>(
              parts + ((size_t)min(k0 + k, ks - 1) * T * top_k + t * top_k + min(j0 + j, top_k - 1)) * rows + n);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (k0 + k < ks)
#pragma unroll
          for (int j = 0; j < J; ++j) d[j] += more[k][j];
    }
    // (what lies at a pair without an expert is not used)
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (j0 + j < top_k && (uint32_t)e[j] < (uint32_t)E)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w[j], d[j][r], v[r]);
  }
  uint16_t* o = y + (size_t)t * rows + n;
  uint32_t h[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) h[r] = f32_to_bf16_rne(v[r]);
  if (vec) {
    *reinterpret_cast<u32x2_t*>(o) = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (uint16_t)h[r];
  }
}

size_t al256(size_t v) { return (v + 255) & ~(size_t)255; }

constexpr int kRowTiles = 4;      // per wave (gate and up of few rows)
constexpr int kWideRowTiles = 2;  // per wave (workgroups that share the activations)
// Pairs per expert in use from which the gate and up products share the
// activations in workgroups (24 of them on eight experts of 2 x 14336 x 5120:
// 192 us against 222; 4 on 128 of 2 x 768 x 2048 58 either way; 4 on 16 of
// 2 x 1536 x 5120 45 against 41), and the down products take 32 pairs a pass
// (24 on eight of 5120 x 14336: 115 us against 165 with passes of 16; up to
// 16 on 16 of 5120 x 1536 26.3 against 24.1).
constexpr int64_t kManyPairs = 18;
// workgroups that the chip holds at a time (two per CU, by LDS and registers)
constexpr int64_t kResident = 512;

// Into how many shares (of those below) to split `stages` stages of K, handed
// out in runs of `unit`, when `groups` workgroups take a whole K each: the
// rounds of resident workgroups times the longest share's stages and the
// `extra` that a workgroup's start and end cost; in runs, among equals of as
// many rounds the most shares, whose lengths are more even on the whole.  No
// share is empty (12 tokens on all of seven experts, inner 960: 28.7 us with
// two shares, 35.4 with two and six empty ones).
int k_split(int64_t groups, int64_t stages, int64_t unit, int64_t extra, int64_t most, bool powers) {
  const int64_t units = (stages + unit - 1) / unit;
  int best = 1;
  int64_t cost = INT64_MAX, fewest = 0;
  for (int64_t s = 1; s <= most && s <= units; s = powers ? 2 * s : s + 1) {
    const int64_t rounds = (groups * s + kResident - 1) / kResident;
    const int64_t longest = (units + s - 1) / s * unit;
    const int64_t c = rounds * ((longest < stages ? longest : stages) + extra);
    if (c < cost || (unit > 1 && c == cost && rounds == fewest)) {
      cost = c;
      fewest = rounds;
      best = (int)s;
    }
  }
  return best;
}
// experts in use, at most (the routing is not known here)
int64_t experts_hit(const MoeArgs& a) {
  const int64_t pairs = a.t * a.top_k;
  return pairs < a.experts ? pairs : a.experts;
}
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// rows of workgroups: pairs or experts, the fewer (block_expert; three tokens
// on six of seven experts each: gate and up 12 us with seven rows, 22 with 18)
unsigned grid_rows(const MoeArgs& a) {
  const int64_t pairs = a.t * a.top_k;
  return (unsigned)(pairs <= kPairGrid && pairs < a.experts ? pairs : a.experts);
}

// Whether one launch makes the down products and their sums: a single token,
// or a few that share few experts (16 waves for every 16 or 32 rows of y; two
// launches fewer, but an expert is read again for every token that chose it),
// while a workgroup's rows of all pairs are short.  The layer in us, in one
// launch / in three: one token, 9 pairs of inner 3904 on 1088 rows 38 / 42, 16
// of 2816 on 2048 44 / 48, 8 of 7168 on 2048 50 / 51, 16 of 4096 on 2048 56 /
// 55, 20 of 5120 on 640 70 / 61; two tokens, 16 pairs of 1792 on 2048 32 / 34;
// four, 16 of 1856 on 2048 33 / 33, 24 of 1408 40 / 40; three, 9 of 3904 on
// 1088 38.3 / 36.6; eight, 16 of 2048 on 1024 27 / 25.
constexpr int64_t kFewColumnsOne = 56 * 1024, kFewColumns = 30 * 1024;
bool few_pairs(const MoeArgs& a) {
  const int64_t pairs = a.t * a.top_k;
  if (a.t == 1) return pairs * a.inner <= kFewColumnsOne;
  return a.t <= kFewTokens && pairs <= kPairGrid && 2 * pairs <= a.experts && pairs * a.inner <= kFewColumns;
}
// parts of the down products' sums (moe_wide_kernel hands out whole quads of
// stages)
int down_parts(const MoeArgs& a) {
  return k_split(ceil_div(a.k, kWideWaves * 16 * kWideRowTiles) * experts_hit(a), ceil_div(a.inner, 128), kWideQuad, 4,
                 8, false);
}

hipError_t launch_gated(const MoeArgs& a, void* h, const double* lg, hipStream_t s) {
  // (lg: the choice is made here)
  const int P = (int)(a.t * a.top_k);
  const unsigned slots = grid_rows(a);
  auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  const uint32_t x_bytes = (uint32_t)(a.t * a.k * 2);
  if (lg == nullptr && P / experts_hit(a) >= kManyPairs) {
    constexpr int R = kWideRowTiles;
    // workgroups per pass where all of them are resident (60 tokens on each of
    // four experts of 2 x 1600 x 1280: 16 us against 28)
    const int64_t blocks = ceil_div(a.inner, kWideWaves * 8 * R), passes = ceil_div(P / experts_hit(a), 32);
    const int64_t room = kResident / (blocks * experts_hit(a));
    const dim3 grid((unsigned)blocks, slots, (unsigned)(room < 1 ? 1 : room < passes ? room : passes));
    moe_wide_kernel<R, false, 32><<<grid, dim3(64 * kWideWaves), 0, s>>>(
        u16(a.x), u8(a.codes_gate), u16(a.scales_gate), u8(a.codes_up), u16(a.scales_up),
        static_cast<const int*>(a.ids), h, (int)a.k, (int)a.inner, (int)a.experts, P, (int)a.top_k, x_bytes);
    return hipGetLastError();
  }
  constexpr int R = kRowTiles;
  const int wk = k_split(ceil_div(a.inner, kWaves * 8 * R) * experts_hit(a), ceil_div(a.k, 256), 1, 2, kWaves, true);
  const unsigned blocks = (unsigned)ceil_div(a.inner, kWaves / wk * 8 * R);
  auto go = [&](auto kern, unsigned rows) {
    kern<<<dim3(blocks, rows), dim3(kThreads), 0, s>>>(
        u16(a.x), u8(a.codes_gate), u16(a.scales_gate), u8(a.codes_up), u16(a.scales_up),
        static_cast<const int*>(a.ids), static_cast<uint16_t*>(h), (int)a.k, (int)a.inner, (int)a.experts, P,
        (int)a.top_k, x_bytes, wk,
        Choice{lg, static_cast<int*>(a.ids), static_cast<float*>(a.weights), (int)a.t, a.renorm});
  };
  auto pick = [&](auto hint) {
    constexpr int HINT = decltype(hint)::value;
    // (keys of 64 B experts per token: 7 tokens on 60 experts 17.5 us with B = 1, 22 with 4)
    auto choose = [&](auto width) {
      constexpr int B = decltype(width)::value;
      if (a.t == 1) go(moe_gated_kernel<R, 1, HINT, B>, slots + 1);
      else go(moe_gated_kernel<R, kFewTokens, HINT, B>, slots + 1);
    };
    if (lg == nullptr) go(moe_gated_kernel<R, 0, HINT, 1>, slots);
    else if (a.experts <= 64) choose(Slot<1>{});
    else if (a.experts <= 128) choose(Slot<2>{});
    else choose(Slot<kFewExperts / 64>{});
  };
  // Rows of whole 128-byte lines: every line is fetched once, by one load, and
  // need not stay in the caches (one token, two experts of 2 x 14336 x 5120
  // 34.9 us against 36.5; 16 on 64 of 2 x 1408 x 2048 39.6 against 41.2).
  // Where two loads share a line it has to: 7 on 60 of 2 x 704 x 1984 24.8
  // against 21.8.
  if (a.k % 256 == 0) pick(Slot<kOnce>{});
  else pick(Slot<0>{});
  return hipGetLastError();
}

hipError_t launch_down(const MoeArgs& a, const void* h, float* parts, hipStream_t s) {
  constexpr int R = kWideRowTiles;
  const int P = (int)(a.t * a.top_k);
  const dim3 grid((unsigned)ceil_div(a.k, kWideWaves * 16 * R), grid_rows(a), (unsigned)down_parts(a));
  const auto codes = static_cast<const uint8_t*>(a.codes_down);
  const auto scales = static_cast<const uint16_t*>(a.scales_down);
  auto go = [&](auto kern) {
    kern<<<grid, dim3(64 * kWideWaves), 0, s>>>(
        static_cast<const uint16_t*>(h), codes, scales, codes, scales, static_cast<const int*>(a.ids), parts,
        (int)a.inner, (int)a.k, (int)a.experts, P, (int)a.top_k, (uint32_t)((int64_t)P * a.inner * 4));
  };
  if (P / experts_hit(a) >= kManyPairs) go(moe_wide_kernel<R, true, 32>);
  else go(moe_wide_kernel<R, true, 16>);
  return hipGetLastError();
}

}  // namespace

// Up to this many router values one workgroup per token makes them all
// (one launch).
constexpr int64_t kSmallRouter = 64 * 1024;
constexpr int64_t kFewLogits = 1024;

size_t moe_route_workspace_bytes(int64_t k, int64_t experts, int64_t t) {
  return experts * k <= kSmallRouter ? 0 : al256((size_t)(t * experts * 8));
}

hipError_t launch_moe_route(const MoeArgs& a, void* workspace, hipStream_t s) {
  const auto x = static_cast<const uint16_t*>(a.x), router = static_cast<const uint16_t*>(a.router);
  int* ids = static_cast<int*>(a.ids);
  float* weights = static_cast<float*>(a.weights);
  const int K = (int)a.k, E = (int)a.experts, T = (int)a.t, top_k = (int)a.top_k;
  if (workspace == nullptr || moe_route_workspace_bytes(a.k, a.experts, a.t) == 0) {
    moe_route_kernel<<<dim3((unsigned)T), dim3(kRouteThreads), 0, s>>>(x, router, ids, weights, K, E, top_k, a.renorm);
    return hipGetLastError();
  }
  double* lg = static_cast<double*>(workspace);
  // Few logits: a workgroup each (16 tokens, 64 experts of 4096: 4.7 us).  Many: four a wave (64 tokens, 128 experts
  // of 2048: 4.8 us; sixteen a wave 6.5, and the same time from 256 tokens on).
  if ((int64_t)T * E <= kFewLogits) moe_one_logit_kernel<<<dim3((unsigned)E, (unsigned)T), dim3(256), 0, s>>>(x, router, lg, K, E);
  else moe_logits_kernel<2, 2><<<dim3((unsigned)((T + 1) / 2), (unsigned)((E + 7) / 8)), dim3(256), 0, s>>>(x, router, lg, K, E, T);
  if (E <= 256) moe_choose_kernel<4><<<dim3((unsigned)T), dim3(64), 0, s>>>(lg, ids, weights, E, top_k, a.renorm);
  else moe_choose_kernel<kMaxExperts / 64><<<dim3((unsigned)T), dim3(64), 0, s>>>(lg, ids, weights, E, top_k, a.renorm);
  return hipGetLastError();
}

// h of every pair in two bf16 parts, then every pair's down products (the
// router's logits lie where h comes to lie)
size_t moe_workspace_bytes(int64_t inner, int64_t k, int64_t experts, int64_t top_k, int64_t t) {
  const size_t route = moe_route_workspace_bytes(k, experts, t);
  MoeArgs a{};
  a.inner = inner, a.k = k, a.experts = experts, a.top_k = top_k, a.t = t;
  const size_t sums = few_pairs(a) ? 0 : (size_t)down_parts(a) * (size_t)(t * top_k * k * 4);
  // (a few tokens' logits lie where the sums would)
  const size_t lg = t <= kFewTokens ? (size_t)(t * experts * 8) : 0;
  const size_t all = al256((size_t)(t * top_k * inner * 4)) + al256(sums > lg ? sums : lg);
  return route > all ? route : all;
}

hipError_t launch_moe_experts(const MoeArgs& a, const double* lg, void* workspace, hipStream_t s) {
  void* h = workspace;
  const int64_t h_bytes = a.t * a.top_k * a.inner * 4;
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + al256((size_t)h_bytes));
  hipError_t e = launch_gated(a, h, lg, s);
  if (e != hipSuccess) return e;
  const int* ids = static_cast<const int*>(a.ids);
  const float* weights = static_cast<const float*>(a.weights);
  uint16_t* y = static_cast<uint16_t*>(a.y);
  if (few_pairs(a)) {
    // 32 rows a workgroup where that is half a workgroup per CU or more
    const bool two = a.k >= 32 * 128;
    auto go = [&](auto kern) {
      kern<<<dim3((unsigned)ceil_div(a.k, two ? 32 : 16)), dim3(64 * kFewWaves), 0, s>>>(
          static_cast<const uint16_t*>(h), static_cast<const uint8_t*>(a.codes_down),
          static_cast<const uint16_t*>(a.scales_down), ids, weights, y, (int)a.inner, (int)a.k, (int)a.experts,
          (int)a.t, (int)a.top_k, (uint32_t)h_bytes);
    };
    if (two) go(moe_down_few_kernel<2>);
    else go(moe_down_few_kernel<1>);
    return hipGetLastError();
  }
  e = launch_down(a, h, parts, s);
  if (e != hipSuccess) return e;
  const int64_t quads = a.t * (a.k / 4);
  const int vec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
  const dim3 grid((unsigned)((quads + 255) / 256));
  // pairs whose loads are in flight together: eight of eight 4.7 us, one after the other 5.5 (64 tokens, 2048
  // outputs); two of two 5.6, eight loads 7.0 (96 tokens, 5120 outputs)
  (a.top_k <= 2 ? moe_combine_kernel<2> : a.top_k <= 4 ? moe_combine_kernel<4> : moe_combine_kernel<8>)
      <<<grid, dim3(256), 0, s>>>(parts, ids, weights, y, (int)a.k, (int)a.experts, (int)a.top_k, (int)a.t,
      down_parts(a), vec);
  return hipGetLastError();
}

hipError_t launch_moe_experts(const MoeArgs& a, void* workspace, hipStream_t s) {
  return launch_moe_experts(a, nullptr, workspace, s);
}

// The whole layer.  A few tokens' logits lie behind h and the choice is made
// where it is used (every workgroup of the gate and up products makes it for
// itself): a launch fewer.
hipError_t launch_moe(const MoeArgs& a, void* workspace, hipStream_t s) {
  if (a.t > kFewTokens || a.experts > kFewExperts || a.t * a.top_k > kPairGrid) {
    const hipError_t e = launch_moe_route(a, workspace, s);
    return e == hipSuccess ? launch_moe_experts(a, nullptr, workspace, s) : e;
  }
  double* lg = reinterpret_cast<double*>(static_cast<uint8_t*>(workspace) + al256((size_t)(a.t * a.top_k * a.inner * 4)));
  moe_one_logit_kernel<<<dim3((unsigned)a.experts, (unsigned)a.t), dim3(256), 0, s>>>(
      static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.router), lg, (int)a.k, (int)a.experts);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? launch_moe_experts(a, lg, workspace, s) : e;
}

}  // namespace q4lin
