// q4lin_moe.hip -- a mixture-of-experts layer for few tokens, experts in
// Q4_G64_FP16:
//
//     l[t][e] = sum_k router[e][k] x[t][k],  p = softmax over e,
//     the top_k largest l of a token (equals: the lowest e) with weights p,
//     h_j = silu(Wg_e x) * (Wu_e x),         e = ids[t][j],
//     y[t] = bf16( sum_j weights[t][j] Wd_e h_j ).
//
// A choice (t, j) is a "pair" p = t top_k + j.  Launches: route (one
// workgroup per token), the gate and up products with the gate applied, the
// down products of every pair, and their weighted sum per token.  A pair
// whose id is outside 0..E-1 takes part in nothing.
//
// Expert products, bound by the weight stream (34 bytes per 64 weights of
// each expert that some token chose, read once for up to 32 activation
// rows): a wave takes 64 rows of one expert (32 gate rows and the same 32 up
// rows, or 64 down rows) and all of its pairs, and streams its share of K
// through an LDS ring; the four waves of a workgroup share K or the rows.
// The arithmetic is that of the library's other matrix-core routes: exact
// bf16 values 128 + q, products of a constant all-8 operand through the same
// instructions subtracted, the group's scale applied in binary32; the waves'
// partials are summed in binary64.  h is kept as two bf16 parts (16
// significant bits), as two activation rows per pair: one bf16 would cost as
// much precision as the store of y.
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

// One workgroup per token.  The logits are sums of exact bf16 products,
// eight at a time in binary32 and those in binary64, so that the order of
// two experts is that of their exact logits but for differences near 2^-24
// of the terms.  The rank of an expert is the number of experts before it,
// counted by all threads; a NaN counts as the lowest.
__global__ void __launch_bounds__(kRouteThreads)
moe_route_kernel(const uint16_t* __restrict__ x, const uint16_t* __restrict__ router, int* __restrict__ ids,
                 float* __restrict__ weights, int K, int E, int top_k, int renorm) {
  __shared__ double lg[kMaxExperts];
  __shared__ int rank[kMaxExperts];
  __shared__ double part[kRouteThreads / 64];
  __shared__ double top;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const size_t t = blockIdx.x;
  const uint16_t* xr = x + t * K;
  rank[tid] = 0;
  for (int e0 = 4 * wave; e0 < E; e0 += 4 * (kRouteThreads / 64)) {
    const uint16_t* r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = router + (size_t)min(e0 + i, E - 1) * K;
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 2
    for (int k = 8 * lane; k < K; k += 512) {
      const u32x4_t xv = *reinterpret_cast<const u32x4_t*>(xr + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += (double)dot8(*reinterpret_cast<const u32x4_t*>(r[i] + k), xv);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double s = sum64_lanes(acc[i]);
      if (lane == 0 && e0 + i < E) lg[e0 + i] = s;
    }
  }
  __syncthreads();
  // ranks: thread (part, e) counts the experts j = part, part + parts, ... before e
  int ep = 64;
  while (ep < E) ep <<= 1;
  {
    const int e = tid & (ep - 1), parts = kRouteThreads / ep;
    if (e < E) {
      const double le = lg[e], ke = le != le ? -__builtin_inf() : le;
      int n = 0;
      for (int j = tid / ep; j < E; j += parts) {
        const double lj = lg[j], kj = lj != lj ? -__builtin_inf() : lj;
        n += kj > ke || (kj == ke && j < e);
      }
      atomicAdd(&rank[e], n);  // (whole numbers: any order)
    }
  }
  __syncthreads();
  const bool on = tid < E;
  const int rk = on ? rank[tid] : kMaxExperts;
  if (rk == 0) top = lg[tid];
  __syncthreads();
  const double pe = on && (rk < top_k || !renorm) ? exp(lg[tid] - top) : 0.0;
  const double ps = sum64_lanes(pe);
  if (lane == 0) part[wave] = ps;
  __syncthreads();
  if (rk < top_k) {
    double sum = 0.0;
    for (int w = 0; w < kRouteThreads / 64; ++w) sum += part[w];
    ids[t * top_k + rk] = tid;
    weights[t * top_k + rk] = (float)(pe / sum);
  }
}

// ---------------------------------------------------------------------------
// Expert products
// ---------------------------------------------------------------------------
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
// up to this many pairs the grid has a row of workgroups per pair (that of
// an expert's first pair works), beyond it one per expert
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
//   * Activations, GP = 1 (NT tiles of 16 activation rows): four lanes load
//     from one row; a lane exchange hands them over.
//   * Activations, GP = 2 or 4 (at most 8 or 4 activation rows): a tile's 16
//     rows are those rows times GP scale groups, zero but for the products
//     of the own group.  A product of GP groups' codes with such operands
//     keeps the groups' sums apart in different rows of one accumulator, so
//     that the scales (lane l: row l % 16, the group of its accumulator
//     rows) cost one multiplication for GP groups.
constexpr int kTileStage = 16 * 128;  // code bytes of a row tile in a stage

template <int NT, int GP>
struct Acts {
  u32x4_t v[NT][8 / GP];
};
template <bool DOWN>
struct Scales {
  u32x4_t v[DOWN ? 1 : 2];
  uint32_t next[DOWN ? 1 : 2];
};

// Gate and up (DOWN false): act = x, codes[0]/[1] the gate and up weights,
// out = h in two parts, [pair][part][rows] in the paired order.  Down: act =
// h, codes0 the down weight, out float [pair][rows].  K: the inner dimension
// of this product, rows: the rows of one expert, wk: waves that share K (the
// other kWaves / wk share the workgroup's rows).
template <int R, bool DOWN>
__global__ void __launch_bounds__(kThreads, 2)
moe_expert_kernel(const uint16_t* act, const uint8_t* codes0, const uint16_t* scales0, const uint8_t* codes1,
                  const uint16_t* scales1, const int* __restrict__ ids, void* out, int K, int rows, int E, int P,
                  int top_k, uint32_t act_bytes, int wk) {
  constexpr int RP = DOWN ? 2 : 1;       // activation rows per pair
  constexpr int BT = 32 / RP;            // pairs per pass, at most
  constexpr int RT = DOWN ? R : R / 2;   // row tiles of the output per wave
  constexpr int SLOT = R * kTileStage;   // bytes of one stage's codes
  typedef float Red[R][16][20];
  static_assert(sizeof(Red) <= (size_t)SLOT, "the waves' sums reuse a ring slot");
  // the rings' two slots (two objects, so that a read of one is known not to
  // depend on a copy in flight into the other)
  __shared__ __attribute__((aligned(16))) uint8_t ring0[kWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t ring1[kWaves * SLOT];
  __shared__ int list[kWaves][BT];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int wr = kWaves / wk, kp = wave % wk, rp = wave / wk;

  int e = blockIdx.y;
  if (P <= kPairGrid) {
    const int id = lane < P ? ids[lane] : -1;
    e = __builtin_amdgcn_readlane(id, blockIdx.y);
    if ((uint32_t)e >= (uint32_t)E) return;
    const uint64_t mask = __builtin_amdgcn_ballot_w64(id == e);
    if ((mask & ((1ull << blockIdx.y) - 1)) != 0) return;  // an earlier pair's workgroups serve it
  }

  const int n0 = (blockIdx.x * wr + rp) * (16 * RT);  // this wave's first output row
  const int G = K >> 6, stages = (G + 3) >> 2;
  const int sb = stages * kp / wk, se = stages * (kp + 1) / wk;
  const uint32_t crow = (uint32_t)K >> 1, srow = (uint32_t)G * 2;
  rsrc_t rc[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t0 = n0 + 16 * (r % RT);
    // (rows are multiples of 16: a tile is whole or absent)
    rc[r] = make_rsrc((r < RT ? codes0 : codes1) + ((size_t)e * rows + t0) * crow, t0 < rows ? 16u * crow : 0u);
  }
  const rsrc_t rx = make_rsrc(act, act_bytes);
  const uint32_t c_off = (uint32_t)(lane >> 3) * crow + 16u * ((lane & 7) ^ (lane >> 3));
  // the scales of row `lane` of the wave's 16 R rows: relative to the dword
  // that holds the first of the wave's rows in its plane
  const int srows = min(16 * RT, rows - n0);
  const bool mine0 = lane < srows, mine1 = !DOWN && lane >= 16 * RT && lane - 16 * RT < srows;
  const size_t s0 = ((size_t)e * rows + n0) * G;
  const uintptr_t sa0 = reinterpret_cast<uintptr_t>(scales0 + s0), sa1 = reinterpret_cast<uintptr_t>(scales1 + s0);
  const uint32_t skew0 = (uint32_t)(sa0 & 2), skew1 = (uint32_t)(sa1 & 2);
  const rsrc_t rs0 = make_rsrc(reinterpret_cast<const void*>(sa0 - skew0),
                               srows > 0 ? (skew0 + (uint32_t)srows * srow + 3u) & ~3u : 0u);
  const rsrc_t rs1 = make_rsrc(reinterpret_cast<const void*>(sa1 - skew1),
                               srows > 0 ? (skew1 + (uint32_t)srows * srow + 3u) & ~3u : 0u);
  const uint32_t so0 = skew0 + (uint32_t)lane * srow, so1 = skew1 + (uint32_t)(lane - 16 * RT) * srow;
  const uint32_t s_off0 = mine0 ? so0 & ~3u : kNowhere, s_off1 = mine1 ? so1 & ~3u : kNowhere;
  const uint32_t s_shift = ((mine1 ? so1 : so0) & 2) * 8;
  const bool skewed = (G & 1) != 0 || skew0 != 0 || skew1 != 0;

  int rd[4];  // this lane's 8 code bytes of group g in a slot: row li, byte 32 g + 8 lq of a tile
#pragma unroll
  for (int g = 0; g < 4; ++g)
    rd[g] = wave * SLOT + li * 128 + 16 * ((2 * g + (lq >> 1)) ^ (li & 7)) + 8 * (lq & 1);
  const int xsrc4 = (4 * li + lq) * 4;  // the lane holding this lane's activations after an exchange (byte address)

  // One pass over the wave's share of K for the mr activation rows of the
  // list, then the workgroup's sums
  auto pass = [&](auto ntc, auto gpc, int mr) __device__ {
    constexpr int NT = decltype(ntc)::value, GP = decltype(gpc)::value;
    static_assert(GP == 1 || NT == 1, "packed groups take one tile");
    constexpr int MT = 16 / GP;                 // activation rows of a tile
    constexpr int LOADS = 2 * R + NT * 8 / GP;  // of one stage, the scales not counted
    constexpr bool PAIRED = DOWN || NT == 1;    // code order of the products (x is permuted into it up to one tile)
    uint32_t x_off[NT];
  #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int a = GP == 1 ? 16 * nt + (lane >> 2) : li % MT;
      const int p = list[wave][min(a, mr - 1) / RP];
      const uint32_t row = DOWN ? 2u * p + (a & 1) : (uint32_t)(p / top_k);
      // (rows past the last read as zeros)
      x_off[nt] = a < mr ? row * (uint32_t)K * 2u + (GP == 1 ? 32u * (lane & 3) : 32u * lq + 128u * (li / MT)) : kNowhere;
    }
    f32x4_t acc[NT][R];
  #pragma unroll
    for (int nt = 0; nt < NT; ++nt)
  #pragma unroll
      for (int r = 0; r < R; ++r) acc[nt][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // (a stage past the wave's share and groups past K: offsets past every
    // range, which read as zeros)
    auto load_scales = [&](Scales<DOWN>& L, int s) __device__ {
      const uint32_t away = s < se ? 0u : kNowhere;
      const uint32_t o0 = (s_off0 + 8u * (uint32_t)s) | away, o1 = (s_off1 + 8u * (uint32_t)s) | away;
      L.v[0] = __builtin_amdgcn_raw_buffer_load_b128(rs0, o0, 0, 0);
      if constexpr (!DOWN) L.v[1] = __builtin_amdgcn_raw_buffer_load_b128(rs1, o1, 0, 0);
      if (skewed) {
        L.next[0] = __builtin_amdgcn_raw_buffer_load_b32(rs0, o0 + 16, 0, 0);
        if constexpr (!DOWN) L.next[1] = __builtin_amdgcn_raw_buffer_load_b32(rs1, o1 + 16, 0, 0);
      }
      in_order();
    };
    auto load = [&](Acts<NT, GP>& L, uint8_t* ring, int s) __device__ {
      const uint32_t away = s < se ? 0u : kNowhere;
  #pragma unroll
      for (int r = 0; r < R; ++r)
  #pragma unroll
        for (int h = 0; h < 2; ++h)
          dma16(rc[r], (c_off + 8u * h * crow + 128u * (uint32_t)s) | away, 0,
                ring + wave * SLOT + (2 * r + h) * (kTileStage / 2));
      in_order();
  #pragma unroll
      for (int g = 0; g < 4 / GP; ++g) {
        const uint32_t away_g = s < se && 4 * s + GP * g + (GP == 1 ? 0 : li / MT) < G ? 0u : kNowhere;
  #pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t o = (x_off[nt] + 512u * (uint32_t)s) | away_g;
          L.v[nt][2 * g] = __builtin_amdgcn_raw_buffer_load_b128(rx, o + 128 * GP * g, 0, 0);
          L.v[nt][2 * g + 1] = __builtin_amdgcn_raw_buffer_load_b128(rx, o + 128 * GP * g + 16, 0, 0);
        }
      }
      in_order();
    };
    // the scales of row `lane`, groups 8 s2 .. 8 s2 + 7 of the wave's share, two a dword
    auto row_scales = [&](const Scales<DOWN>& L, int s, uint32_t (&d)[4]) __device__ {
      u32x4_t v = L.v[0];
      if constexpr (!DOWN) v = v | L.v[1];
      if (skewed) {
        const uint32_t n = DOWN ? L.next[0] : L.next[0] | L.next[1 % (DOWN ? 1 : 2)];
        v = u32x4_t{__builtin_amdgcn_alignbit(v.y, v.x, s_shift), __builtin_amdgcn_alignbit(v.z, v.y, s_shift),
                    __builtin_amdgcn_alignbit(v.w, v.z, s_shift), __builtin_amdgcn_alignbit(n, v.w, s_shift)};
      }
  #pragma unroll
      for (int i = 0; i < 4; ++i) {  // (groups past K belong to another row)
        const int left = G - 4 * s - 2 * i;
        d[i] = v[i] & (left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u);
      }
    };
    auto compute = [&](const Acts<NT, GP>& L, const uint8_t* ring, uint32_t d0, uint32_t d1, int s) __device__ {
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
        w[0] = PAIRED ? q4_paired(cw.x) : q4_natural(cw.x);
        w[1] = PAIRED ? q4_paired(cw.y) : q4_natural(cw.y);
      };
      if constexpr (GP == 1) {
  #pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g > 0 && 4 * s + g >= G) break;
          u32x4_t x[NT][2];
          f32x4_t cr[NT];
  #pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
  #pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[nt][h] = lane_piece(L.v[nt][2 * g + h], xsrc4);
              if constexpr (PAIRED && !DOWN) x[nt][h] = to_paired(x[nt][h]);
            }
            cr[nt] = mfma(x[nt][0], eights, zero);
            cr[nt] = mfma(x[nt][1], eights, cr[nt]);
          }
  #pragma unroll
          for (int r = 0; r < R; ++r) {
            u32x4_t w[2];
            codes(r, g, w);
            const uint32_t sb16 = (g & 1) ? sc[r][g >> 1] >> 16 : sc[r][g >> 1] & 0xFFFFu;
            const float sv = f16_bits_to_f32((uint16_t)sb16);
  #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              f32x4_t p = mfma(x[nt][0], w[0], zero);
              p = mfma(x[nt][1], w[1], p);
  #pragma unroll
              for (int i = 0; i < 4; ++i) acc[nt][r][i] = __builtin_fmaf(sv, p[i] - cr[nt][i], acc[nt][r][i]);
            }
          }
        }
      } else {
  #pragma unroll
        for (int g = 0; g < 4 / GP; ++g) {
          u32x4_t x[GP][2];
          f32x4_t cr = zero;
  #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t v = DOWN ? L.v[0][2 * g + h] : to_paired(L.v[0][2 * g + h]);
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
            for (int i = 0; i < 4; ++i) acc[0][r][i] = __builtin_fmaf(sv, p[i] - cr[i], acc[0][r][i]);
          }
        }
      }
    };
    Acts<NT, GP> L[2];
    Scales<DOWN> S;
    load_scales(S, sb);
    load(L[0], ring0, sb);
    load(L[1], ring1, sb + 1);
    // the stage's copies have landed when only the next stage's loads are
    // outstanding; a slot's reads are done before it is written again
    for (int s = sb; s < se; s += 2) {
      wait_vm<LOADS>();
      in_order();
      uint32_t d[4];
      row_scales(S, s, d);
      compute(L[0], ring0, d[0], d[1], s);
      wait_lgkm0();
      in_order();
      load_scales(S, s + 2);
      load(L[0], ring0, s + 2);
      wait_vm<LOADS>();
      in_order();
      if (s + 1 < se) compute(L[1], ring1, d[2], d[3], s + 1);
      wait_lgkm0();
      in_order();
      load(L[1], ring1, s + 3);
    }
    wait_vm<0>();  // (nothing lands in the rings any more)
    in_order();

    // the sums of the waves that share K (and of a tile's groups)
  #pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (MT * nt >= mr) break;
      if (nt > 0) __syncthreads();
      Red& red = *reinterpret_cast<Red*>(ring0 + wave * SLOT);
      if (MT * nt + 4 * lq % MT < mr)
  #pragma unroll
        for (int r = 0; r < R; ++r)
  #pragma unroll
          for (int i = 0; i < 4; ++i) red[r][4 * lq + i][li] = acc[nt][r][i];
      __syncthreads();
      const int tiles = wr * RT, pairs = min(MT, mr - MT * nt) / RP;
      for (int o = tid; o < 16 * tiles * pairs; o += kThreads) {
        const int c = o & 15, tile = (o >> 4) % tiles, t = (o >> 4) / tiles;
        const int w0 = tile / RT * wk, r = tile % RT, n = (blockIdx.x * tiles + tile) * 16 + c;
        if (n >= rows) continue;
        const int p = list[wave][MT / RP * nt + t];
        auto sum = [&](int rr, int tt) __device__ {
          double v = 0.0;
          for (int w = 0; w < wk; ++w)
  #pragma unroll
            for (int j = 0; j < GP; ++j)
              v += (double)(*reinterpret_cast<const Red*>(ring0 + (w0 + w) * SLOT))[rr][MT * j + tt][c];
          return v;
        };
        if constexpr (DOWN) {
          static_cast<float*>(out)[(size_t)p * rows + n] = (float)(sum(r, 2 * t) + sum(r, 2 * t + 1));
        } else {
          const float g = (float)sum(r, t);
          uint32_t hi, lo;
          split_bf16(g / (1.0f + expf(-g)) * (float)sum(RT + r, t), hi, lo);
          uint16_t* o2 = static_cast<uint16_t*>(out) + (size_t)p * 2 * rows + (n & ~7) + paired_place(n & 7);
          o2[0] = (uint16_t)hi;
          o2[rows] = (uint16_t)lo;
        }
      }
    }
  };

  int m = 1;
  for (int b0 = 0; b0 < m; b0 += BT) {
    // pairs b0 .. b0 + BT - 1 of the expert, in order (each wave its own copy)
    m = 0;
    for (int p0 = 0; p0 < P; p0 += 512) {
      int v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = p0 + 64 * j + lane < P ? ids[p0 + 64 * j + lane] : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t bm = __builtin_amdgcn_ballot_w64(v[j] == e);
        const int r = m + __builtin_popcountll(bm & ((1ull << lane) - 1)) - b0;
        if (v[j] == e && r >= 0 && r < BT) list[wave][r] = p0 + 64 * j + lane;
        m += __builtin_popcountll(bm);
      }
    }
    if (m == 0) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int mr = min(BT, m - b0) * RP;
    // the smallest tiles that hold the rows
    if (mr <= 4) pass(Slot<1>{}, Slot<4>{}, mr);
    else if (mr <= 8) pass(Slot<1>{}, Slot<2>{}, mr);
    else if (mr <= 16) pass(Slot<1>{}, Slot<1>{}, mr);
    else pass(Slot<2>{}, Slot<1>{}, mr);
    __syncthreads();
  }
}

// y[t][n .. n + 3] = bf16( sum_j weights[t][j] parts[t top_k + j][n .. n + 3] ), j in order
__global__ void __launch_bounds__(256)
moe_combine_kernel(const float* __restrict__ parts, const int* __restrict__ ids, const float* __restrict__ weights,
                   uint16_t* __restrict__ y, int rows, int E, int top_k, int T, int vec) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = rows >> 2;
  if (i >= (int64_t)T * per) return;
  const int t = (int)(i / per), n = 4 * (int)(i - (int64_t)t * per);
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < top_k; ++j) {
    const int p = t * top_k + j;
    if ((uint32_t)ids[p] >= (uint32_t)E) continue;
    const f32x4_t d = *reinterpret_cast<const f32x4_t*>(parts + (size_t)p * rows + n);
    const float w = weights[p];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w, d[r], v[r]);
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

constexpr int kRowTiles = 4;  // per wave

template <bool DOWN>
hipError_t launch_experts(const MoeArgs& a, void* h, float* parts, hipStream_t s) {
  constexpr int R = kRowTiles, RT = DOWN ? R : R / 2;
  const int P = (int)(a.t * a.top_k);
  const unsigned slots = (unsigned)(P <= kPairGrid ? P : a.experts);
  const int* ids = static_cast<const int*>(a.ids);
  auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  const int64_t rows = DOWN ? a.k : a.inner;
  // waves that share K: so many that about six waves per CU run (experts in
  // use: at most one per pair)
  const int64_t waves = rows / (16 * RT) * (P < a.experts ? P : a.experts);
  const int wk = waves >= 1400 ? 1 : waves >= 700 ? 2 : 4;
  const int64_t per = kWaves / wk * 16 * RT;
  const dim3 grid((unsigned)((rows + per - 1) / per), slots);
  if (DOWN)
    moe_expert_kernel<R, true><<<grid, dim3(kThreads), 0, s>>>(
        u16(h), u8(a.codes_down), u16(a.scales_down), u8(a.codes_down), u16(a.scales_down), ids, parts, (int)a.inner,
        (int)rows, (int)a.experts, P, (int)a.top_k, (uint32_t)((int64_t)P * a.inner * 4), wk);
  else
    moe_expert_kernel<R, false><<<grid, dim3(kThreads), 0, s>>>(
        u16(a.x), u8(a.codes_gate), u16(a.scales_gate), u8(a.codes_up), u16(a.scales_up), ids, h, (int)a.k, (int)rows,
        (int)a.experts, P, (int)a.top_k, (uint32_t)(a.t * a.k * 2), wk);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_route(const MoeArgs& a, hipStream_t s) {
  moe_route_kernel<<<dim3((unsigned)a.t), dim3(kRouteThreads), 0, s>>>(
      static_cast<const uint16_t*>(a.x), static_cast<const uint16_t*>(a.router), static_cast<int*>(a.ids),
      static_cast<float*>(a.weights), (int)a.k, (int)a.experts, (int)a.top_k, a.renorm);
  return hipGetLastError();
}

// h of every pair in two bf16 parts, then every pair's down products
size_t moe_workspace_bytes(int64_t inner, int64_t k, int64_t experts, int64_t top_k, int64_t t) {
  (void)experts;
  return al256((size_t)(t * top_k * inner * 4)) + al256((size_t)(t * top_k * k * 4));
}

hipError_t launch_moe_experts(const MoeArgs& a, void* workspace, hipStream_t s) {
  void* h = workspace;
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + al256((size_t)(a.t * a.top_k * a.inner * 4)));
  hipError_t e = launch_experts<false>(a, h, parts, s);
  if (e == hipSuccess) e = launch_experts<true>(a, h, parts, s);
  if (e != hipSuccess) return e;
  const int64_t quads = a.t * (a.k / 4);
  const int vec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
  moe_combine_kernel<<<dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s>>>(
      parts, static_cast<const int*>(a.ids), static_cast<const float*>(a.weights), static_cast<uint16_t*>(a.y),
      (int)a.k, (int)a.experts, (int)a.top_k, (int)a.t, vec);
  return hipGetLastError();
}

}  // namespace q4lin
