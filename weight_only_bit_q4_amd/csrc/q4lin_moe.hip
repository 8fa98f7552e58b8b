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
// each expert that some token chose, read once for up to 16 NT pairs): a
// workgroup takes 32 rows of one expert (16 gate rows and the same 16 up
// rows, or 32 down rows), all of its pairs, and its eight waves split K; no
// loop over experts, so the chip's workgroups are (rows / 32) x experts and
// the loads of many resident workgroups cover each other's latency.  The
// arithmetic is that of the library's other matrix-core routes: exact bf16
// values 128 + q, products of a constant all-8 operand through the same
// instructions subtracted, the group's scale applied in binary32; the eight
// waves' partials are summed in binary64.  h is kept as two bf16 parts (16
// significant bits): one bf16 would cost as much precision as the store of y.
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
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
// up to this many pairs the grid has a row of workgroups per pair (that of
// an expert's first pair works), beyond it one per expert
constexpr int kPairGrid = 64;

// Code dword w (k0..k7) -> exact bf16 128 + q in natural order: byte b gives
// its low nibble and, through w >> 4, its high nibble
__device__ __forceinline__ u32x4_t q4_operand(uint32_t w) {
  const uint32_t u = w >> 4;
  u32x4_t r;
  r.x = and_or(__builtin_amdgcn_perm(u, w, 0x04040000u), 0x000F000Fu, 0x43004300u);
  r.y = and_or(__builtin_amdgcn_perm(u, w, 0x05050101u), 0x000F000Fu, 0x43004300u);
  r.z = and_or(__builtin_amdgcn_perm(u, w, 0x06060202u), 0x000F000Fu, 0x43004300u);
  r.w = and_or(__builtin_amdgcn_perm(u, w, 0x07070303u), 0x000F000Fu, 0x43004300u);
  return r;
}

// What a wave loads for one unit (128 k, two scale groups): the codes and
// scales of its two 16-row tiles, the activations of its 16 NT pairs
template <int NT, bool DOWN>
struct Unit {
  static constexpr int XP = DOWN ? 4 : 2;  // 16-byte pieces of activations per group
  u32x4_t c[2];
  uint16_t s[2];
  u32x4_t x[NT][2][XP];
};

// Gate and up (DOWN false): act = x, codes[0]/[1] the gate and up weights,
// out = h in two parts [pair][rows / 8][hi 8 | lo 8].  Down: act = h,
// codes[0] the down weight (the workgroup's rows 0..15 and 16..31), out
// float [pair][rows].  K: the inner dimension of this product, rows: the
// rows of one expert.
template <int NT, bool DOWN>
__global__ void __launch_bounds__(kThreads)
moe_expert_kernel(const uint16_t* __restrict__ act, const uint8_t* __restrict__ codes0,
                  const uint16_t* __restrict__ scales0, const uint8_t* __restrict__ codes1,
                  const uint16_t* __restrict__ scales1, const int* __restrict__ ids, void* __restrict__ out, int K,
                  int rows, int E, int P, int top_k, uint32_t act_bytes) {
  using U = Unit<NT, DOWN>;
  constexpr int BT = 16 * NT;  // pairs per pass
  __shared__ float red[kWaves][2][16][20];
  __shared__ int list[kWaves][BT];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 15, lq = lane >> 4;

  // this workgroup's expert and how many pairs chose it
  int e, m = 0;
  uint64_t mask = 0;
  if (P <= kPairGrid) {
    const int id = lane < P ? ids[lane] : -1;
    e = __builtin_amdgcn_readlane(id, blockIdx.y);
    if ((uint32_t)e >= (uint32_t)E) return;
    mask = __builtin_amdgcn_ballot_w64(id == e);
    if ((mask & ((1ull << blockIdx.y) - 1)) != 0) return;  // an earlier pair's workgroups serve it
    m = __builtin_popcountll(mask);
  } else {
    e = blockIdx.y;
    for (int p = 0; p < P; p += 64)
      m += __builtin_popcountll(__builtin_amdgcn_ballot_w64(p + lane < P && ids[p + lane] == e));
    if (m == 0) return;
  }

  const int n0 = blockIdx.x * (DOWN ? 32 : 16);
  const int G = K >> 6, units = (G + 1) >> 1;
  const int ub = units * wave / kWaves, ue = units * (wave + 1) / kWaves;
  const uint32_t crow = (uint32_t)K >> 1, srow = (uint32_t)G * 2;
  const size_t r0 = (size_t)e * rows + n0, r1 = DOWN ? r0 + 16 : r0;
  const rsrc_t rc0 = make_rsrc(codes0 + r0 * crow, 16 * crow), rc1 = make_rsrc(codes1 + r1 * crow, 16 * crow);
  const rsrc_t rs0 = make_rsrc(scales0 + r0 * G, 16 * srow), rs1 = make_rsrc(scales1 + r1 * G, 16 * srow);
  const rsrc_t rx = make_rsrc(act, act_bytes), rnull = make_rsrc(act, 0u);
  const uint32_t c_off = (uint32_t)li * crow + 16u * lq;
  const uint32_t s_off = (uint32_t)li * srow + 2u * (lq & 1);
  // first activation of this lane in a group (the order that the exchange
  // of code halves in unit_products gives), in bytes
  constexpr int XB = DOWN ? 4 : 2;
  const uint32_t x_in = (uint32_t)(32 * (lq & 1) + 16 * (lq >> 1)) * XB;

  for (int b0 = 0; b0 < m; b0 += BT) {
    // pairs b0 .. b0 + BT - 1 of the expert, in order (each wave its own copy)
    if (P <= kPairGrid) {
      const int r = __builtin_popcountll(mask & ((1ull << lane) - 1)) - b0;
      if (((mask >> lane) & 1) != 0 && r >= 0 && r < BT) list[wave][r] = lane;
    } else {
      int seen = -b0;
      for (int p = 0; p < P && seen < BT; p += 64) {
        const bool hit = p + lane < P && ids[p + lane] == e;
        const uint64_t bm = __builtin_amdgcn_ballot_w64(hit);
        const int r = seen + __builtin_popcountll(bm & ((1ull << lane) - 1));
        if (hit && r >= 0 && r < BT) list[wave][r] = p + lane;
        seen += __builtin_popcountll(bm);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int mb = min(BT, m - b0);
    uint32_t x_off[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int p = list[wave][min(16 * nt + li, mb - 1)];  // places past the last repeat it and are not stored
      x_off[nt] = (uint32_t)(DOWN ? p : p / top_k) * (uint32_t)K * XB + x_in;
    }

    f32x4_t acc[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto load = [&](U& L, int u) {
      const bool live = u < ue;
      L.c[0] = __builtin_amdgcn_raw_buffer_load_b128(live ? rc0 : rnull, c_off + 64u * u, 0, 0);
      L.c[1] = __builtin_amdgcn_raw_buffer_load_b128(live ? rc1 : rnull, c_off + 64u * u, 0, 0);
      // (the second group of an odd K's last unit does not exist: its scale
      // is another row's and is not used)
      L.s[0] = __builtin_amdgcn_raw_buffer_load_b16(live ? rs0 : rnull, s_off + 4u * u, 0, 0);
      L.s[1] = __builtin_amdgcn_raw_buffer_load_b16(live ? rs1 : rnull, s_off + 4u * u, 0, 0);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const rsrc_t r = live && 2 * u + g < G ? rx : rnull;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < U::XP; ++i)
            L.x[nt][g][i] = __builtin_amdgcn_raw_buffer_load_b128(r, x_off[nt], (uint32_t)(128 * u + 64 * g) * XB + 16u * i, 0);
      }
    };
    auto compute = [&](const U& L, int u) {
      const u32x4_t eights = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      // lanes l and l + 32 exchange half of their 16 code bytes: then every
      // lane holds 8 code bytes of each group; a scale row of 16 lanes holds
      // one group, and the row swap gives every lane both
      uint32_t cw[2][2][2];  // [tile][group][dword]
      float sv[2][2];        // [tile][group]
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto sx = __builtin_amdgcn_permlane32_swap(L.c[i].x, L.c[i].z, false, false);
        const auto sy = __builtin_amdgcn_permlane32_swap(L.c[i].y, L.c[i].w, false, false);
        cw[i][0][0] = sx[0];
        cw[i][0][1] = sy[0];
        cw[i][1][0] = sx[1];
        cw[i][1][1] = sy[1];
        const uint32_t f = __builtin_bit_cast(uint32_t, f16_bits_to_f32(L.s[i]));
        const auto ss = __builtin_amdgcn_permlane16_swap(f, f, false, false);
        const uint32_t s0 = ss[0], s1 = ss[1];
        sv[i][0] = __builtin_bit_cast(float, s0);
        sv[i][1] = __builtin_bit_cast(float, s1);
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (g == 1 && 2 * u + 1 >= G) break;
        u32x4_t w[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          w[i][0] = q4_operand(cw[i][g][0]);
          w[i][1] = q4_operand(cw[i][g][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          auto product = [&](u32x4_t b0v, u32x4_t b1v) {
            f32x4_t p;
            if constexpr (DOWN) {
              p = mfma(L.x[nt][g][0], b0v, zero);
              p = mfma(L.x[nt][g][2], b1v, p);
              p = mfma(L.x[nt][g][1], b0v, p);
              p = mfma(L.x[nt][g][3], b1v, p);
            } else {
              p = mfma(L.x[nt][g][0], b0v, zero);
              p = mfma(L.x[nt][g][1], b1v, p);
            }
            return p;
          };
          const f32x4_t cr = product(eights, eights);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f32x4_t p = product(w[i][0], w[i][1]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[nt][i][r] = __builtin_fmaf(sv[i][g], p[r] - cr[r], acc[nt][i][r]);
          }
        }
      }
    };
    U L0, L1;
    load(L0, ub);
    load(L1, ub + 1);
    for (int u = ub; u < ue; u += 2) {
      compute(L0, u);
      load(L0, u + 2);
      if (u + 1 < ue) compute(L1, u + 1);
      load(L1, u + 3);
    }

    // the eight waves' sums
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (16 * nt >= mb) break;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][i][4 * lq + r][li] = acc[nt][i][r];
      __syncthreads();
      const int t = (tid >> 4) & 15, c = tid & 15;
      if (16 * nt + t < mb && (DOWN || tid < 256)) {
        const int p = list[wave][16 * nt + t];
        if constexpr (DOWN) {
          const int i = tid >> 8;
          double v = 0.0;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) v += (double)red[w][i][t][c];
          static_cast<float*>(out)[(size_t)p * rows + n0 + 16 * i + c] = (float)v;
        } else {
          double gv = 0.0, uv = 0.0;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            gv += (double)red[w][0][t][c];
            uv += (double)red[w][1][t][c];
          }
          const float g = (float)gv;
          uint32_t hi, lo;
          split_bf16(g / (1.0f + expf(-g)) * (float)uv, hi, lo);
          uint16_t* o = static_cast<uint16_t*>(out) + ((size_t)p * rows + ((n0 + c) & ~7)) * 2 + (c & 7);
          o[0] = (uint16_t)hi;
          o[8] = (uint16_t)lo;
        }
      }
    }
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

template <int NT>
hipError_t launch_experts(const MoeArgs& a, uint16_t* h, float* parts, hipStream_t s) {
  const int P = (int)(a.t * a.top_k);
  const unsigned slots = (unsigned)(P <= kPairGrid ? P : a.experts);
  const int* ids = static_cast<const int*>(a.ids);
  auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  moe_expert_kernel<NT, false><<<dim3((unsigned)(a.inner / 16), slots), dim3(kThreads), 0, s>>>(
      u16(a.x), u8(a.codes_gate), u16(a.scales_gate), u8(a.codes_up), u16(a.scales_up), ids, h, (int)a.k,
      (int)a.inner, (int)a.experts, P, (int)a.top_k, (uint32_t)(a.t * a.k * 2));
  moe_expert_kernel<NT, true><<<dim3((unsigned)(a.k / 32), slots), dim3(kThreads), 0, s>>>(
      h, u8(a.codes_down), u16(a.scales_down), u8(a.codes_down), u16(a.scales_down), ids, parts, (int)a.inner,
      (int)a.k, (int)a.experts, P, (int)a.top_k, (uint32_t)((int64_t)P * a.inner * 4));
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
  uint16_t* h = static_cast<uint16_t*>(workspace);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + al256((size_t)(a.t * a.top_k * a.inner * 4)));
  // pairs per pass over an expert's rows: about the mean number of its pairs
  const int64_t mean = a.t * a.top_k / a.experts;
  const hipError_t e = mean <= 8 ? launch_experts<1>(a, h, parts, s) : launch_experts<2>(a, h, parts, s);
  if (e != hipSuccess) return e;
  const int64_t quads = a.t * (a.k / 4);
  const int vec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;
  moe_combine_kernel<<<dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, s>>>(
      parts, static_cast<const int*>(a.ids), static_cast<const float*>(a.weights), static_cast<uint16_t*>(a.y),
      (int)a.k, (int)a.experts, (int)a.top_k, (int)a.t, vec);
  return hipGetLastError();
}

}  // namespace q4lin
