// q4lin_logprobs.hip -- log probabilities of given tokens, entropy and the
// most likely alternatives from rows of logits.
//
//   m = max l    z = sum e^(l - m)    w = sum e^(l - m) (l - m)
//   logprob(i) = l_i - m - log z      entropy = log z - w / z
//
// Bound: bytes (the logits, read once).  A row is cut into shares (few rows)
// or left whole (many), one workgroup each, which goes through it in tiles of
// kTile logits held in registers: every thread keeps its own m, z and w
// (rescaled when its m grows), the workgroup its `top` best so far.  A second
// kernel joins a row's shares.
//
// The best are found without sorting.  Every logit becomes a key of 64 bits
// (its order as an integer, then the lowest index first), so no two are
// equal.  The 64 lanes' largest keys of a tile (four threads each) give a
// bound: the top-th of them is no larger than the tile's top-th key.  Keys at
// or above it (and above the row's top-th so far) go to a list in LDS, at
// most top lanes' whole share of the tile; a key's place is the number of
// larger ones in that list.  The list's order depends on the atomic counter,
// the places do not.
//
// -inf counts for nothing (a row of nothing but -inf: entropy 0, every log
// probability -inf).  A NaN or +inf makes the row's numbers NaN; NaN is the
// lowest key.  Sums are binary32 in a thread, binary64 across threads.
#include "q4lin_kernels.h"
#include "q4lin_device.h"

namespace q4lin {
namespace {

constexpr int kThreads = 256;
constexpr int kTop = 32;  // alternatives, at most
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ uint64_t key_of(float l, uint32_t index) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.f);  // -0 counts as 0
  uint32_t o = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  if (l != l) o = 0;
  return ((uint64_t)o << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  if (o == 0) return __builtin_nanf("");
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

struct Stats {
  double m, z, w;
};
// sums over the larger maximum; a share without any finite logit adds nothing
__device__ __forceinline__ Stats joined(const Stats& a, const Stats& b) {
  const double m = fmax(a.m, b.m);
  Stats s{m, 0.0, 0.0};
  auto add = [&](const Stats& p) __device__ {
    if (p.m == (double)kNegInf) {
      s.z += p.z;  // zero, or NaN from a NaN
      return;
    }
    const double d = p.m - m, f = exp(d);
    s.z += p.z * f;
    s.w += (p.w + p.z * d) * f;
  };
  add(a);
  add(b);
  return s;
}
// (each value by its two halves: shuffles move 32 bits)
__device__ __forceinline__ double lane_xor(double v, int mask) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)b, mask), hi = (uint32_t)__shfl_xor((int)(b >> 32), mask);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ Stats lanes_joined(Stats s, int lanes) {
  for (int d = 1; d < lanes; d *= 2) {
    const Stats o{lane_xor(s.m, d), lane_xor(s.z, d), lane_xor(s.w, d)};
    s = joined(s, o);
  }
  return s;
}

// The workgroup's list of candidates and the `top` best of them.
template <int CAP>
struct Best {
  uint64_t list[CAP];
  uint64_t lane_max[kThreads];
  uint64_t best[kTop];  // largest first; 0: none
  uint64_t bound;
  int count;

  // before the first tile
  __device__ void clear(int tid) {
    if (tid < kTop) best[tid] = 0;
    __syncthreads();
  }
  // Takes the threads' keys of a tile, given by each(f): f(key) for all of
  // them, in two passes; `mine` is the thread's largest.
  template <class Each>
  __device__ void take(uint64_t mine, int top, int tid, Each&& each) {
    lane_max[tid] = mine;
    if (tid == 0) count = 0;
    __syncthreads();
    if (tid < 64) {
      uint64_t k = lane_max[tid];
#pragma unroll
      for (int j = 1; j < kThreads / 64; ++j) k = lane_max[tid + 64 * j] > k ? lane_max[tid + 64 * j] : k;
      // its place among the 64 (keys differ but for zeros, which lanes order)
      int place = 0;
#pragma unroll 8
      for (int l = 0; l < 64; ++l) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, l) |
                           ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), l) << 32);
        place += o > k || (o == k && l < tid) ? 1 : 0;
      }
      if (place == top - 1) {
        uint64_t b = best[top - 1];
        b = b > k ? b : k;
        bound = b > 0 ? b : 1;
      }
      // what was best so far stands in the list first (all of it is in
      // order; what the bound rules out only takes room)
      if (tid < top && best[tid] != 0) {
        list[atomicAdd(&count, 1)] = best[tid];
      }
    }
    __syncthreads();
    const uint64_t b = bound;
    if (mine >= b)
      each([&](uint64_t k) __device__ {
        if (k >= b) {
          const int at = atomicAdd(&count, 1);
          list[at] = k;
        }
      });
    __syncthreads();
    const int n = count;
    if (n > 0) {
      for (int i = tid; i < n; i += kThreads) {
        const uint64_t k = list[i];
        int place = 0;
        for (int j = 0; j < n; ++j) place += list[j] > k ? 1 : 0;
        if (place < top) best[place] = k;
      }
    }
    __syncthreads();
  }
};

template <class T>
struct Logit;
template <>
struct Logit<float> {
  static constexpr int V = 4;  // logits of a 16-byte load
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void vec(const float* p, float* o) {
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = v[i];
  }
};
template <>
struct Logit<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  static __device__ __forceinline__ void vec(const uint16_t* p, float* o) {
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
      o[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xFFFF0000u);
    }
  }
};

// One share of a row: blockIdx.x the row, blockIdx.y the share of `share`
// logits (a multiple of the tile).  stats: 3 doubles per share, keys: top
// each.
template <class T, int EPT>
__global__ void __launch_bounds__(kThreads)
logprobs_share_kernel(const T* logits, int64_t stride, int N, int share, int top, double* stats, uint64_t* keys) {
  using L = Logit<T>;
  constexpr int V = L::V, TILE = kThreads * EPT;
  // a tile's list: at most the whole share of `top` lanes (EPT keys of each
  // of four threads), and the best so far
  __shared__ Best<(kTop * EPT * (kThreads / 64) < TILE ? kTop * EPT * (kThreads / 64) : TILE) + kTop> best;
  __shared__ double part[kThreads / 64][3];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* lr = logits + row * stride;
  const int begin = blockIdx.y * share, end = min(begin + share, N);
  const bool wide = ((uintptr_t)lr & 15u) == 0;  // (a tile starts on a multiple of V logits)
  if (top > 0) best.clear(tid);
  float m = kNegInf, z = 0.f, w = 0.f;
  for (int t0 = begin; t0 < end; t0 += TILE) {
    float l[EPT];
    // logit j V + i of a thread: t0 + (j kThreads + tid) V + i
    if (wide && t0 + TILE <= end) {
#pragma unroll
      for (int j = 0; j < EPT / V; ++j) L::vec(lr + t0 + (j * kThreads + tid) * V, l + j * V);
    } else {
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int at = t0 + (j / V * kThreads + tid) * V + j % V;
        l[j] = at < end ? L::one(lr + at) : kNegInf;
      }
    }
    float tm = kNegInf;
#pragma unroll
    for (int j = 0; j < EPT; ++j) tm = fmaxf(tm, l[j]);
    if (tm > m) {  // (never for a thread without a finite logit)
      if (m > kNegInf) {
        const float d = m - tm, f = __expf(d);
        w = f > 0.f ? (w + z * d) * f : 0.f;  // (z d may have left binary32)
        z *= f;
      }
      m = tm;
    }
    const float base = m > kNegInf ? m : 0.f;
#pragma unroll
    for (int j = 0; j < EPT; ++j) {
      const float d = l[j] - base, e = __expf(d);
      z += e;
      w += e > 0.f ? e * d : 0.f;
    }
    if (top > 0) {
      uint64_t mine = 0;
      // (past the end: no key; the largest of a thread's equal ones is its first)
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int at = t0 + (j / V * kThreads + tid) * V + j % V;
        const uint64_t k = at < end ? key_of(l[j], (uint32_t)at) : 0;
        mine = k > mine ? k : mine;
      }
      best.take(mine, top, tid, [&](auto&& f) __device__ {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const int at = t0 + (j / V * kThreads + tid) * V + j % V;
          f(at < end ? key_of(l[j], (uint32_t)at) : 0);
        }
      });
    }
  }
  Stats s = lanes_joined(Stats{(double)m, (double)z, (double)w}, 64);
  if ((tid & 63) == 0) {
    part[tid >> 6][0] = s.m;
    part[tid >> 6][1] = s.z;
    part[tid >> 6][2] = s.w;
  }
  __syncthreads();
  const int64_t at = row * gridDim.y + blockIdx.y;
  if (tid == 0) {
    for (int i = 1; i < kThreads / 64; ++i) s = joined(s, Stats{part[i][0], part[i][1], part[i][2]});
    stats[3 * at] = s.m;
    stats[3 * at + 1] = s.z;
    stats[3 * at + 2] = s.w;
  }
  if (tid < top) keys[at * top + tid] = best.best[tid];
}

// Joins the shares of a row (at most 64) and writes its numbers.
template <class T>
__global__ void __launch_bounds__(kThreads)
logprobs_join_kernel(const T* logits, int64_t stride, int N, int shares, int top, const double* stats,
                     const uint64_t* keys, const int* tokens, float* logprob, float* entropy, float* top_logprobs,
                     int* top_ids) {
  constexpr int KPT = 64 * kTop / kThreads;  // keys of a thread
  __shared__ Best<64 * kTop + kTop> best;
  __shared__ double total[3];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (tid < 64) {
    const double* p = stats + 3 * (row * shares + tid);
    Stats s{(double)kNegInf, 0.0, 0.0};
    if (tid < shares) s = Stats{p[0], p[1], p[2]};
    s = lanes_joined(s, 64);
    if (tid == 0) {
      total[0] = s.m;
      total[1] = s.z;
      total[2] = s.w;
    }
  }
  if (top > 0) best.clear(tid);
  __syncthreads();
  const double m = total[0], z = total[1], logz = log(z);
  const bool nothing = m == (double)kNegInf && z == 0.0;
  auto prob = [&](float l) __device__ -> float {
    if (nothing) return kNegInf;
    return (float)((double)l - m - logz);
  };
  if (tid == 0) {
    if (entropy != nullptr) entropy[row] = nothing ? 0.f : (float)(logz - total[2] / z);
    if (tokens != nullptr) {
      const int t = tokens[row];
      logprob[row] = (uint32_t)t < (uint32_t)N ? prob(Logit<T>::one(logits + row * stride + t)) : 0.f;
    }
  }
  if (top > 0) {
    const int n = shares * top;
    uint64_t k[KPT], mine = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int i = tid + j * kThreads;
      k[j] = i < n ? keys[row * n + i] : 0;
      mine = k[j] > mine ? k[j] : mine;
    }
    best.take(mine, top, tid, [&](auto&& f) __device__ {
#pragma unroll
      for (int j = 0; j < KPT; ++j) f(k[j]);
    });
    if (tid < top) {
      const uint64_t b = best.best[tid];
      top_logprobs[row * top + tid] = prob(key_value(b));
      top_ids[row * top + tid] = (int)~(uint32_t)b;
    }
  }
}

// Shares of a row: enough workgroups for the chip, each at least one tile.
// Few rows take small tiles (eight logits a thread), so that one row spreads
// over many workgroups.
struct SharePlan {
  int ept, shares, share;
};
SharePlan plan(int64_t n, int64_t t) {
  const int ept = t * n < (int64_t)1024 * 8192 ? 8 : 32;
  const int64_t tile = (int64_t)kThreads * ept, tiles = (n + tile - 1) / tile;
  int64_t shares = (1024 + t - 1) / t;
  shares = shares < 64 ? shares : 64;
  shares = shares < tiles ? shares : tiles;
  const int64_t per = (tiles + shares - 1) / shares;  // tiles a share
  return SharePlan{ept, (int)((tiles + per - 1) / per), (int)(per * tile)};
}

template <class T>
hipError_t launch(const LogprobsArgs& a, void* workspace, hipStream_t stream) {
  const SharePlan p = plan(a.n, a.t);
  double* stats = static_cast<double*>(workspace);
  uint64_t* keys = reinterpret_cast<uint64_t*>(stats + 3 * a.t * p.shares);
  const T* l = static_cast<const T*>(a.logits);
  const dim3 grid((unsigned)a.t, (unsigned)p.shares);
  if (p.ept == 8)
    logprobs_share_kernel<T, 8><<<grid, kThreads, 0, stream>>>(l, a.stride, (int)a.n, p.share, a.top, stats, keys);
  else
    logprobs_share_kernel<T, 32><<<grid, kThreads, 0, stream>>>(l, a.stride, (int)a.n, p.share, a.top, stats, keys);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  logprobs_join_kernel<T><<<dim3((unsigned)a.t), kThreads, 0, stream>>>(
      l, a.stride, (int)a.n, p.shares, a.top, stats, keys, static_cast<const int*>(a.tokens),
      static_cast<float*>(a.logprob), static_cast<float*>(a.entropy), static_cast<float*>(a.top_logprobs),
      static_cast<int*>(a.top_ids));
  return hipGetLastError();
}

}  // namespace

size_t logprobs_workspace_bytes(int64_t n, int64_t t, int top) {
  const SharePlan p = plan(n, t);
  return ((size_t)t * p.shares * (3 * sizeof(double) + top * sizeof(uint64_t)) + 255) & ~(size_t)255;
}

hipError_t launch_logprobs(const LogprobsArgs& a, void* workspace, hipStream_t stream) {
  return a.f32 ? launch<float>(a, workspace, stream) : launch<uint16_t>(a, workspace, stream);
}

}  // namespace q4lin
