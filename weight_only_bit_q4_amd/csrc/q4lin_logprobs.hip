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
// equal.  In each wave a bound comes from the lanes' largest logits: the
// largest 16-bit prefix of an order that `top` lanes reach, which is no larger
// than the wave's top-th.  What reaches it and the workgroup's top-th so far
// goes to a list in LDS; a key's place is the number of larger ones in that
// list.  (The list's order depends on the atomic counter, the places do not.)
// Where more logits are equal to the bound than a list holds, a bound of
// whole keys over the 64 lanes of all waves takes its place: then the list is
// at most top lanes' whole share of the tile.
//
// -inf counts for nothing (a row of nothing but -inf: entropy 0, every log
// probability -inf).  A NaN or +inf makes the row's numbers NaN; NaN is the
// lowest key.  Sums are binary32 in a thread, binary64 across threads.
//
// Measured: 500 float32 rows of 50001 25 us without alternatives (100 MB, 4
// TB/s), 40 with five (bounds and lists); one bf16 row of 131072 with twenty
// 12: two dependent launches.
#include "q4lin_kernels.h"
#include "q4lin_device.h"

namespace q4lin {
namespace {

constexpr int kThreads = 256;
constexpr int kTop = 32;  // alternatives, at most
constexpr int64_t kEnough = 512, kWorkgroups = 1024;
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.f);  // -0 counts as 0
  const uint32_t o = b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  return l != l ? 0u : o;
}
__device__ __forceinline__ uint64_t key_of(float l, uint32_t index) {
  return ((uint64_t)order_of(l) << 32) | (uint32_t)~index;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  if (o == 0) return __builtin_nanf("");
  return __builtin_bit_cast(float, o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// Lane maxima without NaN, and the lanes' sums over a common maximum.
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
// z and w over the maximum `to` instead of m (to >= m; a part without any
// finite logit adds nothing, a NaN stays one)
__device__ __forceinline__ void rescale(float m, float to, double& z, double& w) {
  const float d = m > kNegInf ? m - to : 0.f, f = m > kNegInf ? __expf(d) : 0.f;
  w = f > 0.f ? (w + z * (double)d) * (double)f : 0.0;
  z *= (double)f;
}

// The largest 16-bit prefixes of an order that the values of `top` lanes, and
// of `some` lanes, reach (0: fewer lanes have any).
__device__ __forceinline__ void wave_bounds(uint32_t order, int top, int some, uint32_t& bt, uint32_t& bs) {
  bt = bs = 0;
#pragma unroll 4
  for (int bit = 31; bit >= 16; --bit) {
    const uint32_t ct = bt | (1u << bit), cs = bs | (1u << bit);
    bt = __builtin_popcountll(__builtin_amdgcn_ballot_w64(order >= ct)) >= top ? ct : bt;
    bs = __builtin_popcountll(__builtin_amdgcn_ballot_w64(order >= cs)) >= some ? cs : bs;
  }
}

// How many of the n keys are larger than k (eight reads in flight together).
__device__ __forceinline__ int larger(const uint64_t* v, int n, uint64_t k) {
  int c = 0;
  for (int j = 0; j < n; j += 8) {
    uint64_t o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = v[min(j + u, n - 1)];
#pragma unroll
    for (int u = 0; u < 8; ++u) c += j + u < n && o[u] > k ? 1 : 0;
  }
  return c;
}

// The waves' lists of candidates and the `top` best of the tiles so far.
template <int SEG>
struct Best {
  static constexpr int WAVES = kThreads / 64;
  uint64_t list[WAVES * SEG];
  uint64_t lane_max[kThreads];
  uint64_t best[2][kTop];  // largest first, 0: none; a tile reads one and writes the other
  uint64_t bound;
  uint32_t bounds[WAVES];
  int count[WAVES], all;

  // before the first tile (a barrier follows)
  __device__ void clear(int tid) {
    if (tid < 2 * kTop) (&best[0][0])[tid] = 0;
  }
  // Takes the threads' keys of a tile.  each(f) passes them to f one by one (0:
  // none); near(b, f) those of all lanes in which any lane's order may reach
  // b; `order`: the largest order among the thread's.  Reads best[turn], writes
  // the other.
  template <class Each, class Near>
  __device__ __forceinline__ void take(uint32_t order, int top, int tid, int turn, Each&& each, Near&& near) {
    const int lane = tid & 63, wave = tid >> 6;
    const uint64_t* const old = best[turn];
    uint64_t* const now = best[turn ^ 1];
    uint32_t b, of_some;
    wave_bounds(order, top, (top + WAVES - 1) / WAVES, b, of_some);
    if (lane == 0) bounds[wave] = of_some;
    __syncthreads();
    uint32_t least = bounds[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) least = bounds[w] < least ? bounds[w] : least;
    const uint32_t so_far = (uint32_t)(old[top - 1] >> 32);
    const int had = old[0] != 0 ? top : 0;
    b = b > least ? b : least;
    b = b > so_far ? b : so_far;
    int n = 0;
    if (__builtin_amdgcn_ballot_w64(order >= b) != 0)
      near(b, [&](uint64_t k) __device__ {
        const bool hit = k != 0 && (uint32_t)(k >> 32) >= b;
        const uint64_t mask = __builtin_amdgcn_ballot_w64(hit);
        const int at = n + __builtin_popcountll(mask & ((1ull << lane) - 1));
        if (hit && at < SEG) list[wave * SEG + at] = k;
        n += __builtin_popcountll(mask);
      });
    if (lane == 0) count[wave] = n;
    __syncthreads();
    int c[WAVES], total = 0, most = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      c[w] = count[w];
      total += c[w];
      most = c[w] > most ? c[w] : most;
    }
    if (most <= SEG) {
      for (int i = tid; i < total + had; i += kThreads) {
        int at = i, w = 0;
#pragma unroll
        for (int v = 0; v < WAVES - 1; ++v)
          if (w == v && at >= c[v]) {
            at -= c[v];
            w = v + 1;
          }
        const uint64_t k = i < total ? list[w * SEG + at] : old[i - total];
        int place = larger(old, had, k);
#pragma unroll
        for (int v = 0; v < WAVES; ++v) place += larger(list + v * SEG, c[v], k);
        if (k != 0 && place < top) now[place] = k;
      }
    } else {
      whole_keys(old, now, top, tid, each);
    }
    __syncthreads();
  }
  // the same by a bound of whole keys
  template <class Each>
  __device__ __forceinline__ void whole_keys(const uint64_t* old, uint64_t* now, int top, int tid, Each&& each) {
    uint64_t mine = 0;
    each([&](uint64_t k) __device__ { mine = k > mine ? k : mine; });
    lane_max[tid] = mine;
    if (tid == 0) all = 0;
    __syncthreads();
    if (tid < 64) {
      uint64_t k = lane_max[tid];
      for (int j = 1; j < WAVES; ++j) k = lane_max[tid + 64 * j] > k ? lane_max[tid + 64 * j] : k;
      // its place among the 64 (keys differ but for zeros, which lanes order)
      int place = 0;
      for (int l = 0; l < 64; ++l) {
        const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)k, l) |
                           ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(k >> 32), l) << 32);
        place += o > k || (o == k && l < tid) ? 1 : 0;
      }
      if (place == top - 1) {
        const uint64_t b = old[top - 1] > k ? old[top - 1] : k;
        bound = b > 0 ? b : 1;
      }
    }
    __syncthreads();
    const uint64_t b = bound;
    if (mine >= b)
      each([&](uint64_t k) __device__ {
        if (k >= b) list[atomicAdd(&all, 1)] = k;
      });
    __syncthreads();
    const int n = all;
    for (int i = tid; i < n + top; i += kThreads) {
      const uint64_t k = i < n ? list[i] : old[i - n];
      const int place = larger(old, top, k) + larger(list, n, k);
      if (k != 0 && place < top) now[place] = k;
    }
  }
};

template <class T>
struct Logit;
template <>
struct Logit<float> {
  static constexpr int V = 4;  // logits of a 16-byte load
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ void vec(const float* p, float* o) {
    __builtin_memcpy(o, p, 16);
  }
};
template <>
struct Logit<uint16_t> {
  static constexpr int V = 8;
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  static __device__ __forceinline__ void vec(const uint16_t* p, float* o) {
    uint32_t w[4];
    __builtin_memcpy(w, p, 16);
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
  // a wave's list holds the whole share of kTop lanes (and the waves' lists
  // together that of kTop lanes of all waves)
  __shared__ Best<kTop * EPT> best;
  __shared__ double part[kThreads / 64][2];
  __shared__ float wave_max[kThreads / 64];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* lr = logits + row * stride;
  const int begin = blockIdx.y * share, end = min(begin + share, N);
  if (top > 0) {
    best.clear(tid);
    __syncthreads();
  }
  float m = kNegInf, z = 0.f, w = 0.f;
  int turn = 0;
  for (int t0 = begin; t0 < end; t0 += TILE, turn ^= 1) {
    float l[EPT];
    // logit j V + i of a thread: t0 + (j kThreads + tid) V + i
    // (16 bytes at a time from wherever the row begins)
    if (t0 + TILE <= end) {
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
      // (past the end there is no key; a NaN is lost in the maximum: it makes
      // z a NaN)
      uint32_t order = order_of(tm);
      if (t0 + TILE > end || z != z) {
        order = 0;
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const int at = t0 + (j / V * kThreads + tid) * V + j % V;
          const uint32_t o = at < end ? order_of(l[j]) : 0u;
          order = o > order ? o : order;
        }
      }
      best.take(order, top, tid, turn, [&](auto&& f) __device__ {
#pragma unroll
        for (int j = 0; j < EPT; ++j) {
          const int at = t0 + (j / V * kThreads + tid) * V + j % V;
          f(at < end ? key_of(l[j], (uint32_t)at) : (uint64_t)0);
        }
      }, [&](uint32_t b, auto&& f) __device__ {
        // (a logit's order reaches b where it is not below b's number, which
        // is a NaN for a bound at -inf or under it: then every logit passes)
        const float low = key_value((uint64_t)b << 32);
#pragma unroll
        for (int j = 0; j < EPT; ++j)
          if (__builtin_amdgcn_ballot_w64(!(l[j] < low)) != 0) {
            const int at = t0 + (j / V * kThreads + tid) * V + j % V;
            f(at < end ? key_of(l[j], (uint32_t)at) : (uint64_t)0);
          }
      });
    }
  }
  // the workgroup's maximum, then its sums over it
  float all = lanes_max(m);
  if ((tid & 63) == 0) wave_max[tid >> 6] = all;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) all = fmaxf(all, wave_max[i]);
  double zs = (double)z, ws = (double)w;
  rescale(m, all, zs, ws);
  zs = sum64_lanes(zs);
  ws = sum64_lanes(ws);
  if ((tid & 63) == 0) {
    part[tid >> 6][0] = zs;
    part[tid >> 6][1] = ws;
  }
  __syncthreads();
  const int64_t at = row * gridDim.y + blockIdx.y;
  if (tid == 0) {
    for (int i = 1; i < kThreads / 64; ++i) {
      zs += part[i][0];
      ws += part[i][1];
    }
    stats[3 * at] = (double)all;
    stats[3 * at + 1] = zs;
    stats[3 * at + 2] = ws;
  }
  if (tid < top) keys[at * top + tid] = best.best[turn][tid];
}

// Joins the shares of a row (at most 64) and writes its numbers.
template <class T>
__global__ void __launch_bounds__(kThreads)
logprobs_join_kernel(const T* logits, int64_t stride, int N, int shares, int top, const double* stats,
                     const uint64_t* keys, const int* tokens, float* logprob, float* entropy, float* top_logprobs,
                     int* top_ids) {
  constexpr int KPT = 64 * kTop / kThreads;  // keys of a thread
  __shared__ Best<kTop * KPT> best;
  __shared__ double total[3];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  if (tid < 64) {
    const double* p = stats + 3 * (row * shares + tid);
    float m = kNegInf;
    double z = 0.0, w = 0.0;
    if (tid < shares) {
      m = (float)p[0];
      z = p[1];
      w = p[2];
    }
    const float all = lanes_max(m);
    rescale(m, all, z, w);
    z = sum64_lanes(z);
    w = sum64_lanes(w);
    if (tid == 0) {
      total[0] = (double)all;
      total[1] = z;
      total[2] = w;
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
    uint64_t k[KPT];
    uint32_t order = 0;
#pragma unroll
    for (int j = 0; j < KPT; ++j) {
      const int i = tid + j * kThreads;
      k[j] = i < n ? keys[row * n + i] : 0;
      order = (uint32_t)(k[j] >> 32) > order ? (uint32_t)(k[j] >> 32) : order;
    }
    best.take(order, top, tid, 0, [&](auto&& f) __device__ {
#pragma unroll
      for (int j = 0; j < KPT; ++j) f(k[j]);
    }, [&](uint32_t b, auto&& f) __device__ {
#pragma unroll
      for (int j = 0; j < KPT; ++j)
        if (__builtin_amdgcn_ballot_w64((uint32_t)(k[j] >> 32) >= b) != 0) f(k[j]);
    });
    if (tid < top) {
      const uint64_t b = best.best[1][tid];
      top_logprobs[row * top + tid] = prob(key_value(b));
      top_ids[row * top + tid] = (int)~(uint32_t)b;
    }
  }
}

// Shares of a row: enough workgroups for the chip, each at least one tile.
// Where tiles of 32 logits a thread are too few for that, tiles of eight: one
// row spreads over many workgroups.
struct SharePlan {
  int ept, shares, share;
};
SharePlan plan(int64_t n, int64_t t) {
  const int ept = t * ((n + 32 * kThreads - 1) / (32 * kThreads)) < kEnough ? 8 : 32;
  const int64_t tile = (int64_t)kThreads * ept, tiles = (n + tile - 1) / tile;
  int64_t shares = (kWorkgroups + t - 1) / t;
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
