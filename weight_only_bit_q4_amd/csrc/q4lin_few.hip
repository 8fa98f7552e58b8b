// q4lin_few.hip -- a Q4 weight times a few tokens, as one stream over the
// weight: MXFP8 activations (q4lin_linear_mx8 up to 16 tokens) and bf16 ones
// with exact codes and binary32 outputs (the logits of q4lin_linear_logprobs
// up to 8 tokens).
//
// Bound: HBM.  Workgroups of eight waves stay on their CU and go through
// their blocks of BN rows one after the other; the waves share K.  A wave's
// codes come in chunks of four groups (128 bytes of a row, whole lines), its
// activations and scales beside them, all copied or loaded NS - 1 chunks ahead
// and across the blocks' borders, so that a CU has some 64 KiB in flight from
// its first block's start to its last block's end.  A block's sums meet in one
// of two LDS buffers behind one barrier; no wave waits for its own stores.
//
// Measured: 34816 x 5120 at two tokens 23 us (4.1 TB/s), at eight 26, at
// sixteen (two slots instead of three) 34; the logits of three tokens on
// 131072 x 5120 73 (4.9 TB/s).  Shares of K that split a line of codes between
// two waves read 492 MB there for 357, and took 87.
//
// On the matrix cores 32 rows x 32 tokens are one instruction's outputs; the
// tokens past T are not scaled or stored (tokens 0..3 and 4..7 are four
// registers of a lane).
#include "q4lin_kernels.h"
#include "q4lin_mx8.h"

namespace q4lin {
namespace {

using mfma16::dma16;
using mfma16::kNowhere;
using mfma16::make_rsrc;
using mfma16::rsrc_t;
using mfma16::wait_lgkm0;
using mfma16::wait_vm;
using mx8::OpBf16;
using mx8::OpMx8;

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kChunk = 4;  // groups

__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// groups of a wave whose offsets fit the table below (bf16 activations)
constexpr int kTable = 64;

struct FewKernel {
  const uint8_t* x;   // OpMx8: E4M3 [T][K]; OpBf16: bf16 [T][K], paired order
  const uint8_t* xs;     // OpMx8: E8M0 [T][K/32]
  const float* offsets;  // OpBf16: [T][K/64]
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* res;  // bf16 [T][N] or nullptr
  void* y;              // bf16, or (F32) float [T][N]
  int N, K, T, BN, blocks;
};

// NS: slots of the rings; TOK: rows of activations in a slot (T at most)
template <class OP, int TOK, int NS, bool F32>
__global__ void __launch_bounds__(kThreads, 2)
few_kernel(FewKernel a) {
  constexpr int REGS = TOK <= 8 ? 4 : 8;       // accumulator registers of a lane that hold tokens
  constexpr int CSLOT = 32 * kChunk * 32;      // a wave's codes of a chunk
  constexpr int XROW = kChunk * OP::XB;        // bytes of a token in a chunk
  constexpr int XSLOT = TOK * XROW;
  constexpr int NC = CSLOT / 1024, NI = XSLOT / 1024;
  constexpr int PPT = XROW / 16, TPI = 64 / PPT;       // pieces of a token, tokens of a copy
  constexpr int ISSUED = 1 + (OP::kScaled ? 1 : 0) + NI + NC;  // loads and copies of a chunk
  static_assert(NS == 2 || NS == 3, "slots");
  // (an object per slot, so that a read of one is known not to depend on a
  // copy in flight into another; one for both kinds: the compiler tells few
  // objects apart)
  constexpr int SLOT = CSLOT + XSLOT;
  __shared__ __attribute__((aligned(16))) uint8_t l0[kWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t l1[kWaves * SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t l2[NS > 2 ? kWaves * SLOT : 16];
  constexpr int RED = kWaves * TOK * 32;  // a block's sums of all waves
  __shared__ __attribute__((aligned(16))) float red[2 * RED];  // [wave][row][token]
  // bf16 activations: the offsets of the codes of each of the wave's groups
  // (four instructions on the constant 136 in each block took 22 of 110 us at
  // three tokens on 131072 x 5120); [wave][group][token]
  constexpr bool TABLE = !OP::kScaled;
  __shared__ __attribute__((aligned(16))) float table[TABLE ? kWaves * kTable * TOK : 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  const int K = a.K, G = K >> 6;
  // (whole chunks to a wave: lines of codes belong to one wave)
  const int all = (G + kChunk - 1) / kChunk;
  const int gb = all * wave / kWaves * kChunk, cnt = min(G, all * (wave + 1) / kWaves * kChunk) - gb;
  const int chunks = cnt > kChunk ? (cnt + kChunk - 1) / kChunk : 1;  // (a wave without groups still meets the others)
  const uint32_t crow = (uint32_t)K >> 1;
  const rsrc_t rx = make_rsrc(a.x, (uint32_t)a.T * (uint32_t)K * (OP::XB / 64));

  // Pieces of row r lie permuted by its key, so that reads of one piece of
  // neighbouring rows spread over the banks.
  uint32_t coff[NC], xoff[NI];
  int cgroup, xgroup[NI];
  {
    const int r = lane >> 3, p = (lane & 7) ^ r;
    cgroup = p >> 1;
#pragma unroll
    for (int j = 0; j < NC; ++j) coff[j] = (uint32_t)(8 * j + r) * crow + 32u * gb + 16u * p;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int t = j * TPI + lane / PPT, xp = (lane % PPT) ^ (t & 7);
      xgroup[j] = xp / (OP::XB / 16);
      xoff[j] = t < a.T ? (uint32_t)t * (uint32_t)K * (OP::XB / 64) + (uint32_t)(OP::XB * gb + 16 * xp) : kNowhere;
    }
  }
  const uint32_t xsrow = (uint32_t)min(li & (TOK - 1), a.T - 1) * 2u * (uint32_t)G;

  struct Scales {
    uint64_t w, x;  // of the chunk's four groups: the row's fp16 scales, the token's pairs of E8M0 bytes
  };
  // The rows' last chunk may have fewer groups: its eight bytes end with the
  // row (G >= 4), and are shifted when they are used.
  auto issue = [&](uint8_t* slot, Scales& s, int block, int c) __device__ {
    const bool in = block < a.blocks;
    const int n0 = in ? block * a.BN : 0;
    const int rows = in ? min(a.BN, a.N - n0) : 0;
    const uint32_t from = 2u * (uint32_t)min(gb + c * kChunk, G - kChunk);
    in_order();
    {
      const uint8_t* base = reinterpret_cast<const uint8_t*>(a.scales) + (size_t)n0 * (2u * (uint32_t)G) + from;
      const uint32_t row = (uint32_t)min(li, rows > 0 ? rows - 1 : 0) * 2u * (uint32_t)G;
      __builtin_memcpy(&s.w, base + row, 8);
      if constexpr (OP::kScaled) __builtin_memcpy(&s.x, a.xs + from + xsrow, 8);
    }
    in_order();
    // (offsets made to pass the range, not branches around the copies: the
    // waits count on every one)
    const uint32_t away = in ? 0u : kNowhere;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      dma16(rx, (xoff[j] + (uint32_t)(c * XROW)) | away | (c * kChunk + xgroup[j] < cnt ? 0u : kNowhere), 0,
            slot + wave * SLOT + CSLOT + j * 1024);
    const rsrc_t rc = make_rsrc(a.codes + (size_t)n0 * crow, (uint32_t)rows * crow);
    const uint32_t caway = c * kChunk + cgroup < cnt ? 0u : kNowhere;  // (no rows: an empty range)
#pragma unroll
    for (int j = 0; j < NC; ++j)
      dma16<mfma16::kOnce>(rc, (coff[j] + (uint32_t)(c * kChunk * 32)) | caway, 0,
                           slot + wave * SLOT + j * 1024);
    in_order();
  };

  float acc[REGS];
#pragma unroll
  for (int i = 0; i < REGS; ++i) acc[i] = 0.f;
  const int tok = li & (TOK - 1);
  // group J of the chunk whose first is `at` of the wave's
  auto group = [&](auto jc, const uint8_t* slot, const Scales& s, int at) __device__ {
    constexpr int J = decltype(jc)::value;
    const uint32_t e = (uint32_t)(s.x >> (32 * (J >> 1))) >> (8 * lh);
    constexpr int SEL = 2 * (J & 1);
    const typename OP::X v = OP::template load_x<J>(slot + wave * SLOT + CSLOT + tok * XROW, tok & 7, lh);
    const typename OP::Q q = OP::template load_q<J>(slot + wave * SLOT + li * (kChunk * 32), li & 7, lh);
    f32x16_t d;
    if constexpr (TABLE) {
      static_assert(!TABLE || REGS == 4, "one read of a lane's tokens");
      d = OP::template product<SEL>(v, q, f32x16_t{}, e);
      const f32x4_t o = *reinterpret_cast<const f32x4_t*>(table + (wave * kTable + at + J) * TOK + (TOK > 4 ? 4 * lh : 0));
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] += o[i];
    } else {
      d = OP::template product<SEL>(v, q, OP::template offset<SEL>(v, e), e);
    }
    const float f = f16_bits_to_f32((uint16_t)(s.w >> (16 * J)));
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
      acc[i] = __builtin_fmaf(f, d[i], acc[i]);
      asm volatile("" : "+v"(acc[i]));  // (here, and not behind the chunk's branches)
    }
  };
  int half = 0;
  // the sums of a block's waves, one output a thread
  auto finish = [&](int block) __device__ {
    // (whole 16-byte writes: smaller ones the compiler pairs, and holds a pair
    // back until every copy in flight has landed)
    float* const mine = red + half + (wave * 32 + li) * TOK + 4 * lh;
#pragma unroll
    for (int i = 0; i < REGS; i += 4)
      if (2 * i + 4 * lh < TOK) *reinterpret_cast<f32x4_t*>(mine + 2 * i) = f32x4_t{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
#pragma unroll
    for (int i = 0; i < REGS; ++i) acc[i] = 0.f;
    wait_lgkm0();
    __builtin_amdgcn_s_barrier();
    in_order();
    const int n0 = block * a.BN;
    for (int o = tid; o < TOK * 32; o += kThreads) {
      const int r = o & 31, t = o >> 5;
      if (r >= a.BN || n0 + r >= a.N || t >= a.T) continue;
      double v = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += (double)red[half + (w * 32 + r) * TOK + t];
      const size_t at = (size_t)t * a.N + n0 + r;
      if constexpr (F32) {
        static_cast<float*>(a.y)[at] = (float)v;
      } else {
        if (a.res != nullptr) v += (double)bf16_bits_to_f32(a.res[at]);
        static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rne((float)v);
      }
    }
    half = RED - half;  // (the next block's sums go to the other buffer: this one is read until its barrier)
    asm("" : "+s"(half));
  };

  Scales sc[NS];
  int ib = blockIdx.x, ic = 0;
  auto advance = [&](int& b, int& c) __device__ {
    if (++c == chunks) {
      c = 0;
      b += gridDim.x;
    }
  };
  auto slot_of = [&](int s) __device__ -> uint8_t* { return s == 0 ? l0 : s == 1 ? l1 : l2; };
  static_for<NS>([&](auto sl) __device__ {
    constexpr int S = decltype(sl)::value;
    issue(slot_of(S), sc[S], ib, ic);
    advance(ib, ic);
  });
  if constexpr (TABLE) {
    for (int i = lane; i < cnt * TOK; i += 64)
      table[wave * kTable * TOK + i] = a.offsets[(size_t)min(i & (TOK - 1), a.T - 1) * G + gb + i / TOK];
    wait_lgkm0();
    in_order();
  }
  int pb = blockIdx.x, pc = 0;
  // A chunk.  (Past the last one the turn of the loop goes on with copies of
  // nothing: an exit between the slots would make the compiler count the
  // copies in flight as if it could return to the loop's start.)
  auto chunk = [&](auto sl) __device__ {
    constexpr int S = decltype(sl)::value;
    in_order();
    wait_vm<(NS - 1) * ISSUED>();  // this chunk has landed, the next NS - 1 are in flight
    in_order();
    Scales s = sc[S];
    const int past = gb + pc * kChunk - min(gb + pc * kChunk, G - kChunk);
    if (past > 0) {
      s.w >>= 16 * (past & 3);
      s.x >>= 16 * (past & 3);
    }
    const int n = pb < a.blocks ? cnt - pc * kChunk : 0;
    if (n >= kChunk)
      static_for<kChunk>([&](auto j) __device__ { group(j, slot_of(S), s, pc * kChunk); });
    else
      static_for<kChunk - 1>([&](auto j) __device__ {
        if (decltype(j)::value < n) group(j, slot_of(S), s, pc * kChunk);
      });
    wait_lgkm0();
    issue(slot_of(S), sc[S], ib, ic);
    advance(ib, ic);
    if (pc == chunks - 1 && pb < a.blocks) finish(pb);
    advance(pb, pc);
  };
  do static_for<NS>(chunk);
  while (pb < a.blocks);
  wait_vm<0>();  // (nothing lands in the slots any more)
}

constexpr int kCUs = 256;

template <class OP, int TOK, int NS, bool F32>
hipError_t launch(FewKernel k, hipStream_t stream) {
  // rows per block: whole rounds of one workgroup per CU
  const int rounds = (k.N + 32 * kCUs - 1) / (32 * kCUs);
  k.BN = (k.N + kCUs * rounds - 1) / (kCUs * rounds);
  k.blocks = (k.N + k.BN - 1) / k.BN;
  few_kernel<OP, TOK, NS, F32><<<dim3((unsigned)(k.blocks < kCUs ? k.blocks : kCUs)), kThreads, 0, stream>>>(k);
  return hipGetLastError();
}

}  // namespace

bool few_mx8_ok(int64_t k, int64_t t) { return t >= 1 && t <= 16 && k >= 64 * kChunk; }
bool few_bf16_ok(int64_t k, int64_t t) {
  return t >= 1 && t <= 8 && k >= 64 * kChunk && k <= 64 * kTable * kWaves;
}

hipError_t launch_few_mx8(const Mx8Args& a, hipStream_t stream) {
  const FewKernel k{static_cast<const uint8_t*>(a.x), static_cast<const uint8_t*>(a.xs), nullptr,
                    static_cast<const uint8_t*>(a.codes), static_cast<const uint16_t*>(a.scales),
                    static_cast<const uint16_t*>(a.res), a.y, (int)a.n, (int)a.k, (int)a.t, 0, 0};
  return a.t <= 8 ? launch<OpMx8, 8, 3, false>(k, stream) : launch<OpMx8, 16, 2, false>(k, stream);
}

hipError_t launch_few_logits(const void* x_paired, const float* offsets, const void* codes, const void* scales,
                             float* logits, int64_t n, int64_t k, int64_t t, hipStream_t stream) {
  const FewKernel f{static_cast<const uint8_t*>(x_paired), nullptr, offsets, static_cast<const uint8_t*>(codes),
                    static_cast<const uint16_t*>(scales), nullptr, logits, (int)n, (int)k, (int)t, 0, 0};
  return t <= 4 ? launch<OpBf16, 4, 3, true>(f, stream) : launch<OpBf16, 8, 2, true>(f, stream);
}

}  // namespace q4lin
