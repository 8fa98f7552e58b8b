// q4lin_mx8.hip -- Y = Q4 weight x MXFP8 activations on the scaled matrix
// cores (the operands: q4lin_mx8.h).
//
//   y[t][n] = bf16( sum_g s[n][g] P[t][n][g] (+ residual) ),
//   P = sum over the group of (q - 8) x 2^e, on the matrix cores
//
// A matrix instruction's K is one 64-group: per group and 32 x 32 outputs
// one v_mfma_scale_f32_32x32x64_f8f6f4 (64 clocks) and sixteen multiply-adds
// with the group's scale (64 clocks of the vector ALU), against four bf16
// instructions of 32 clocks for bf16 activations.  One instruction more for
// each group and 32 tokens of a wave forms the codes' offsets (-8 times the
// activations' sum): one of three in the 256- and 128-row tiles, of four in the
// 192-row ones, of two where a wave has 32 rows.  The products' own sums are
// binary32 with the instruction's alignment: terms below about 2^-17 of a
// group's largest q x are cut, also where the offset takes that one away again
// (measured 1e-5 of an output's standard deviation per group; 1e-2 of it in all
// for activations 1000 times the others' on weights that are all zero); the
// sums over groups are binary32 (and binary64 across waves).
//
// Measured, replayed with weights from memory: 6144 x 5120 at 32, 64, 128 and
// 1024 tokens 12.0, 16.4, 24.1 and 54 us (bf16 activations 14.4, 19.1, 24.3 and
// 74); 8192 x 5120 at 1024 tokens 70 (1230 TFLOP/s).  From 129 tokens on the
// bound is instruction issue: sixteen multiply-adds with the group's scale
// beside each matrix instruction, and the codes' unpacking.
//
// Tokens are the rows of D and weight rows its columns, so that a lane holds
// one weight row and its scale is one register.
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
using mx8::v8i_t;

struct Mx8Kernel {
  const uint8_t* x;    // E4M3 [T][K]
  const uint8_t* xs;   // E8M0 [T][K/32]
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* res;  // nullptr: none
  uint16_t* y;
  float* part;  // K split: binary32 sums [share][T][N]; OpBf16: the outputs
  int N, K, T;
  const float* offsets;  // OpBf16: [T][K/64]
};

// Two bytes per group (a weight row's fp16 scales, a token's two block
// scales) of GROUPS groups from group g on, groups at or past `end` as zeros.
// The rows need not be aligned.
template <int GROUPS>
struct Strip {
  uint32_t w[(GROUPS + 1) / 2];
};
template <int GROUPS>
__device__ __forceinline__ Strip<GROUPS> load_strip(const uint8_t* base, uint32_t row, int g, int end) {
  Strip<GROUPS> s;
  const uint8_t* p = base + 2 * (size_t)g;
  if (g + GROUPS <= end) {
    __builtin_memcpy(&s, p + row, 2 * GROUPS);
  } else {
#pragma unroll
    for (int j = 0; j < (GROUPS + 1) / 2; ++j) s.w[j] = 0;
#pragma unroll
    for (int j = 0; j < GROUPS; ++j)
      if (g + j < end) {
        uint16_t v;
        __builtin_memcpy(&v, p + 2 * j + row, 2);
        s.w[j / 2] |= (uint32_t)v << (16 * (j & 1));
      }
  }
  return s;
}
// (opaque, so that the multiply-adds take the converted scale: left to choose,
// the compiler converts in each of them)
__device__ __forceinline__ float scale_of(uint32_t w, int odd) {
  float f = f16_bits_to_f32((uint16_t)(odd ? w >> 16 : w));
  asm("" : "+v"(f));
  return f;
}

__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// one output: the sum, the residual, one rounding
__device__ __forceinline__ uint16_t finished(double v, const uint16_t* res, size_t at) {
  if (res != nullptr) v += (double)bf16_bits_to_f32(res[at]);
  return f32_to_bf16_rne((float)v);
}

// ---------------------------------------------------------------------------
// Up to 128 tokens.  One workgroup of eight waves per block of BN rows; the
// waves share K, so the weight is read once (twice above 64 tokens, by two
// token ranges).  Each wave copies its codes (chunks of CH groups, two slots)
// and activations (groups, NX slots) straight into its own part of LDS,
// whole runs of memory per instruction, and reads them back in operand order;
// no barrier until the eight waves' sums meet.
//
// Every copy of the loop is issued whether or not its group exists (past the
// wave's share it reads nothing), so that the counts of the waits hold.  They
// hold within a chunk only: the scales' loads branch at a row's end, and where
// the branches join the compiler waits for all that is in flight, so that each
// chunk begins with a latency of memory.
// ---------------------------------------------------------------------------
constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

template <int RT, int TT, int CH, int NX>
__global__ void __launch_bounds__(kThreads, 2)
mx8_stream_kernel(Mx8Kernel a, int BN, int ranges) {
  static_assert(NX <= CH && (2 * CH) % NX == 0, "slots");
  constexpr int CROW = CH * 32;                // bytes of a row in a chunk
  constexpr int CPC = CROW / 16;               // 16-byte pieces of it
  constexpr int CSLOT = RT * 32 * CROW;        // a wave's codes of a chunk
  constexpr int XSLOT = TT * 32 * 64;          // a wave's activations of a group
  constexpr int NC = CSLOT / 1024, NI = XSLOT / 1024;
  // (an object per slot, so that a read of one is known not to depend on a
  // copy in flight into another)
  __shared__ __attribute__((aligned(16))) uint8_t c0[kWaves * CSLOT];
  __shared__ __attribute__((aligned(16))) uint8_t c1[kWaves * CSLOT];
  __shared__ __attribute__((aligned(16))) uint8_t x0[kWaves * XSLOT];
  __shared__ __attribute__((aligned(16))) uint8_t x1[kWaves * XSLOT];
  __shared__ __attribute__((aligned(16))) uint8_t x2[NX > 2 ? kWaves * XSLOT : 16];
  __shared__ __attribute__((aligned(16))) uint8_t x3[NX > 2 ? kWaves * XSLOT : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  const int K = a.K, G = K >> 6;
  // (the two ranges of tokens of a block of rows on one XCD, eight apart)
  const int block = ranges == 1 ? blockIdx.x : (int)(blockIdx.x >> 4) * 8 + (int)(blockIdx.x & 7);
  const int n0 = block * BN, rows = min(BN, a.N - n0);
  if (rows <= 0) return;
  const int t0 = ranges == 1 ? 0 : (int)(blockIdx.x >> 3 & 1) * (32 * TT), tokens = min(32 * TT, a.T - t0);
  const int gb = (int)((int64_t)G * wave / kWaves), cnt = (int)((int64_t)G * (wave + 1) / kWaves) - gb;
  const uint32_t crow = (uint32_t)K >> 1;

  const rsrc_t rc = make_rsrc(a.codes + (size_t)n0 * crow, (uint32_t)rows * crow);
  const rsrc_t rx = make_rsrc(a.x + (size_t)t0 * K, (uint32_t)tokens * (uint32_t)K);
  // Row r keeps its pieces permuted (piece p at p ^ key(r)), so that reads of
  // one piece of neighbouring rows spread over the banks.
  auto ckey = [](int r) { return CPC == 8 ? r & 7 : (r >> 1) & 3; };
  auto xkey = [](int r) { return (r >> 1) & 3; };
  constexpr int CPI = 64 / CPC;  // rows of a copy
  uint32_t coff[NC], xoff[NI];
  int cgroup;  // the group of this lane's piece (the key of a row repeats with the copies' rows)
  {
    const int r = lane / CPC, p = (lane % CPC) ^ ckey(r);
    cgroup = p >> 1;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int row = j * CPI + r;
      coff[j] = row < rows ? (uint32_t)row * crow + 32u * gb + 16u * p : kNowhere;
    }
    const int t = lane >> 2, xp = (lane & 3) ^ xkey(t);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int tok = 16 * j + t;
      xoff[j] = tok < tokens ? (uint32_t)tok * (uint32_t)K + 64u * gb + 16u * xp : kNowhere;
    }
  }
  static_assert(CPC == 8 ? CPI % 8 == 0 : CPI % 8 == 0, "a key per lane");
  auto issue_codes = [&](uint8_t* slot, int c) __device__ {
    const bool in = c * CH + cgroup < cnt;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      dma16<mfma16::kOnce>(rc, in ? coff[j] + (uint32_t)c * CROW : kNowhere, 0, slot + wave * CSLOT + j * 1024);
  };
  auto issue_x = [&](uint8_t* slot, int q) __device__ {
    const bool in = q < cnt;
#pragma unroll
    for (int j = 0; j < NI; ++j) dma16(rx, in ? xoff[j] + 64u * (uint32_t)q : kNowhere, 0, slot + wave * XSLOT + j * 1024);
  };
  struct Scales {
    Strip<CH> w[RT], x[TT];
  };
  // (32-bit offsets from the workgroup's first row)
  const uint8_t* const wbase = reinterpret_cast<const uint8_t*>(a.scales + (size_t)n0 * G);
  const uint8_t* const xbase = a.xs + (size_t)t0 * (K >> 5);
  uint32_t wrow[RT], xrow[TT];
#pragma unroll
  for (int r = 0; r < RT; ++r) wrow[r] = (uint32_t)min(32 * r + li, rows - 1) * 2u * (uint32_t)G;
#pragma unroll
  for (int t = 0; t < TT; ++t) xrow[t] = (uint32_t)min(32 * t + li, tokens - 1) * 2u * (uint32_t)G;
  auto load_scales = [&](Scales& s, int c) __device__ {
    const int g = gb + c * CH;
#pragma unroll
    for (int r = 0; r < RT; ++r) s.w[r] = load_strip<CH>(wbase, wrow[r], g, G);
#pragma unroll
    for (int t = 0; t < TT; ++t) s.x[t] = load_strip<CH>(xbase, xrow[t], g, G);
  };

  f32x16_t acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x16_t{};

  // group J of a chunk
  auto group = [&](auto jc, const uint8_t* cs, const uint8_t* xs, const Scales& s) __device__ {
    constexpr int J = decltype(jc)::value, SEL = 2 * (J & 1);
    const uint8_t* cw = cs + wave * CSLOT;
    const uint8_t* xw = xs + wave * XSLOT;
    v8i_t q[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint8_t* p = cw + (32 * r + li) * CROW + 8 * lh;
      q[r] = mx8::code_operand(*reinterpret_cast<const u32x2_t*>(p + 16 * ((2 * J) ^ ckey(li))),
                               *reinterpret_cast<const u32x2_t*>(p + 16 * ((2 * J + 1) ^ ckey(li))));
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const uint8_t* p = xw + (32 * t + li) * 64;
      const v8i_t v = mx8::value_operand(*reinterpret_cast<const u32x4_t*>(p + 16 * (lh ^ xkey(li))),
                                         *reinterpret_cast<const u32x4_t*>(p + 16 * ((2 + lh) ^ xkey(li))));
      const uint32_t e = s.x[t].w[J / 2] >> (8 * lh);
      const f32x16_t off = mx8::offset_sums<SEL>(v, e);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x16_t d = mx8::product<SEL>(v, q[r], off, e);
        const float f = scale_of(s.w[r].w[J / 2], J & 1);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[r][t][i] = __builtin_fmaf(f, d[i], acc[r][t][i]);
      }
    }
  };
  auto xslot = [&](int q) __device__ -> uint8_t* { return q % NX == 0 ? x0 : q % NX == 1 ? x1 : q % NX == 2 ? x2 : x3; };

  if (cnt > 0) {
    Scales s0, s1;
    issue_codes(c0, 0);
    load_scales(s0, 0);
    in_order();
    static_for<NX>([&](auto q) __device__ { issue_x(xslot(decltype(q)::value), decltype(q)::value); });
    issue_codes(c1, 1);
    in_order();
    if (CH < cnt) load_scales(s1, 1);
    // a chunk; false: it held the wave's last group.  Before group q the
    // copies issued after x(q) may be in flight: NX - 1 groups of
    // activations, and the codes of the next chunk if they lie between.
    auto chunk = [&](auto oddc, uint8_t* cs, Scales& s, int c) __device__ {
      bool more = true;
      static_for<CH>([&](auto jc) __device__ {
        constexpr int J = decltype(jc)::value, Q = CH * decltype(oddc)::value + J;
        if (!more) return;
        in_order();
        wait_vm<(NX - 1) * NI + (J < NX ? NC : 0)>();
        in_order();
        group(jc, cs, xslot(Q), s);
        more = c * CH + J + 1 < cnt;
        wait_lgkm0();
        in_order();
        issue_x(xslot(Q), c * CH + J + NX);
        in_order();
      });
      if (!more) return false;
      issue_codes(cs, c + 2);
      in_order();
      if ((c + 2) * CH < cnt) load_scales(s, c + 2);
      return true;
    };
    for (int c = 0;; c += 2) {
      if (!chunk(Slot<0>{}, c0, s0, c)) break;
      if (!chunk(Slot<1>{}, c1, s1, c + 1)) break;
    }
    wait_vm<0>();  // (nothing lands in the slots any more)
  }
  __syncthreads();

  // the waves' sums: a tile of 32 tokens x 32 rows per wave in each of RT TT
  // slots of LDS
  constexpr int TILE = 32 * 32 * 4;
  static_assert(kWaves * CSLOT >= kWaves * TILE && (RT * TT <= 2 || kWaves * XSLOT >= kWaves * TILE), "room");
  auto room = [&](int i) __device__ -> float* {
    return reinterpret_cast<float*>(i == 0 ? c0 : i == 1 ? c1 : i == 2 ? x0 : x1);
  };
  static_for<RT * TT>([&](auto ic) __device__ {
    constexpr int I = decltype(ic)::value;
    float* p = room(I) + wave * 1024 + 128 * lh + li;
#pragma unroll
    for (int i = 0; i < 16; ++i) p[32 * (8 * (i >> 2) + (i & 3))] = acc[I % RT][I / RT][i];
  });
  __syncthreads();
  static_for<RT * TT>([&](auto ic) __device__ {
    constexpr int I = decltype(ic)::value;
    const float* p = room(I);
#pragma unroll
    for (int o = tid; o < 1024; o += kThreads) {
      const int r = 32 * (I % RT) + (o & 31), t = 32 * (I / RT) + (o >> 5);
      if (r >= rows || t >= tokens) continue;
      double v = 0.0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += (double)p[w * 1024 + o];
      const size_t at = (size_t)(t0 + t) * a.N + n0 + r;
      a.y[at] = finished(v, a.res, at);
    }
  });
}

// ---------------------------------------------------------------------------
// More tokens.  A workgroup of WR x WT waves takes WR RT 32 rows and WT TT 32
// tokens.  Stages of two groups (128 bytes of a token, 64 of a row) go
// straight into four slots of LDS, asked for three stages ahead, their copies
// spread over a stage's products (a burst of them holds the waves up at the
// address unit); one barrier per stage.  The scales of kRun groups are read
// row by row (whole runs of memory), one thread a row or token, and put into
// LDS by group, where a lane finds its row's without a gather.
// blockIdx.y: a share of K (binary32 sums to `part`).  OpBf16: bf16 activations
// in the paired order with the offsets of their groups, binary32 outputs to
// `part` (the logits of q4lin_linear_logprobs; twice the bytes of an
// activation, four matrix instructions of 32 clocks a tile instead of one of
// 64, none for the offsets).  Registers: 134 to 211, in the 256 x 128 tiles all
// 256 with one spilled.
// ---------------------------------------------------------------------------
constexpr int kRun = 16;   // groups between two loads of scales: eight stages
constexpr int kSlots = 4;

template <class OP, int WR, int WT, int RT, int TT>
__global__ void __launch_bounds__(64 * WR * WT, 2)
mx8_tile_kernel(Mx8Kernel a, int tiles_n, int tiles_t, int shares) {
  constexpr int WAVES = WR * WT, ROWS = WR * RT * 32, TOKENS = WT * TT * 32, LINES = ROWS + TOKENS;
  constexpr bool F32 = !OP::kScaled;                                 // outputs
  constexpr int XROW = 2 * OP::XB, PPT = XROW / 16, TPC = 64 / PPT;  // bytes of a token in a stage, pieces; tokens of a copy
  // a wave's copies of a stage, 16 rows' codes or TPC tokens each (the last may
  // be of no row: it reads nothing)
  constexpr int NC = (ROWS / 16 + WAVES - 1) / WAVES, NI = TOKENS / TPC / WAVES, LOADS = NC + NI;
  static_assert(NI * WAVES * TPC == TOKENS, "whole copies");
  constexpr int CBYTES = NC * WAVES * 1024, XBYTES = TOKENS * XROW, SLOT = CBYTES + XBYTES;
  static_assert(LINES <= 64 * WAVES, "a thread per row and token");
  // (an object per slot: see the kernel above)
  __shared__ __attribute__((aligned(16))) uint8_t l0[SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t l1[SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t l2[SLOT];
  __shared__ __attribute__((aligned(16))) uint8_t l3[SLOT];
  // by group: the rows' fp16 scales, then the tokens' two E8M0 bytes; those of
  // a lane's rows (tokens), 32 apart, beside each other
  constexpr int RP = RT == 3 ? 4 : RT, ROWROOM = WR * RP * 32, ROOM = ROWROOM + TOKENS;
  static_assert(RT <= 4 && TT <= 2, "one read of a lane's scales");
  // OpBf16: the tokens' offsets by group
  __shared__ __attribute__((aligned(16))) float offs[OP::kScaled ? 4 : 2 * kRun * TOKENS];
  __shared__ __attribute__((aligned(8))) uint16_t table[2 * kRun * ROOM];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int li = lane & 31, lh = lane >> 5;
  const int wr = wave % WR, wt = wave / WR;
  // consecutive workgroups go to the eight XCDs in turn: each XCD takes a run
  // of tiles, the tokens of a few rows, so that its L2 holds those rows once
  int tile = blockIdx.x;
  {
    const int total = tiles_n * tiles_t, each = total / 8, rest = total % 8;
    const int xcd = tile & 7, at = tile >> 3;
    tile = xcd * each + min(xcd, rest) + at;
  }
  const int n0 = tile / tiles_t * ROWS, t0 = tile % tiles_t * TOKENS;
  const int K = a.K, G = K >> 6;
  const int rows = min(ROWS, a.N - n0), tokens = min(TOKENS, a.T - t0);
  const int stages = (G + 1) >> 1;
  const int gb = (int)((int64_t)stages * blockIdx.y / shares) * 2;
  const int ge = min((int)((int64_t)stages * (blockIdx.y + 1) / shares) * 2, G);
  const uint32_t crow = (uint32_t)K >> 1;

  const rsrc_t rc = make_rsrc(a.codes + (size_t)n0 * crow, (uint32_t)rows * crow);
  const uint32_t xrow = (uint32_t)K * (OP::XB / 64);  // bytes of a token
  const rsrc_t rx = make_rsrc(a.x + (size_t)t0 * xrow, (uint32_t)tokens * xrow);
  auto ckey = [](int r) { return (r >> 1) & 3; };
  auto xkey = [](int r) { return r & 7; };
  uint32_t coff[NC], xoff[NI];
  int cgroup, xgroup[NI];  // of this lane's pieces
  {
    const int r = lane >> 2, p = (lane & 3) ^ ckey(r);
    cgroup = p >> 1;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int row = (j * WAVES + wave) * 16 + r;
      coff[j] = row < rows ? (uint32_t)row * crow + 16u * p : kNowhere;
    }
    const int t = lane / PPT;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int tok = (j * WAVES + wave) * TPC + t, xp = (lane % PPT) ^ xkey(tok);
      xgroup[j] = xp / (OP::XB / 16);
      xoff[j] = tok < tokens ? (uint32_t)tok * xrow + 16u * xp : kNowhere;
    }
  }
  // Copy j of the stage at group g.  (Every copy is issued, past the share's
  // end it reads nothing: the waits count on it.  CHECK: g + 2 may pass it.)
  auto copy = [&](auto jc, auto check, uint8_t* slot, int g) __device__ {
    constexpr int J = decltype(jc)::value;
    constexpr bool X = J < NI;
    constexpr int I = X ? J : J - NI;
    const rsrc_t r = X ? rx : rc;
    uint8_t* const to = slot + (X ? CBYTES : 0) + (I * WAVES + wave) * 1024;
    const uint32_t step = X ? (uint32_t)OP::XB : 32u;
    uint32_t off = X ? xoff[X ? I : 0] : coff[X ? 0 : I];
    if constexpr (decltype(check)::value) {
      off = g + (X ? xgroup[X ? I : 0] : cgroup) < ge ? off + step * (uint32_t)g : kNowhere;
      dma16(r, off, 0, to);
    } else {
      dma16(r, off, step * (uint32_t)g, to);
    }
  };

  // this thread's line of scales (32-bit offsets from the workgroup's first)
  const bool of_rows = tid < ROWS;
  const bool has_line = tid < (OP::kScaled ? LINES : ROWS), of_offsets = !OP::kScaled && !of_rows && tid < LINES;
  const float* const obase = OP::kScaled ? nullptr : a.offsets + (size_t)(t0 + min(max(tid - ROWS, 0), tokens - 1)) * G;
  const uint8_t* const lbase = of_rows || !OP::kScaled ? reinterpret_cast<const uint8_t*>(a.scales + (size_t)n0 * G)
                                       : a.xs + (size_t)t0 * (K >> 5);
  const uint32_t line = (uint32_t)(of_rows ? min(tid, rows - 1) : min(tid - ROWS, tokens - 1)) * 2u * (uint32_t)G;
  f32x4_t strip_offs[OP::kScaled ? 1 : kRun / 4];
  auto load_line = [&](Strip<kRun>& s, int g) __device__ {
    if constexpr (!OP::kScaled)
      if (of_offsets)
#pragma unroll
        for (int j = 0; j < kRun; j += 4) {
          if (g + j + 4 <= ge) {
            __builtin_memcpy(&strip_offs[j / 4], obase + g + j, 16);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) strip_offs[j / 4][i] = g + j + i < ge ? obase[g + j + i] : 0.f;
          }
        }
    if (has_line) s = load_strip<kRun>(lbase, line, g, ge);
  };
  // (half: where the table's half begins, 0 or kRun ROOM; an index that the
  // compiler must compute keeps every access a plain one of this object)
  const int at32 = tid >> 5, tok32 = at32 - ROWS / 32;
  const int place = of_rows ? at32 / RT * (RP * 32) + (tid & 31) * RP + at32 % RT
                            : ROWROOM + tok32 / TT * (TT * 32) + (tid & 31) * TT + tok32 % TT;
  auto put_line = [&](const Strip<kRun>& s, int half) __device__ {
    if constexpr (!OP::kScaled)
      if (of_offsets)
#pragma unroll
        for (int j = 0; j < kRun; ++j)
          offs[(half != 0 ? kRun * TOKENS : 0) + j * TOKENS + tid - ROWS] = strip_offs[j / 4][j % 4];
    if (has_line)
#pragma unroll
      for (int j = 0; j < kRun; ++j) table[half + j * ROOM + place] = (uint16_t)(s.w[j / 2] >> (16 * (j & 1)));
  };

  f32x16_t acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = f32x16_t{};

  // (offsets that the compiler cannot relate: it would pair the reads of two
  // row tiles, and hold the pair back until every copy in flight has landed)
  uint32_t roff[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    roff[r] = (uint32_t)(((wr * RT + r) * 32 + li) * 64);
    asm("" : "+v"(roff[r]));
  }
  // group J of a stage; scales: where its line of the table begins; copies(i):
  // room for a copy beside the i-th of two products
  auto group = [&](auto jc, const uint8_t* slot, int scales, auto&& copies) __device__ {
    constexpr int H = decltype(jc)::value;
    typename OP::X v[TT];
    f32x16_t off[TT];
    const uint16_t* const fp = table + scales + (wr * 32 + li) * RP;
    const uint16_t* const ep = table + scales + ROWROOM + (wt * 32 + li) * TT;
    u32x2_t fs;
    if constexpr (RP == 4) fs = *reinterpret_cast<const u32x2_t*>(fp);
    else if constexpr (RP == 2) fs.x = *reinterpret_cast<const uint32_t*>(fp);
    else fs.x = *fp;
    uint32_t e = 0;
    if constexpr (OP::kScaled) e = (TT == 2 ? *reinterpret_cast<const uint32_t*>(ep) : (uint32_t)*ep) >> (8 * lh);
    static_for<TT>([&](auto tc) __device__ {
      constexpr int t = decltype(tc)::value;
      v[t] = OP::template load_x<H>(slot + CBYTES + ((wt * TT + t) * 32 + li) * XROW, xkey(li), lh);
      if constexpr (OP::kScaled) {
        off[t] = OP::template offset<2 * t>(v[t], e);
      } else {
        const float* const o = offs + scales / ROOM * TOKENS + (wt * TT + t) * 32 + 4 * lh;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4_t four = *reinterpret_cast<const f32x4_t*>(o + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) off[t][4 * i + j] = four[j];
        }
      }
    });
    copies(Slot<0>{});
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const typename OP::Q q = OP::template load_q<H>(slot + roff[r], ckey(li), lh);
      const float f = scale_of(r < 2 ? fs.x : fs.y, r & 1);
      static_for<TT>([&](auto tc) __device__ {
        constexpr int t = decltype(tc)::value;
        const f32x16_t d = OP::template product<2 * t>(v[t], q, off[t], e);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[r][t][i] = __builtin_fmaf(f, d[i], acc[r][t][i]);
        // (the sums are needed here: left alone, the compiler moves them past
        // the stages and keeps every product until then)
        asm volatile("" : "+v"(acc[r][t]));
      });
      if (r == 0) copies(Slot<1>{});
    }
  };
  auto slot_of = [&](int s) __device__ -> uint8_t* {
    return s % kSlots == 0 ? l0 : s % kSlots == 1 ? l1 : s % kSlots == 2 ? l2 : l3;
  };

  if (gb < ge) {
    Strip<kRun> strip;
    load_line(strip, gb);
    in_order();
    static_for<kSlots - 1>([&](auto sc) __device__ {
      constexpr int S = decltype(sc)::value;
      static_for<LOADS>([&](auto j) __device__ { copy(j, Slot<1>{}, slot_of(S), gb + 2 * S); });
    });
    in_order();
    put_line(strip, 0);
    // A turn of the loop: a run of scales, eight stages.  WHOLE: all of its
    // groups exist, and those of the three stages behind it.
    auto turn = [&](auto whole, int half, int g0) __device__ {
      constexpr bool WHOLE = decltype(whole)::value;
      static_for<kRun / 2>([&](auto sc) __device__ {
        constexpr int S = decltype(sc)::value;
        const int g = g0 + 2 * S;
        if (!WHOLE && g >= ge) return;
        in_order();
        wait_vm<(kSlots - 2) * LOADS>();  // this stage's copies; two stages' are in flight
        wait_lgkm0();                     // and the reads of the slot that is filled next are done
        __builtin_amdgcn_s_barrier();
        in_order();
        if (S == 0 && g0 + kRun < ge) load_line(strip, g0 + kRun);
        if (S == 4 && g0 + kRun < ge) put_line(strip, kRun * ROOM - half);
        uint8_t* const next = slot_of(S + kSlots - 1);
        // a stage's copies in four places
        auto some = [&](auto place) __device__ {
          constexpr int P = decltype(place)::value;
          in_order();
          static_for<LOADS>([&](auto j) __device__ {
            if constexpr (decltype(j)::value * 4 / LOADS == P) copy(j, Slot<WHOLE ? 0 : 1>{}, next, g + 2 * (kSlots - 1));
          });
          in_order();
        };
        group(Slot<0>{}, slot_of(S), half + 2 * S * ROOM, some);
        if (WHOLE || g + 1 < ge)
          group(Slot<1>{}, slot_of(S), half + (2 * S + 1) * ROOM,
                [&](auto p) __device__ { some(Slot<2 + decltype(p)::value>{}); });
        else {
          some(Slot<2>{});
          some(Slot<3>{});
        }
      });
    };
    int g0 = gb, half = 0;
    auto next_run = [&]() __device__ {
      g0 += kRun;
      half = kRun * ROOM - half;
      asm("" : "+s"(half));
    };
    for (; g0 + kRun + 2 * (kSlots - 1) <= ge; next_run()) turn(Slot<1>{}, half, g0);
    for (; g0 < ge; next_run()) turn(Slot<0>{}, half, g0);
    wait_vm<0>();  // (nothing lands in the slots any more)
  }

  // The sums by way of LDS, each wave's own part of the slots (two 32 x 32
  // tiles at most at a time), so that a lane stores eight rows of a token: 16
  // bytes, whole runs of y.
  __syncthreads();
  constexpr int WIDTH = RT * 32, LD = WIDTH + 4;  // (a token's row of sums, shifted by four banks from the last)
  constexpr int PER = SLOT / (32 * LD * 4);  // waves of a slot
  static_assert(PER * kSlots >= WAVES, "room");
  float* const mine = reinterpret_cast<float*>(slot_of(wave / PER) + wave % PER * (32 * LD * 4));
  // (rows of y that begin on 16 bytes; of binary32 sums too)
  const bool wide = (a.N & 7) == 0 && (F32 || shares > 1 || (((uintptr_t)a.y & 15) == 0 && ((uintptr_t)a.res & 15) == 0));
  static_for<TT>([&](auto tc) __device__ {
    constexpr int t = decltype(tc)::value;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i) mine[(8 * (i >> 2) + 4 * lh + (i & 3)) * LD + 32 * r + li] = acc[r][t][i];
    wait_lgkm0();
    in_order();
    const int tok0 = (wt * TT + t) * 32, row0 = wr * RT * 32;
    for (int o = lane; o < 32 * WIDTH / 8; o += 64) {
      const int tok = o / (WIDTH / 8), c = o % (WIDTH / 8) * 8;
      if (tok0 + tok >= tokens || row0 + c >= rows) continue;
      const float* const v = mine + tok * LD + c;
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(v), hi = *reinterpret_cast<const f32x4_t*>(v + 4);
      const size_t at = (size_t)(t0 + tok0 + tok) * a.N + n0 + row0 + c;
      if (wide && (F32 || shares > 1)) {
        float* const to = a.part + (size_t)blockIdx.y * a.T * a.N + at;
        *reinterpret_cast<f32x4_t*>(to) = lo;
        *reinterpret_cast<f32x4_t*>(to + 4) = hi;
      } else if (wide) {
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = i < 4 ? lo[i] : hi[i - 4];
        if (a.res != nullptr) {
          const u32x4_t r = *reinterpret_cast<const u32x4_t*>(a.res + at);
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            s[i] = (float)((double)s[i] + (double)bf16_bits_to_f32(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu));
        }
        u32x4_t out;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          out[i] = (uint32_t)f32_to_bf16_rne(s[2 * i]) | ((uint32_t)f32_to_bf16_rne(s[2 * i + 1]) << 16);
        *reinterpret_cast<u32x4_t*>(a.y + at) = out;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (row0 + c + i >= rows) break;
          const float sum = i < 4 ? lo[i] : hi[i - 4];
          if (F32 || shares > 1) a.part[(size_t)blockIdx.y * a.T * a.N + at + i] = sum;
          else a.y[at + i] = finished((double)sum, a.res, at + i);
        }
      }
    }
    wait_lgkm0();
    in_order();
  });
}

// y = bf16(the shares' sums (+ residual)); a thread takes four outputs
__global__ void __launch_bounds__(256)
mx8_join_kernel(const float* part, const uint16_t* res, uint16_t* y, int64_t outputs, int shares) {
  const int64_t at = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x);
  if (at >= outputs) return;
  double v[4] = {};
  const int n = outputs - at < 4 ? (int)(outputs - at) : 4;
  if (n == 4 && (outputs & 3) == 0) {
    for (int s = 0; s < shares; ++s) {
      const f32x4_t p = *reinterpret_cast<const f32x4_t*>(part + (size_t)s * outputs + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += (double)p[i];
    }
  } else {
    for (int s = 0; s < shares; ++s)
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] += (double)part[(size_t)s * outputs + at + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) y[at + i] = finished(v[i], res, (size_t)(at + i));
}

constexpr int kCUs = 256;
constexpr int64_t kStreamTokens = 128;

// Tile shapes: rows and tokens of a workgroup, the time of a stage (us; alone
// on its CU, and two workgroups there if so many fit), of a workgroup's start
// and end.  Measured on 6144 x 5120 at 256 to 2048 tokens and 34816 x 5120 at
// 1024: 63 / 53 / 69 us at 1024 tokens, 61 / 49 / 39 at 512, 48 / 49 / 33 at
// 256; the shape for up to 32 tokens on 5120 x 17408 and 10240 x 8704 (at 23
// tokens 27 us streamed, 22 and 21 in six shares).
struct TileShape {
  int rows, tokens;
  double stage, both, ends;
};
constexpr TileShape kTiles[] = {{256, 128, 1.42, 0, 6.0}, {192, 128, 1.17, 0, 6.0}, {128, 64, 0.70, 0.84, 5.0},
                                {128, 32, 0.60, 1.1, 5.0}};
struct TilePlan {
  int shape, tiles_n, tiles_t, shares;
  double time;
};
TilePlan tile_plan(int64_t n, int64_t k, int64_t t) {
  TilePlan best{};
  best.time = -1.0;
  const int64_t stages = (k / 64 + 1) / 2;
  const int first = t <= 32 ? 3 : t <= 64 ? 2 : 0, last_shape = t <= 32 ? 3 : 2;
  for (int c = first; c <= last_shape; ++c) {
    const TileShape& s = kTiles[c];
    const int64_t tiles_n = (n + s.rows - 1) / s.rows, tiles_t = (t + s.tokens - 1) / s.tokens, tiles = tiles_n * tiles_t;
    for (int shares = 1; shares <= 8 && (shares == 1 || (4 * shares <= stages && tiles * shares <= 4 * kCUs)); ++shares) {
      const double length = (double)((stages + shares - 1) / shares);
      const int64_t all = tiles * shares, full = s.both > 0 ? all / (2 * kCUs) : 0, rest = all - full * 2 * kCUs;
      const int64_t rounds = (rest + kCUs - 1) / kCUs;
      // the rest: one workgroup a CU, or (two fit) two on some of them, where
      // HBM limits them if the weight is read once (1.1 us for 512 x 8 KiB)
      const double both = s.both < 1.1 / tiles_t ? 1.1 / tiles_t : s.both;
      const double last = s.both > 0 && rounds == 2 ? both : rounds * s.stage;
      const double time = length * (full * both + last) + (full + (s.both > 0 && rounds > 0 ? 1 : rounds)) * s.ends +
                          (shares > 1 ? 3.0 + (double)shares * n * t * (n % 8 == 0 ? 2e-6 : 6e-6) : 0.0);
      if (best.time < 0.0 || time < best.time) best = TilePlan{c, (int)tiles_n, (int)tiles_t, shares, time};
    }
  }
  return best;
}

// The kernel for up to kStreamTokens tokens: rows per workgroup (whole rounds
// of one workgroup per CU, the token ranges' together), and its time in the
// tiles' terms (us; a group of a wave measured on 6144 x 5120 at 32, 64 and 128
// tokens, past 32 rows on 12288 x 2048 and 16384 x 5120: at 23 tokens 9 and 22
// us, in tiles 12 and 19).  Tiles take over where its rounds are many: 20000 x 2048 at 100
// tokens 33 us here, 34816 x 2048 at 50 31.
struct StreamPlan {
  int bn, ranges;
  double time;
};
StreamPlan stream_plan(int64_t n, int64_t k, int64_t t) {
  StreamPlan p{};
  p.ranges = t <= 64 ? 1 : 2;
  const int64_t blocks = kCUs / p.ranges, rounds = (n + 64 * blocks - 1) / (64 * blocks);
  p.bn = (int)((n + blocks * rounds - 1) / (blocks * rounds));
  const double group = p.bn <= 32 ? (t <= 32 ? 0.65 : 1.08) : (t <= 32 ? 1.7 : 2.2);
  p.time = (double)rounds * (5.0 + group * (double)((k / 64 + kWaves - 1) / kWaves));
  return p;
}
bool takes_stream(int64_t n, int64_t k, int64_t t, const TilePlan& tiles) {
  return t <= kStreamTokens && stream_plan(n, k, t).time <= tiles.time;
}

template <int RT, int TT, int CH, int NX>
void launch_stream(const Mx8Kernel& k, int bn, int ranges, hipStream_t stream) {
  const unsigned blocks = (unsigned)((k.N + bn - 1) / bn);
  mx8_stream_kernel<RT, TT, CH, NX><<<dim3(ranges == 1 ? blocks : (blocks + 7) / 8 * 16), kThreads, 0, stream>>>(k, bn, ranges);
}

// One token: the bf16 product's single-token kernel on the same values where
// it takes one piece per lane (6144 x 5120 6.1 against 8.1 us of the few-token
// stream).
bool decode_takes(int64_t n, int64_t k, int64_t t) {
  DecodePlan p;
  return t == 1 && decode_plan(n, k, t, &p) && p.pl == 1;
}

}  // namespace

size_t mx8_workspace_bytes(int64_t n, int64_t k, int64_t t) {
  if (decode_takes(n, k, t) || few_mx8_ok(k, t)) return 0;
  const TilePlan p = tile_plan(n, k, t);
  return p.shares > 1 && !takes_stream(n, k, t, p) ? (size_t)p.shares * n * t * 4 : 0;
}

hipError_t launch_mx8(const Mx8Args& a, void* workspace, hipStream_t stream) {
  const Mx8Kernel k{static_cast<const uint8_t*>(a.x),      static_cast<const uint8_t*>(a.xs),
                    static_cast<const uint8_t*>(a.codes),  static_cast<const uint16_t*>(a.scales),
                    static_cast<const uint16_t*>(a.res),   static_cast<uint16_t*>(a.y),
                    static_cast<float*>(workspace),        (int)a.n,
                    (int)a.k,                              (int)a.t,
                    nullptr};
  if (decode_takes(a.n, a.k, a.t)) {
    GemvArgs g{a.x, a.codes, a.scales, a.y, a.n, a.k, a.t, a.res};
    g.xs = a.xs;
    return launch_decode(g, stream);
  }
  if (few_mx8_ok(a.k, a.t)) return launch_few_mx8(a, stream);
  const TilePlan p = tile_plan(a.n, a.k, a.t);
  if (takes_stream(a.n, a.k, a.t, p)) {
    const StreamPlan f = stream_plan(a.n, a.k, a.t);
    const bool two = a.t > 32;
    if (f.bn <= 32 && !two) launch_stream<1, 1, 4, 4>(k, f.bn, f.ranges, stream);
    else if (f.bn <= 32) launch_stream<1, 2, 4, 2>(k, f.bn, f.ranges, stream);
    else if (!two) launch_stream<2, 1, 2, 2>(k, f.bn, f.ranges, stream);
    else launch_stream<2, 2, 2, 2>(k, f.bn, f.ranges, stream);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(p.tiles_n * p.tiles_t), (unsigned)p.shares);
  if (p.shape == 0) mx8_tile_kernel<OpMx8, 4, 2, 2, 2><<<grid, 512, 0, stream>>>(k, p.tiles_n, p.tiles_t, p.shares);
  else if (p.shape == 1) mx8_tile_kernel<OpMx8, 2, 4, 3, 1><<<grid, 512, 0, stream>>>(k, p.tiles_n, p.tiles_t, p.shares);
  else if (p.shape == 2) mx8_tile_kernel<OpMx8, 2, 2, 2, 1><<<grid, 256, 0, stream>>>(k, p.tiles_n, p.tiles_t, p.shares);
  else mx8_tile_kernel<OpMx8, 4, 1, 1, 1><<<grid, 256, 0, stream>>>(k, p.tiles_n, p.tiles_t, p.shares);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.shares == 1) return e;
  const int64_t outputs = a.n * a.t;
  mx8_join_kernel<<<dim3((unsigned)((outputs + 1023) / 1024)), 256, 0, stream>>>(k.part, k.res, k.y, outputs, p.shares);
  return hipGetLastError();
}

hipError_t launch_tile_logits(const void* x_paired, const float* offsets, const void* codes, const void* scales,
                              float* logits, int64_t n, int64_t k, int64_t t, hipStream_t stream) {
  const Mx8Kernel m{static_cast<const uint8_t*>(x_paired), nullptr, static_cast<const uint8_t*>(codes),
                    static_cast<const uint16_t*>(scales), nullptr, nullptr, logits, (int)n, (int)k, (int)t, offsets};
  const int tiles_n = (int)((n + 255) / 256), tiles_t = (int)((t + 63) / 64);
  mx8_tile_kernel<OpBf16, 4, 2, 2, 1><<<dim3((unsigned)(tiles_n * tiles_t)), 512, 0, stream>>>(m, tiles_n, tiles_t, 1);
  return hipGetLastError();
}

}  // namespace q4lin
