// The LDS-tile kernel of the linear layers and their gradients (linear.h).
//
//  * A persistent grid goes over items (expert, tile of m, tile of c).  Which
//    rows an expert has is known on the device only: every workgroup counts the
//    experts' tiles from expert_offsets when it starts, and the grid depends on
//    the sizes alone.  Neighbouring items share an operand's tile; workgroups
//    are renumbered so that an XCD takes a run of them.
//  * A stage is KG sub-steps of 64 q of both operands, copied straight to LDS
//    while the stages before are multiplied, on from item to item without a
//    pause (8192 x 4096 x 2048 forward 133 -> 112 us, with the fragments' reads
//    and the copies between the multiplications).  Rows behind an expert's last,
//    and q behind the end, are outside the copy's buffer range and come as zeros.
//  * An expert's rows are cut into tiles of nearly equal height, and the blocks
//    of 16 rows go to the waves in turn, so that a tile of few rows costs few
//    multiplications on every wave.
//  * Sums are fp32; bias, activation, residual and the one rounding happen on
//    the accumulators.
//
// Measured (us; TFLOP/s), one session: 8192^3 forward 910 (1208), gradient of the
// rows 826 (1330), of the matrices 892 (1233); torch's library products of the same
// 814, 971 and 1086.  SQ_LDS_BANK_CONFLICT is 0 in all three.  The
// matrix units are busy half of the cycles at the 2.0 GHz that the card then runs
// at.  Copies of the kernel without the copies ran the first in 784 us, without the
// LDS reads in 826, without both in 645.  Few rows an expert are bound by the
// weights' way from HBM: 32 experts of 256 rows, 7168 x 2048, take 292 us forward
// (3.2 TB/s of weights), 221 where all experts share one matrix: a stage's copies
// are late by more than the stage and a half that LDS can hold ahead.  Loads ahead
// of them into L2 made it slower (358 us: they share the CU's address path), and so
// did other orders of q by column (306).
#pragma once

#include <type_traits>

#include "linear.h"
#include "linear_shape.h"

namespace moe {

constexpr int kXcds = 8;
constexpr int kSumStages = 64;   // whose sums of dy stay in fp32

// f(0), f(1) .. f(N - 1), each number a constant of its own type.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void repeat(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    repeat<N, I + 1>(f);
  }
}

// Workgroups are dealt to the XCDs in turn: renumber them so that each XCD has a run.
__device__ __forceinline__ int xcd_order(int b, int G) {
  const int xcd = b % kXcds, slot = b / kXcds;
  const int per = G / kXcds, extra = G % kXcds;
  return (xcd < extra ? xcd * (per + 1) : extra * (per + 1) + (xcd - extra) * per) + slot;
}

// Every vector-memory and LDS operation of this wave is done.
__device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(0x0070); }

// All but the youngest N vector-memory operations are, and every LDS one.
template <int N>
__device__ __forceinline__ void wait_but() {
  static_assert(N >= 0 && N < 64, "vmcnt is a 6-bit field");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (0x7 << 4) | ((N >> 4) << 14));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Rows [begin, end) of an expert.
struct RowRange {
  int begin, end;
};

// What every workgroup knows of the experts: the first item of each (at E their
// number) and its rows, kept inside [0, rows) so that a routing buffer that does
// not belong to these sizes cannot lead an access out of bounds.
struct Experts {
  int first[kMaxExperts + 1];
  RowRange rows[kMaxExperts + 1];
};

// Wave 0 fills it; `tiles` are an expert's items by its number of rows.
template <typename F>
__device__ __forceinline__ void count_items(const moe_host::LinearArgs& g, Experts* x, int lane, F&& tiles) {
  int n[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int e = lane * 8 + i;
    n[i] = 0;
    if (e < g.E) {
      RowRange r = {0, g.rows};
      if (g.expert_offsets) {
        r.begin = min(max(g.expert_offsets[e], 0), g.rows);
        r.end = min(max(g.expert_offsets[e + 1], r.begin), g.rows);
      }
      x->rows[e] = r;
      n[i] = tiles(r.end - r.begin);
    }
    sum += n[i];
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(before, o, 64);
    if (lane >= o) before += v;
  }
  before -= sum;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (lane * 8 + i <= g.E) x->first[lane * 8 + i] = before;
    before += n[i];
  }
}

// The expert of an item: the last whose first item is not behind it.
__device__ __forceinline__ int find_expert(const Experts* x, int E, int item, int lane) {
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    n += __popcll(__ballot(e < E && x->first[e] <= item));
  }
  return uniform(n - 1);
}

// Eight neighbouring values of a row from two blocks of accumulators: of blocks
// a and b (16 values each), a lane gets those at 8 (lane / 32) of a or, in odd
// groups of 16 lanes, of b.
__device__ __forceinline__ void pair_blocks(const f32x4& a, const f32x4& b, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(a[i]), __float_as_uint(b[i]), false, false);
    v[i] = __uint_as_float(s[0]);
    v[4 + i] = __uint_as_float(s[1]);
  }
}

// A 16-byte piece of a line that eight lanes store; `past`: past the caches (the
// empty statements keep the compiler from making one plain store of the two).
__device__ __forceinline__ void store_line(u32x4* to, const u32x4& q, bool past) {
  if (past) {
    __asm__ volatile("" ::: "memory");
    __builtin_nontemporal_store(q, to);
    __asm__ volatile("" ::: "memory");
  } else {
    *to = q;
  }
}

// The forward product's epilogue on eight neighbouring sums of a row, from
// column n of expert e's N on: bias, z, activation, residual, the one rounding.
template <typename Elem>
__device__ __forceinline__ void add8(const void* p, size_t at, float (&v)[8]) {
  typedef typename Elem::Row Row;
  float b[8];
  row_load<Row>(static_cast<const typename Row::elem*>(p) + at, b);
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] += b[i];
}
template <typename Elem>
__device__ __forceinline__ void store8(void* p, size_t at, const float (&v)[8], bool past = false) {
  typedef typename Elem::Row Row;
  store_line(reinterpret_cast<u32x4*>(static_cast<typename Row::elem*>(p) + at), Row::pack(v), past);
}
template <typename Elem>
__device__ __forceinline__ void forward_out(const moe_host::LinearArgs& g, int e, size_t row, int n, float (&v)[8]) {
  const size_t o = row * g.N + n;
  if (g.bias) add8<Elem>(g.bias, (size_t)e * g.N + n, v);
  if (g.z_out) store8<Elem>(g.z_out, o, v);
  if (g.act != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = activate(v[i], g.act);
  }
  if (g.residual) add8<Elem>(g.residual, o, v);
  store8<Elem>(g.out, o, v);
}
// SwiGLU: gate and up sums of output column n.
template <typename Elem>
__device__ __forceinline__ void forward_out(const moe_host::LinearArgs& g, int e, size_t row, int n, float (&gate)[8], float (&up)[8]) {
  const int M = g.N / 2;
  if (g.bias) {
    add8<Elem>(g.bias, (size_t)e * g.N + n, gate);
    add8<Elem>(g.bias, (size_t)e * g.N + M + n, up);
  }
  if (g.z_out) {
    store8<Elem>(g.z_out, row * g.N + n, gate);
    store8<Elem>(g.z_out, row * g.N + M + n, up);
  }
#pragma unroll
  for (int i = 0; i < 8; i++) up[i] *= silu(gate[i]);
  const size_t o = row * M + n;
  if (g.residual) add8<Elem>(g.residual, o, up);
  store8<Elem>(g.out, o, up);
}

// The epilogue of the gradient of the rows on eight sums of a row, from column k on.
template <typename Elem>
__device__ __forceinline__ void grad_x_out(const moe_host::LinearArgs& g, size_t row, int k, float (&v)[8]) {
  typedef typename Elem::Row Row;
  const typename Row::elem* const z = static_cast<const typename Row::elem*>(g.z_in);
  const size_t o = row * g.K + k;
  if (g.act == MOE_ACT_SWIGLU) {
    const size_t oz = 2 * row * g.K + k;
    float gate[8], up[8], y[8];
    row_load<Row>(z + oz, gate);
    row_load<Row>(z + oz + g.K, up);
#pragma unroll
    for (int i = 0; i < 8; i++) {
      y[i] = v[i] * silu(gate[i]);
      v[i] = v[i] * up[i] * silu_slope(gate[i]);
    }
    store8<Elem>(g.out, oz, v, g.stream_out);
    store8<Elem>(g.out, oz + g.K, y, g.stream_out);
    return;
  }
  if (g.act != MOE_ACT_NONE) {
    float at[8];
    row_load<Row>(z + o, at);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] *= act_slope(at[i], g.act);
  }
  store8<Elem>(g.out, o, v, g.stream_out);
}

// SUM: grad w with the bias's gradient.
template <typename Elem, LinearOp OP, typename S, bool SUM>
__global__ void __launch_bounds__(S::kThreads, S::kWavesASimd)
linear_tile_kernel(moe_host::LinearArgs g) {
  typedef typename Elem::Row Row;
  typedef typename Row::elem elem;
  constexpr bool TR = OP == kGradW, TC = OP != kForward;
  constexpr int BM = S::BM, BC = S::BC, KG = S::KG, WM = S::WM, WC = S::WC, MB = S::MB, CB = S::CB;
  // the operand of m in two parts, that of c in one, in this order in a sub-step
  typedef OperandTile<TR, S::kRows0> Part0;
  typedef OperandTile<TR, S::kRows1> Part1;
  typedef OperandTile<TC, BC> TileC;
  // copies of a wave; where the first part's do not go round, some copy nothing
  constexpr int N0 = (KG * Part0::kCopies + S::kWaves - 1) / S::kWaves, N1 = KG * Part1::kCopies / S::kWaves;
  constexpr int NC = KG * TileC::kCopies / S::kWaves;
  static_assert(KG * Part1::kCopies % S::kWaves == 0 && KG * TileC::kCopies % S::kWaves == 0, "whole copies a wave");
  static_assert(!TR || S::kRows0 == S::kRows1, "a lane's place in a transposed part goes by its width");
  constexpr bool UNEVEN = KG * Part0::kCopies % S::kWaves != 0;
  constexpr int NA = NC + N0, NALL = NA + N1;
  __shared__ __attribute__((aligned(1024))) char lds[S::kLds];
  Experts* const experts = reinterpret_cast<Experts*>(lds + S::kStage * S::kStages);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int kg = wave / (WM * WC), wm = wave / WC % WM, wc = wave % WC;
  const int lm = lane & 15;
  char* const scratch = lds + S::kLds - (S::kWaves - wave) * S::kScratch;   // the wave's own
  static_assert(!SUM || MB * 16 * 8 <= S::kScratch, "64-bit sums of the wave's columns fit");

  const bool gated = OP == kForward && g.act == MOE_ACT_SWIGLU;
  const int N = g.N, K = g.K;
  const int width_c = OP == kForward ? (gated ? N / 2 : N) : K;   // values of c of an output row
  const int step_c = gated ? BC / 2 : BC;                         // ... and of a tile
  const int tiles_c = (width_c + step_c - 1) / step_c;
  if (wave == 0) {
    count_items(g, experts, lane, [&](int rows) {
      return (OP == kGradW ? (N + BM - 1) / BM : (rows + BM - 1) / BM) * tiles_c;
    });
  }
  __syncthreads();
  const int total = uniform(experts->first[g.E]);

  // --- an item's tile
  struct Tile {
    int e, begin, rows;   // rows: of m (forward, grad x: of the tile; grad w: N, all of them)
    int m0, c0, tc;
    int Q, steps;
  };
  auto decode = [&](int item) {
    Tile t;
    t.e = find_expert(experts, g.E, item, lane);
    const int at = item - uniform(experts->first[t.e]);
    const int begin = uniform(experts->rows[t.e].begin), rows = uniform(experts->rows[t.e].end) - begin;
    const int len_m = OP == kGradW ? N : rows, tiles_m = (len_m + BM - 1) / BM;
    // tiles of m in groups of up to 8, c by c: a run of items is a block of both
    const int group = 8 * tiles_c, m_group = at / group;
    const int ms = min(8, tiles_m - m_group * 8), in_group = at - m_group * group;
    t.tc = in_group / ms;
    const int tm = m_group * 8 + in_group - t.tc * ms;
    // rows of a tile: an expert's share, in whole rounds of blocks over the waves
    const int height = OP == kGradW ? BM : min(BM, ((rows + tiles_m - 1) / tiles_m + 16 * WM - 1) / (16 * WM) * (16 * WM));
    t.m0 = tm * height;
    t.c0 = t.tc * step_c;
    t.begin = begin;
    t.rows = OP == kGradW ? N : min(rows, t.m0 + height);
    t.Q = OP == kForward ? K : OP == kGradX ? N : rows;
    t.steps = (t.Q + kStepQ * KG - 1) / (kStepQ * KG);
    return t;
  };

  // --- the copies run kStages stages ahead of the multiplications, on into the
  // next item: `from` is the tile they are in, from_step its next stage
  Tile from;
  int from_item, from_step;
  const char* baseR;
  const char* baseC;
  uint32_t bytesR, bytesC;        // of the operands that are contiguous in q
  uint32_t offR[N0 + N1], offC[NC];   // a lane's offset of each of its copies, but for the stage's
  const size_t ldR = OP == kForward ? (size_t)K * 2 : (size_t)N * 2, ldC = (size_t)K * 2;   // bytes a row in memory
  const int G = gridDim.x;

  // gate and up rows alternate, 16 by 16, so that a wave has both of a column
  auto weight_row = [&](int row) { return gated ? (row / 32) * 16 + row % 16 + ((row / 16) % 2) * (N / 2) : row; };

  // The copies go to item `item`, or to the first behind it that has any.
  auto enter = [&](int item) {
    from_step = 0;
    for (; item < total; item += G) {
      from = decode(item);
      if (from.steps > 0) break;
    }
    from_item = item;
    if (item >= total) {
      from.steps = 1 << 30;   // copies of nothing
      from.Q = 0;
      return;
    }
    bytesR = bytesC = 0;
    if constexpr (OP == kGradW) {
      baseR = static_cast<const char*>(g.rows_in) + (size_t)from.begin * ldR + from.m0 * 2;
      baseC = static_cast<const char*>(g.x) + (size_t)from.begin * ldC + from.c0 * 2;
    } else {
      baseR = static_cast<const char*>(g.rows_in) + (size_t)(from.begin + from.m0) * ldR;
      bytesR = (uint32_t)((from.rows - from.m0) * ldR);
      const char* w = static_cast<const char*>(g.w) + (size_t)from.e * N * ldC;
      if constexpr (OP == kForward) {
        baseC = w + (size_t)from.c0 * ldC;
        bytesC = (uint32_t)((size_t)(N - from.c0) * ldC);
      } else {
        baseC = w + (size_t)from.c0 * 2;
      }
    }
    baseR = uniform_ptr(baseR);
    baseC = uniform_ptr(baseC);
    repeat<N0 + N1>([&](auto at) {
      constexpr int j = at, part = j < N0 ? 0 : 1, first = part ? S::kRows0 : 0;
      typedef std::conditional_t<part == 0, Part0, Part1> Part;
      const int id = (part ? j - N0 : j) * S::kWaves + wave, sub = id / Part::kCopies, i = id % Part::kCopies;
      const int row = Part::copy_row(i, lane) + (TR ? sub * kStepQ : first);
      offR[j] = (uint32_t)(row * ldR) + Part::copy_byte(i, lane) + (TR ? first * 2 : sub * 128);
      if (UNEVEN && part == 0 && id >= KG * Part0::kCopies) offR[j] = kOutside;
    });
#pragma unroll
    for (int j = 0; j < NC; j++) {
      const int id = j * S::kWaves + wave, sub = id / TileC::kCopies, i = id % TileC::kCopies;
      const int row = TC ? TileC::copy_row(i, lane) + sub * kStepQ : weight_row(TileC::copy_row(i, lane));
      offC[j] = (uint32_t)(row * ldC) + TileC::copy_byte(i, lane) + (TC ? 0 : sub * 128);
    }
  };

  // The copies of the stage at from_step: where they come from, and copy j of the wave.
  struct Source {
    __amdgpu_buffer_rsrc_t r, c;
    int q2;
    char* stage;
  };
  auto source = [&](int slot) {
    Source s;
    const int q0 = from_step * kStepQ * KG, left = min(from.Q - q0, kStepQ * KG);
    const bool any = left > 0;
    // an operand that is contiguous in q moves along its rows; the other's range moves over them
    const char* const r = TR ? baseR + (size_t)q0 * ldR : baseR;
    const char* const c = TC ? baseC + (size_t)q0 * ldC : baseC;
    const uint32_t in_r = TR ? (uint32_t)(left * ldR) - from.m0 * 2 : bytesR, in_c = TC ? (uint32_t)(left * ldC) - from.c0 * 2 : bytesC;
    s.r = range_rsrc(uniform_ptr(r), uniform(any ? in_r : 0));
    s.c = range_rsrc(uniform_ptr(c), uniform(any ? in_c : 0));
    s.q2 = any ? q0 * 2 : 0;   // never more than the range, also where that is nothing
    s.stage = lds + slot * S::kStage;
    return s;
  };
  // copy j: those of c, then of the parts of m
  auto copy_one = [&](const Source& s, auto at) {
    constexpr int j = at, r = j - NC, part = r < N0 ? 0 : 1;
    if constexpr (j < NC) {
      const int id = j * S::kWaves + wave, sub = id / TileC::kCopies, i = id % TileC::kCopies;
      range_dma16(s.c, offC[j], TC ? 0 : s.q2, s.stage + sub * S::kSub + BM * kStepQ * 2 + i * 1024);
    } else {
      typedef std::conditional_t<part == 0, Part0, Part1> Part;
      const int id = (part ? r - N0 : r) * S::kWaves + wave, sub = id / Part::kCopies, i = id % Part::kCopies;
      char* to = s.stage + sub * S::kSub + part * (S::kRows0 * kStepQ * 2) + i * 1024;
      if (UNEVEN && part == 0 && id >= KG * Part0::kCopies) to = lds + S::kStage * S::kStages + S::kRanges;
      range_dma16(s.r, offR[r], TR ? 0 : s.q2, to);
    }
  };
  // Ahead of the copies at from_step: into the next item behind the last stage
  // (`ahead`; else to nothing), and no q behind the end at the last.
  auto advance = [&](bool ahead) {
    if (from_step == from.steps) enter(ahead ? from_item + G : total);
    if (from_step == from.steps - 1) {
      const int q2 = from_step * kStepQ * KG * 2;
      if constexpr (!TR) {
        repeat<N0 + N1>([&](auto at) {
          constexpr int j = at, part = j < N0 ? 0 : 1;
          typedef std::conditional_t<part == 0, Part0, Part1> Part;
          const int id = (part ? j - N0 : j) * S::kWaves + wave;
          if (q2 + id / Part::kCopies * 128 + Part::copy_byte(id % Part::kCopies, lane) >= from.Q * 2) offR[j] = kOutside;
        });
      }
      if constexpr (!TC) {
#pragma unroll
        for (int j = 0; j < NC; j++) {
          const int id = j * S::kWaves + wave;
          if (q2 + id / TileC::kCopies * 128 + TileC::copy_byte(id % TileC::kCopies, lane) >= from.Q * 2) offC[j] = kOutside;
        }
      }
    }
  };
  // The copies of the first stages of an item, and the wait for the first one's.
  auto start = [&](int item) {
    enter(item);
#pragma unroll
    for (int slot = 0; slot < S::kStages; slot++) {
      advance(KG == 1);
      const Source s = source(slot);
      repeat<NALL>([&](auto j) { copy_one(s, j); });
      from_step++;
    }
    wait_but<(S::kStages - 1) * NALL>();
    barrier_nofence();
  };

  int item = xcd_order(blockIdx.x, G);
  if (item >= total) return;
  start(item);
  int slot = 0;   // of the stage that is multiplied
  for (; item < total; item += G) {
    const Tile d = decode(item);
    f32x4 acc[CB][MB];
#pragma unroll
    for (int c = 0; c < CB; c++)
#pragma unroll
      for (int m = 0; m < MB; m++) acc[c][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // grad w with the bias's gradient: sums of dy over the rows.  Eight values of a
    // fragment are added in a tree; what kSumStages stages give is added in 64 bits to
    // the column's sum, which the first 16 lanes keep in the wave's scratch: 2^20
    // values of one sign, added one after another in fp32, came out 3.9e-3 of their sum off;
    // so no sum is off by more than 135 steps of 2^-24, for the same time (61 experts with
    // biases 43 us, 8192 x 7168 x 2048 266 against 268).
    const bool with_bias = SUM && d.tc == 0 && wc == 0;
    float colsum[MB];
    double* const sums = reinterpret_cast<double*>(scratch) + lm;
#pragma unroll
    for (int m = 0; m < MB; m++) {
      colsum[m] = 0.0f;
      if (SUM && with_bias && lane < 16) sums[m * 16] = 0.0;
    }
    auto fold = [&]() {
#pragma unroll
      for (int m = 0; m < MB; m++) {
        float v = colsum[m];
        v += __shfl_xor(v, 16, 64);
        v += __shfl_xor(v, 32, 64);
        if (lane < 16) sums[m * 16] += v;
        colsum[m] = 0.0f;
      }
    };

    // The stages.  A phase multiplies the blocks of c by up to half of the wave's
    // blocks of m for 32 q, and between its multiplications reads the next phase's
    // fragments and issues copies.  The order: first half of m, both 32 q; second
    // half, both 32 q.  At the second phase the waves meet: c and the first half
    // of m are read to the end, and take the copies of the stage kStages on; the
    // second half has come.  At the last phase they meet again: the second half
    // is free, and the next stage's c and first half have come.  So every copy has
    // one and a half stages' time at two stages (the ragged 32 experts 380 -> 353 us).
    // A tile without a second half meets once, and so do the gradients (first q of
    // both halves, then the second): with a transposed operand's reads, two for one,
    // the first two phases are short of LDS (8192^3 gradient of the matrices 1142 us
    // in the forward's order, 1061 in theirs).  (The reads ahead of an item's end are the next one's first,
    // read again there: one loop, whose accumulators stay in their registers.)
    // MA: blocks of m that have rows.
    constexpr bool SPLIT = OP == kForward && KG == 1 && MB > 4;
    constexpr auto q_of = [](int ph, int phases) { return phases == 2 ? ph : SPLIT ? ph % 2 : ph / 2; };
    constexpr auto m_of = [](int ph, int phases) { return phases == 2 ? 0 : SPLIT ? ph / 2 : ph % 2; };
    auto stages = [&](auto blocks) {
      constexpr int MA = blocks, M0 = MB <= 4 || MA <= S::MB0 ? MA : S::MB0, M1 = MA - M0, PHASES = M1 ? 4 : 2;
      u32x4 fa[2][CB], fb[2][M0];
      const uint32_t sub = lds0 + kg * S::kSub;
      const uint32_t placeR = sub + Part0::lane_place(wm, lane);
      const uint32_t placeC = sub + BM * kStepQ * 2 + TileC::lane_place(wc * CB, lane);
      uint32_t atR, atC;
      auto turn = [&]() {   // the places in the stage at `slot`
        atR = placeR + slot * S::kStage;
        atC = placeC + slot * S::kStage;
        __asm__ volatile("" : "+v"(atR), "+v"(atC));   // two registers, and not one for every block
      };
      // fragment r of the reads ahead of phase ph: the first of m, those of c, the others of m
      auto read_one = [&](auto phase, auto at) {
        constexpr int ph = phase, h = q_of(ph, PHASES), mh = m_of(ph, PHASES), r = at, nc = mh == 0 ? CB : 0;
        if constexpr (r == 0 || r > nc) {
          constexpr int m = (r == 0 ? 0 : r - nc) + (mh == 0 ? 0 : M0);
          fb[ph % 2][r == 0 ? 0 : r - nc] = m < S::MB0 ? Part0::fragment(atR, m * WM, h)
                                                       : Part1::fragment(atR + S::kRows0 * kStepQ * 2, (m - S::MB0) * WM, h);
        } else {
          fa[h][r - 1] = TileC::fragment(atC, r - 1, h);
        }
      };
      turn();
      repeat<M0 + CB>([&](auto r) { read_one(std::integral_constant<int, 0>{}, r); });
      for (int step = 0; step < d.steps; step++) {
        advance(KG == 1);
        Source s;
        repeat<PHASES>([&](auto phase) {
          constexpr int ph = phase, next = (ph + 1) % PHASES, h = q_of(ph, PHASES), mh = m_of(ph, PHASES);
          constexpr int first_m = mh == 0 ? 0 : M0, M = mh == 0 ? M0 : M1;
          constexpr bool last = ph == PHASES - 1, once = !SPLIT || M1 == 0, meet = last || (!once && ph == 1);
          constexpr int reads = (m_of(next, PHASES) == 0 ? M0 + CB : M1), mults = M * CB;
          constexpr int copies = !meet ? 0 : once ? NALL : last ? N1 : NA, first_copy = !once && last ? NA : 0;
          constexpr int extra = reads + copies;
          if constexpr (meet) {
            wait_but<once ? (S::kStages - 2) * NALL + (SPLIT ? N1 : 0) : (S::kStages - 1) * NALL>();
            barrier_nofence();
          }
          if constexpr (meet && (once || !last)) s = source(slot);
          if constexpr (last) {
            slot = slot == S::kStages - 1 ? 0 : slot + 1;
            turn();
            from_step++;
          }
          __builtin_amdgcn_sched_barrier(0);
          // as many of them after each multiplication as it takes, none behind the last one
          constexpr int each = (extra + mults - 1) / mults;
          repeat<mults>([&](auto at) {
            constexpr int i = at, m = i / CB, c = i % CB;
            acc[c][first_m + m] = Elem::mfma(fa[h][c], fb[ph % 2][m], acc[c][first_m + m]);
            repeat<each>([&](auto x) {
              constexpr int k = i * each + x;
              if constexpr (k < reads) read_one(std::integral_constant<int, next>{}, std::integral_constant<int, k>{});
              else if constexpr (k < extra) copy_one(s, std::integral_constant<int, first_copy + k - reads>{});
            });
            __builtin_amdgcn_sched_barrier(0);
          });
          if constexpr (SUM) {
            if (with_bias) {
#pragma unroll
              for (int m = 0; m < M; m++) {
                float v[8];
                Row::unpack(fb[ph % 2][m], v);
                colsum[first_m + m] += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
              }
            }
          }
        });
        if constexpr (SUM) {
          if (with_bias && step % kSumStages == kSumStages - 1) fold();
        }
      }
    };
    if (d.steps > 0) {
      if constexpr (OP == kGradW) {
        stages(std::integral_constant<int, MB>{});
      } else {
        const int active = (d.rows - d.m0 + 16 * WM - 1) / (16 * WM);
        repeat<MB>([&](auto i) {
          if (active == i + 1) stages(std::integral_constant<int, i + 1>{});
        });
      }
    }

    if (SUM && with_bias) fold();

    // --- the groups' sums, in ascending order, of blocks m in group m % KG
    if constexpr (KG > 1) {
      wait_all();
      barrier_nofence();   // no copy is on its way, the stages are free
      f32x4* const part = reinterpret_cast<f32x4*>(lds);
      const int w = wave % (WM * WC);
      static_assert(S::kWaves * MB * CB * 1024 <= S::kStage * S::kStages, "partial sums fit");
#pragma unroll
      for (int m = 0; m < MB; m++) {
#pragma unroll
        for (int c = 0; c < CB; c++) part[((wave * CB + c) * MB + m) * 64 + lane] = acc[c][m];
      }
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MB; m++) {
        if (m % KG != kg) continue;
#pragma unroll
        for (int c = 0; c < CB; c++) acc[c][m] = part[((w * CB + c) * MB + m) * 64 + lane];
        for (int k = 1; k < KG; k++) {
          const int other = k * WM * WC + w;
#pragma unroll
          for (int c = 0; c < CB; c++) acc[c][m] += part[((other * CB + c) * MB + m) * 64 + lane];
        }
        if (SUM && with_bias && lane < 16) {
          const double* const first = sums + m * 16 - kg * WM * WC * (S::kScratch / 8);   // group 0's
          double v = first[0];
          for (int k = 1; k < KG; k++) v += first[k * WM * WC * (S::kScratch / 8)];
          sums[m * 16] = v;   // of a block that no other group reads
        }
      }
      __syncthreads();
      start(item + G);   // the stages are the copies' again
      slot = 0;
    }

    // --- epilogue
    // A lane has row lane % 16 of every block of m, and of two blocks of c (pair_blocks)
    // the eight values from `place` on.
    const int place = 8 * (lane >> 5) + 16 * ((lane >> 4) & 1);
    if (SUM && with_bias && lane < 16) {   // ahead of the blocks, which take the scratch
#pragma unroll
      for (int m = 0; m < MB; m++) {
        const int n = d.m0 + (m * WM + wm) * 16 + lm;
        if ((KG > 1 && m % KG != kg) || n >= N) continue;
        const size_t at = (size_t)d.e * N + n;
        const double v = sums[m * 16];
        if (g.out_fp32) {
          float* const p = static_cast<float*>(g.dbias) + at;
          *p = (float)(g.accumulate ? *p + v : v);
        } else {
          elem* const p = static_cast<elem*>(g.dbias) + at;
          *p = Elem::round((float)(g.accumulate ? Elem::widen(*p) + v : v));
        }
      }
    }
#pragma unroll
    for (int m = 0; m < MB; m++) {
      if (KG > 1 && m % KG != kg) continue;
      const int r = d.m0 + (m * WM + wm) * 16 + lm;
      if constexpr (OP == kGradW) {
        // 16 rows of 128 bytes at a time, through LDS, so that eight lanes store a
        // whole line; piece p (16 bytes) of a row at place p ^ (row % 8)
        auto line_out = [&](int c1) {   // from column c1 of the wave's on
#pragma unroll
          for (int part = 0; part < 2; part++) {
            const int row = 8 * part + (lane >> 3), n = d.m0 + (m * WM + wm) * 16 + row;
            u32x4 q = *reinterpret_cast<const u32x4*>(scratch + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
            const int k = d.c0 + wc * CB * 16 + c1 + (lane & 7) * (g.out_fp32 ? 4 : 8);
            if (n >= N || k >= K) continue;
            const size_t at = ((size_t)d.e * N + n) * K + k;
            u32x4* const to = reinterpret_cast<u32x4*>(static_cast<char*>(g.out) + at * (g.out_fp32 ? 4 : 2));
            if (g.accumulate) q = __builtin_bit_cast(u32x4, *reinterpret_cast<const f32x4*>(to) + __builtin_bit_cast(f32x4, q));
            store_line(to, q, g.stream_out);
          }
        };
        if (g.out_fp32) {
#pragma unroll
          for (int c = 0; c < CB; c += 2) {
#pragma unroll
            for (int i = 0; i < 2; i++)
              *reinterpret_cast<f32x4*>(scratch + lm * 128 + (((4 * i + (lane >> 4)) ^ (lm & 7)) << 4)) = acc[c + i][m];
            line_out(c * 16);
          }
        } else if (!g.accumulate) {
#pragma unroll
          for (int c = 0; c < CB; c += 4) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const float v[4] = {acc[c + i][m][0], acc[c + i][m][1], acc[c + i][m][2], acc[c + i][m][3]};
              *reinterpret_cast<u32x2*>(scratch + lm * 128 + (((2 * i + (lane >> 5)) ^ (lm & 7)) << 4) + 8 * ((lane >> 4) & 1)) = Elem::pack4(v);
            }
            line_out(c * 16);
          }
        } else {
#pragma unroll
          for (int c = 0; c < CB; c += 2) {
            float v[8];
            pair_blocks(acc[c][m], acc[c + 1][m], v);
            const int k = d.c0 + (wc * CB + c) * 16 + place;
            if (r >= N || k >= K) continue;
            const size_t at = ((size_t)d.e * N + r) * K + k;
            add8<Elem>(g.out, at, v);
            store8<Elem>(g.out, at, v);
          }
        }
      } else if constexpr (OP == kForward) {
        const size_t row = (size_t)d.begin + r;
        if (gated) {
          // blocks of gate and up values in turn: two of each give eight columns
#pragma unroll
          for (int c = 0; c + 3 < CB; c += 4) {
            float gate[8], up[8];
            pair_blocks(acc[c][m], acc[c + 2][m], gate);
            pair_blocks(acc[c + 1][m], acc[c + 3][m], up);
            const int n = d.c0 + (wc * CB + c) * 8 + place;
            if (r < d.rows && n < width_c) forward_out<Elem>(g, d.e, row, n, gate, up);
          }
        } else {
#pragma unroll
          for (int c = 0; c < CB; c += 2) {
            float v[8];
            pair_blocks(acc[c][m], acc[c + 1][m], v);
            const int n = d.c0 + (wc * CB + c) * 16 + place;
            if (r < d.rows && n < width_c) forward_out<Elem>(g, d.e, row, n, v);
          }
        }
      } else {
        // eight rows of 64 values at a time, through LDS, so that eight lanes have a row
        // (a line of the output); the pieces of 16 bytes change places by 2 (row % 8)
        static_assert(CB == 4, "a wave's columns are 64");
#pragma unroll
        for (int half = 0; half < 2; half++) {
          if ((lm >> 3) == half) {
#pragma unroll
            for (int c = 0; c < CB; c++)
              *reinterpret_cast<f32x4*>(scratch + (lm & 7) * 256 + (((4 * c + (lane >> 4)) ^ (2 * (lm & 7))) << 4)) = acc[c][m];
          }
          const int r8 = lane >> 3, rh = d.m0 + (m * WM + wm) * 16 + 8 * half + r8;
          const int n = d.c0 + wc * CB * 16 + 8 * (lane & 7);
          const char* const from_row = scratch + r8 * 256 + (((2 * (lane & 7)) ^ (2 * r8)) << 4);
          const f32x4 v0 = *reinterpret_cast<const f32x4*>(from_row), v1 = *reinterpret_cast<const f32x4*>(from_row + 16);
          if (rh >= d.rows || n >= width_c) continue;
          float v[8] = {v0[0], v0[1], v0[2], v0[3], v1[0], v1[1], v1[2], v1[3]};
          grad_x_out<Elem>(g, (size_t)d.begin + rh, n, v);
        }
      }
    }
  }
  wait_all();   // no copy may reach LDS that is another workgroup's by then
}

// Whether what a call reads and writes is more than the 256 MiB that the last
// cache holds: its outputs, in whole lines, are then stored past the caches, which
// keep the operands.  Measured (us, plain and past): 8 experts of 512 rows, 28672 x
// 4096, fp32 gradient of the matrices 1739 and 1492, 8192^3 gradient of the rows
// 1006 and 927; with 141 MB in all, 61 experts of 76 rows, 1000 x 520, 33 and 70.
static inline bool past_caches(size_t bytes) { return bytes > (size_t)256 << 20; }

// A persistent grid for at most `items` items.
template <typename Elem, LinearOp OP, typename S, bool SUM = false>
static hipError_t launch_linear_tile(const moe_host::LinearArgs& a, long items, int cus, hipStream_t s) {
  const long most = (long)cus * S::kOccupancy, grid = items < most ? items : most;
  if (grid <= 0) return hipSuccess;
  hipLaunchKernelGGL((linear_tile_kernel<Elem, OP, S, SUM>), dim3((unsigned)grid), dim3(S::kThreads), 0, s, a);
  return hipGetLastError();
}

// Tiles of BM rows that `rows` rows of E experts can need at most.
static inline long max_tiles(const moe_host::LinearArgs& a, int BM) {
  return a.expert_offsets ? a.rows / BM + (a.rows < a.E ? a.rows : a.E) : (a.rows + BM - 1) / BM;
}

inline LinearSizes sizes_of(const moe_host::LinearArgs& a) {
  return {a.rows, a.E, a.expert_offsets != nullptr, a.N, a.K, a.act == MOE_ACT_SWIGLU};
}

typedef LinearShape<256, 256, 2, 4, 1, 2> Tile256;
typedef LinearShape<128, 128, 2, 2, 1, 2> Tile128;
typedef LinearShape<64, 64, 2, 1, 2, 2> Pair64;
typedef LinearShape<64, 64, 2, 1, 4, 2> Quad64;
typedef LinearShape<288, 256, 2, 4, 1, 2> Tile288;

template <typename S>
constexpr bool is_cost_of(LinearTile t) {
  const ShapeCost& c = kShapeCosts[t];
  return S::BM == c.BM && S::BC == c.BC && S::KG * kStepQ == c.q && S::kOccupancy == c.occupancy;
}
static_assert(is_cost_of<Tile256>(kTile256) && is_cost_of<Tile128>(kTile128) && is_cost_of<Pair64>(kPair64) &&
                  is_cost_of<Quad64>(kQuad64) && is_cost_of<Tile288>(kTile288),
              "the shapes that the costs are of");

// f(shape) of a tile; ROWS: m are rows.
template <bool ROWS, typename F>
static hipError_t with_shape(LinearTile tile, F&& f) {
  switch (tile) {
    case kTile256: return f(Tile256{});
    case kTile128: return f(Tile128{});
    case kPair64: return f(Pair64{});
    case kQuad64: return f(Quad64{});
    default: break;
  }
  if constexpr (ROWS) return f(Tile288{});
  else return hipErrorInvalidValue;
}

}  // namespace moe
