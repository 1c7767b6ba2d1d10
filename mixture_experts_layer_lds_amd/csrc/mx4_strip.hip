// MXFP4 grouped GEMM for a few dozen to a few hundred rows per expert: token
// rows staged in LDS, weights streamed to registers.
//
// Same pipeline role as strip_gemm.hip (HPC-Ops x SGLang blog, section
// "MoE": gate-up reads tokens through the route index with no separate
// gather; a persistent grid consumes the per-tile task map), built for MXFP4
// blocks (mx4.h):
//
//  * One workgroup of 8 waves per CU.  Work item = (task tile of 16 MB rows,
//    strip of 256 weight rows).  A wave owns two 16-row weight blocks:
//    gate-up, half of 32 gate rows and the matching half of 32 up rows; down,
//    32 output columns.
//  * A stage is GS groups of G units of K.  Its token rows and their scale
//    codes go to one of two LDS slots by direct buffer->LDS copies spread over
//    the waves, while the other slot is multiplied.  (Buffer copies, not
//    global ones: with those the compiler loses count of the vector-memory
//    queue and waits for all of it at the first fragment of every stage.)
//  * The wave's weights of a unit are loaded into the registers that the
//    multiplication of the same unit has just left, D stages on: 8 KiB a wave
//    and stage at four units, 64 KiB a CU, run straight across work items.
//    Two stages instead of one: DeepSeek-V3-shaped gate-up, T = 4096, 920 ->
//    868 us; Mixtral-shaped T = 512 136 -> 126 us.
//  * Row blocks past the tile are copied and read but not multiplied.
//  * Gate-up epilogue: 32 columns of h are one MXFP4 block a row, held by two
//    neighbouring waves; they exchange the rows' largest magnitudes through
//    LDS and write codes and scale codes in the blocks that the down GEMM
//    copies as contiguous chunks.  Down writes fp32 rows, 32 bytes a lane.
//
// A wave's copies of a stage come before its weight loads of the same stage,
// whose number is fixed, so the wait at the head of a stage is an exact count.
//
// Measured (us by events, passes in a row; TB/s of weights with their scale
// codes): DeepSeek-V3-shaped gate-up / down at T = 1024 610 (6.6) / 386 (5.2),
// at 4096 829 (4.8) / 577 (3.5; with the fp32 rows 5.1, the rate of a large
// copy); Mixtral-8x7B-shaped T = 2048 312 / 173, 3.1 and 2.8 PFLOP/s (303 to 317
// and 170 to 175 from session to session).  Few rows an expert run at the rate
// of the weight stream.  At many, no one part bounds the gate-up.  Copies of the
// kernel with parts left out took, in one session:
//                          DeepSeek-V3 T = 4096    Mixtral-8x7B T = 2048
//   whole                          829                     312
//   no multiplications             767                     237
//   no token copies                750                     233
//   no weight loads                496                     254
//   no epilogue                    766                     260
//   neither load                   428                     220
//   loads, products left out       246                     141
//   all four left out              171                      79
// The first is nearest to its weights (4.0 GB, 568 us at the rate of a large
// read), which the token copies share the CU's queue with; the second takes
// 220 of 312 without a load, 116 of them the MFMA's own time.  (Four waves of
// twice the weight rows, half the LDS reads, ran in the same time.)
#include "lds_dma.h"
#include "mx4_epilogue.h"

namespace moe {

constexpr int kMx4Waves = 8;
// Whether the registers hold two stages of weights beside the accumulators of
// MB row blocks (a stage of one group of four units takes the fewest others).
constexpr int mx4_stages_ahead(int MB, int G, int GS) { return MB * G * GS <= (G == 4 ? 40 : 32) ? 2 : 1; }

// Direct buffer->LDS copies (a lane's N bytes at base + off + soff, to its
// place after dst).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const char* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, 0xffffffffu, 0x00027000);
}
__device__ __forceinline__ void buf_dma16(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, off, soff, 0, 0);
}
__device__ __forceinline__ void buf_dma4(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 4, off, soff, 0, 0);
}

template <int MB, int G, int GS>
struct Mx4Stage {
  static constexpr int U = G * GS;                                   // units
  static constexpr int NA = (MB * U + kMx4Waves - 1) / kMx4Waves;    // token chunks a wave copies
  static constexpr int NS = (MB * GS + kMx4Waves - 1) / kMx4Waves;   // scale chunks
  static constexpr int NW = 2 * U + 2 * GS;                          // weight loads of a wave
  static constexpr int kTokens = MB * U * 1024;
  static constexpr int kSlot = kTokens + MB * GS * 256;
  static constexpr int kRows = MB * 16;
  static constexpr int kPairs = (kRows + 63) / 64 * 64;              // whole copies
};

// Item `item` of the grid's order: a task tile (task ti, rows row_begin ..
// + rows of `expert`) and a strip nt of its expert's weights.  An expert's
// tiles take a strip one after another, so that its weights, once in L2,
// serve them all; the strips of one tile stand side by side where an expert
// has one tile, and meet its token rows in L2.
// With `split` K slices an item is one slice of them, stages k0 on, the
// slices of a strip side by side.
struct Mx4Place {
  int ti, nt, expert, row_begin, rows;
  int slice, k0;
};

template <int MB>
__device__ __forceinline__ Mx4Place mx4_place(const moe_host::Mx4Args& g, int item, int n_strips, int nk) {
  Mx4Place p;
  p.slice = item % g.split;
  p.k0 = p.slice * nk;
  item /= g.split;
  p.ti = item / n_strips;
  p.nt = item - p.ti * n_strips;
  const moe_task_t t = load_task_scalar(g.tasks + p.ti);
  p.expert = t.expert;
  p.row_begin = t.row_begin;
  p.rows = t.rows;
  const int begin = load1_scalar(g.expert_offsets + t.expert), end = load1_scalar(g.expert_offsets + t.expert + 1);
  const int tiles = (end - begin + 16 * MB - 1) / (16 * MB);
  if (tiles > 1) {
    const int first = p.ti - (t.row_begin - begin) / (16 * MB), local = item - first * n_strips;
    const int j = local % tiles;
    p.nt = local / tiles;
    p.ti = first + j;
    p.row_begin = begin + 16 * MB * j;
    p.rows = min(16 * MB, end - p.row_begin);
  }
  return p;
}

template <int MB, int G, int GS>
struct Mx4Item {
  using St = Mx4Stage<MB, G, GS>;
  Mx4Place at;
  const char* abase;               // of the offsets a[] (and, down, s[]): uniform
  uint32_t a[St::NA], s[St::NS];   // this lane's byte offsets
};

// The item's token sources.  pairs: the pair index of each of the tile's rows
// (LDS; gate-up only); inv_topk: 2^31 / topk rounded up (2 pair inv_topk / 2^32
// is less than pair / topk + 2^-15: the quotient, as pair < 2^16, topk <= 16).
template <int MB, int G, int GS, bool GATEUP>
__device__ __forceinline__ Mx4Item<MB, G, GS> mx4_item(const moe_host::Mx4Args& g, const Mx4Place& at, const int* pairs,
                                                       uint32_t inv_topk, int wave, int lane) {
  using St = Mx4Stage<MB, G, GS>;
  Mx4Item<MB, G, GS> it;
  const uint32_t block_bytes = (uint32_t)(g.K / 128) * kMx4Unit;
  it.at = at;
  // x codes take at most 2^31 bytes (T H / 2), a task's blocks of h far less:
  // 32-bit offsets from a uniform base
  it.abase = static_cast<const char*>(g.a) + (GATEUP ? 0 : (size_t)at.ti * MB * block_bytes);
  // rows past the tile re-read its last row (gate-up; a whole block of them
  // one line) or its first block (down): valid addresses, never stored
#pragma unroll
  for (int i = 0; i < St::NA; i++) {
    const int c = (wave + kMx4Waves * i) % (MB * St::U);   // chunk: row block c / U, unit c % U
    const int rb = c / St::U, u = c % St::U;
    if constexpr (GATEUP) {
      const uint32_t tok = __umulhi(2u * (uint32_t)pairs[rb * 16 + tok_copy_row(lane)], inv_topk);
      it.a[i] = tok * (uint32_t)(g.K / 2) + u * 64 + 16 * tok_copy_piece(lane);
    } else {
      it.a[i] = (rb * 16 < at.rows ? rb : 0) * block_bytes + u / G * (G * kMx4Unit) + u % G * 1024 + 16 * lane;
    }
  }
#pragma unroll
  for (int i = 0; i < St::NS; i++) {
    const int c = (wave + kMx4Waves * i) % (MB * GS);      // row block c / GS, group c % GS
    const int rb = c / GS, j = c % GS;
    if constexpr (GATEUP) {
      const uint32_t tok = __umulhi(2u * (uint32_t)pairs[rb * 16 + (lane & 15)], inv_topk);
      it.s[i] = tok * (uint32_t)(g.K / 32) + 4 * G * j + (((lane >> 4) * G) & ~3);
    } else {
      it.s[i] = (rb * 16 < at.rows ? rb : 0) * block_bytes + j * (G * kMx4Unit) + G * 1024 + ((lane * G) & ~3);
    }
  }
  return it;
}

// The wave's two 16-row weight blocks in strip nt.
struct Mx4Blocks {
  int out;      // gate-up: first block of the 32 columns of h that a pair of waves forms; down: the first block
  int k0;       // the item's first stage
  bool store;   // they exist (down: H may end inside a strip; else block 0 is read and nothing stored)
  const char *b0, *b1;
};

template <bool GATEUP>
__device__ __forceinline__ Mx4Blocks mx4_blocks(const moe_host::Mx4Args& g, const Mx4Place& at, int wave) {
  Mx4Blocks r;
  r.k0 = at.k0;
  const size_t block_bytes = (size_t)(g.K / 128) * kMx4Unit;
  int b0, b1;
  if constexpr (GATEUP) {
    r.out = 8 * at.nt + (wave & ~1);   // 128 columns of h a strip, 32 a pair of waves
    r.store = true;
    b0 = r.out + (wave & 1);
    b1 = b0 + g.N_out / 16;
  } else {
    r.out = 16 * at.nt + 2 * wave;
    r.store = r.out < g.N_out / 16;
    b0 = r.store ? r.out : 0;
    b1 = b0 + 1;
  }
  const char* B = static_cast<const char*>(g.b) + (size_t)at.expert * (g.w_rows / 16) * block_bytes;
  r.b0 = B + (size_t)b0 * block_bytes;
  r.b1 = B + (size_t)b1 * block_bytes;
  return r;
}

template <int MB, int G, int GS, int D, bool GATEUP>
__global__ void __launch_bounds__(kMx4Waves * 64, 1)
mx4_strip_kernel(moe_host::Mx4Args g) {
  using St = Mx4Stage<MB, G, GS>;
  using It = Mx4Item<MB, G, GS>;
  constexpr int U = St::U;
  constexpr int CH = 2, NC = MB / CH;   // row blocks multiplied at a time, and how many times
  static_assert(MB % CH == 0, "whole chunks of row blocks");
  static_assert(D == 1 || D == 2, "weights one or two stages ahead (a stage of either slot has its own)");
  static_assert(St::NA + St::NS + St::NW < 64, "vmcnt range");
  // The two slots are two variables, and a stage is compiled for each: the
  // compiler then knows that a fragment read from one does not have to wait
  // for copies into the other (with one array it waits, at the head of every
  // stage, for the copies that the stage has just issued).
  __shared__ __attribute__((aligned(1024))) char slot0[St::kSlot];
  __shared__ __attribute__((aligned(1024))) char slot1[St::kSlot];
  __shared__ uint32_t amax[kMx4Waves * St::kRows];
  __shared__ int pairs[3 * St::kPairs];   // the pair indices of three items
  const int lane = threadIdx.x & 63;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int num_tasks = min(g.header[kHdrNumTasks], g.max_tasks);
  const int n_strips = GATEUP ? g.N_out / 128 : (g.N_out + 255) / 256;
  // tasks < 65536 / 64 + 512, strips <= 512, slices <= 8: under 2^23
  const int total = num_tasks * n_strips * g.split;
  const int nk = g.K / 128 / U / g.split;             // stages per item
  const int units2 = g.N_out / 128, G2 = units2 % 4 == 0 ? 4 : (units2 % 2 == 0 ? 2 : 1);

  // XCD-aware numbering: each XCD takes a contiguous run of items, so the
  // strips of one task tile share its token rows through one L2.
  const int gs = gridDim.x;
  const int xcd = blockIdx.x % 8, xslot = blockIdx.x / 8;
  const int per_xcd = gs / 8, extra = gs % 8;
  const int vid = (xcd < extra ? xcd * (per_xcd + 1) : extra * (per_xcd + 1) + (xcd - extra) * per_xcd) + xslot;
  if (vid >= total) return;
  const int n_items = (total - vid + gs - 1) / gs;

  const int aoff = GATEUP ? tok_frag_off(lane) : 16 * lane;
  const int ash = GATEUP ? 8 * ((lgrp * G) & 3) : 8 * ((lane * G) & 3);
  const int bsh = 8 * ((lane * G) & 3);
  const uint32_t wlane = 16 * lane, slane = G * 1024 + ((lane * G) & ~3);

  // Weights read by one tile each pass by the caches (non-temporal); where an
  // expert has several tiles the later ones find them in L2 (ordinary loads).
  auto body = [&](auto nt_tag) {
    constexpr bool NT_B = decltype(nt_tag)::value;
    // The sources of an item are formed one item ahead of its first stage,
    // from pair indices that were copied to LDS an item earlier still (three
    // places, so that no wave overwrites what another still reads).  Past the
    // last item: the last one again, its first stage loaded and never used.
    const uint32_t inv_topk = ((1u << 31) + g.topk - 1) / g.topk;
    auto place = [&](int i) __attribute__((always_inline)) { return mx4_place<MB>(g, vid + min(i, n_items - 1) * gs, n_strips, nk); };
    auto copy_pairs = [&](const Mx4Place& p, int i) __attribute__((always_inline)) {
      if constexpr (GATEUP) {
        const auto r = rows_rsrc(reinterpret_cast<const char*>(g.sorted_pairs + p.row_begin));
#pragma unroll
        for (int r0 = 0; r0 < St::kRows; r0 += 64)   // every wave all of them: no branch round a copy
          buf_dma4(r, 4 * min(r0 + lane, p.rows - 1), 0, reinterpret_cast<char*>(pairs + i % 3 * St::kPairs + r0));
      }
    };
    auto sources = [&](const Mx4Place& p, int i) __attribute__((always_inline)) {
      return mx4_item<MB, G, GS, GATEUP>(g, p, pairs + i % 3 * St::kPairs, inv_topk, wave, lane);
    };
    const Mx4Place place0 = place(0), place1 = place(1);
    Mx4Place ahead = place(2);   // the item whose pairs are on their way
    copy_pairs(place0, 0);
    copy_pairs(place1, 1);
    copy_pairs(ahead, 2);
    wait_vm<0>();
    barrier_nofence();
    It cur = sources(place0, 0), nxt = sources(place1, 1);

    auto issue_tokens = [&](bool in_cur, int kt, char* slot) __attribute__((always_inline)) {
      kt += in_cur ? cur.at.k0 : nxt.at.k0;
      const int at = kt * (GATEUP ? U * 64 : U * kMx4Unit);
      const auto ra = rows_rsrc(in_cur ? cur.abase : nxt.abase);
      const auto rs = GATEUP ? rows_rsrc(reinterpret_cast<const char*>(g.a_sc)) : ra;
#pragma unroll
      for (int i = 0; i < St::NA; i++)
        buf_dma16(ra, in_cur ? cur.a[i] : nxt.a[i], at, slot + ((wave + kMx4Waves * i) % (MB * U)) * 1024);
#pragma unroll
      for (int i = 0; i < St::NS; i++)
        buf_dma4(rs, in_cur ? cur.s[i] : nxt.s[i], GATEUP ? kt * (4 * U) : at,
                 slot + St::kTokens + ((wave + kMx4Waves * i) % (MB * GS)) * 256);
    };

    // Weights run D stages ahead of the multiplication, over the items by
    // themselves: stage wk of item wi is the next to be loaded.
    Mx4Blocks wb = mx4_blocks<GATEUP>(g, place0, wave);
    int wk = 0, wi = 0;
    auto next_weights = [&]() __attribute__((always_inline)) {
      if (++wk == nk) {
        wk = 0;
        if (++wi < n_items) wb = mx4_blocks<GATEUP>(g, place(wi), wave);
      }
    };
    u32x4 w[D][U][2];
    uint32_t sw[GS][2], swn[D][GS][2];   // scale codes of this stage, and those on their way
    auto load_unit = [&](u32x4 (&to)[2], const char* b0, const char* b1, int u) __attribute__((always_inline)) {
      const int at = u / G * (G * kMx4Unit) + u % G * 1024;
      const u32x4* p0 = reinterpret_cast<const u32x4*>(b0 + at + wlane);
      const u32x4* p1 = reinterpret_cast<const u32x4*>(b1 + at + wlane);
      to[0] = NT_B ? __builtin_nontemporal_load(p0) : *p0;
      to[1] = NT_B ? __builtin_nontemporal_load(p1) : *p1;
    };
    auto load_scales = [&](uint32_t (&to)[GS][2], const char* b0, const char* b1) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < GS; j++) {
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(b0 + j * (G * kMx4Unit) + slane);
        const uint32_t* q1 = reinterpret_cast<const uint32_t*>(b1 + j * (G * kMx4Unit) + slane);
        to[j][0] = NT_B ? __builtin_nontemporal_load(q0) : *q0;
        to[j][1] = NT_B ? __builtin_nontemporal_load(q1) : *q1;
      }
    };
    // The empty asm statements keep the copies ahead of the weights in issue
    // order, which the vmcnt count relies on.
    issue_tokens(true, 0, slot0);
    __asm__ volatile("" ::: "memory");
#pragma unroll
    for (int d = 0; d < D; d++) {
      const size_t at = (size_t)(wb.k0 + wk) * (U * kMx4Unit);
      load_scales(swn[d], wb.b0 + at, wb.b1 + at);
#pragma unroll
      for (int u = 0; u < U; u++) load_unit(w[d][u], wb.b0 + at, wb.b1 + at, u);
      __asm__ volatile("" ::: "memory");
      next_weights();
    }

    f32x4 acc[MB][2];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int m = 0; m < MB; m++) acc[m][0] = acc[m][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    clear();
    int ii = 0;

    // One stage (kt of the item) from slot sb, the next one's copies into `next`; w_, swn_: the
    // stage's weights, replaced by those of D stages on.
    auto stage = [&](int kt, const char* sb, char* next, u32x4 (&w_)[U][2], uint32_t (&swn_)[GS][2]) __attribute__((always_inline)) {
        // the stage's copies have landed in this wave (only its weights were
        // issued after them), then in every wave
        __asm__ volatile("" ::: "memory");
        wait_vm<St::NW>();
        barrier_nofence();
        // the next stage into the slot that every wave had read before the barrier
        const bool in_cur = kt + 1 < nk;
        issue_tokens(in_cur, in_cur ? kt + 1 : 0, next);
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const char* b0 = wb.b0 + (size_t)(wb.k0 + wk) * (U * kMx4Unit);
        const char* b1 = wb.b1 + (size_t)(wb.k0 + wk) * (U * kMx4Unit);
#pragma unroll
        for (int j = 0; j < GS; j++)
#pragma unroll
          for (int q = 0; q < 2; q++) sw[j][q] = swn_[j][q] >> bsh;
        load_scales(swn_, b0, b1);
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(sb + St::kTokens);
        // CH row blocks at a time, their fragments read while the previous
        // ones are multiplied; the scheduling barriers keep the compiler from
        // reading more of them ahead than there are registers for.  Blocks past
        // the tile are read but not multiplied.
        const int chunks = (cur.at.rows + 16 * CH - 1) / (16 * CH);
        u32x4 t[2][CH];
        uint32_t st[MB];
        auto read = [&](u32x4 (&to)[CH], int step) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < CH; i++)
            to[i] = *reinterpret_cast<const u32x4*>(sb + ((step % NC * CH + i) * U + step / NC) * 1024 + aoff);
        };
        read(t[0], 0);
#pragma unroll
        for (int j = 0; j < GS; j++) {
#pragma unroll
          for (int m = 0; m < MB; m++) st[m] = sc[64 * (m * GS + j) + lane] >> ash;
          mx4_units<G>([&](auto uu) {
            constexpr int V = decltype(uu)::value;
            const int un = j * G + V;
            // (uses outside the branch below, so that the waits for the loads stand
            // here and count exactly; under a branch the compiler waits for
            // everything in flight)
            __asm__ volatile("" : "+v"(w_[un][0]), "+v"(w_[un][1]));
#pragma unroll
            for (int mc = 0; mc < NC; mc++) {
              const int step = un * NC + mc;
              if (step + 1 < U * NC) read(t[(step + 1) & 1], step + 1);
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int i = 0; i < CH; i++) __asm__ volatile("" : "+v"(t[step & 1][i]));
              if (mc < chunks) {
#pragma unroll
                for (int i = 0; i < CH; i++) {
                  mfma_mx4<V>(acc[CH * mc + i][0], w_[un][0], t[step & 1][i], sw[j][0], st[CH * mc + i]);
                  mfma_mx4<V>(acc[CH * mc + i][1], w_[un][1], t[step & 1][i], sw[j][1], st[CH * mc + i]);
                }
              }
              __builtin_amdgcn_sched_barrier(0);
            }
            load_unit(w_[un], b0, b1, un);
            __builtin_amdgcn_sched_barrier(0);
          });
        }
        next_weights();
      };
    // The item's results, and the next item's turn.
    auto finish = [&]() __attribute__((always_inline)) {
      const Mx4Blocks blk = mx4_blocks<GATEUP>(g, cur.at, wave);
      if constexpr (GATEUP) {
        // h = SiLU(gate) * up in place of the gate sums; the row's largest
        // magnitude over this wave's 16 columns to LDS
#pragma unroll
        for (int m = 0; m < MB; m++) {
          if (16 * m >= cur.at.rows) break;
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            acc[m][0][i] = mx4_silu(acc[m][0][i]) * acc[m][1][i];
            mx = max(mx, abs_bits(acc[m][0][i]));
          }
          mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
          mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
          if (lgrp == 0) amax[(wave * MB + m) * 16 + lrow] = mx;
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the writes are in LDS
        barrier_nofence();
        // (the next write of `amax` comes after the barriers of the next item's stages)
        const Mx4Out o = mx4_out(g.c, (size_t)cur.at.ti * MB, blk.out / 2, units2, G2);
        // whole blocks, also of rows past the tile's last one: their places are
        // this task's and never read
        int row = lrow;   // (opaque: the places below formed here, not kept in registers through the stages)
        __asm__ volatile("" : "+v"(row));
#pragma unroll
        for (int m = 0; m < MB; m++) {
          if (16 * m >= cur.at.rows) break;
          const uint32_t mx = max(amax[(wave * MB + m) * 16 + lrow], amax[((wave ^ 1) * MB + m) * 16 + lrow]);
          const uint32_t code = mx4_scale_code(mx);
          const uint32_t at = m * (uint32_t)units2 * kMx4Unit;
          *reinterpret_cast<uint16_t*>(o.codes + at + 16 * row + 4 * lgrp + 2 * (wave & 1)) =
              (uint16_t)mx4_encode4(acc[m][0], code);
          o.scale[at + row * o.G] = (char)code;   // (the same byte from every lane and wave of the row)
        }
      } else {
        // fp32 sums: the row is a term of the token's weighted sum, which rounds
        // once.  Rows past the tile are out of the buffer's bounds and dropped
        const auto y = __builtin_amdgcn_make_buffer_rsrc(
            static_cast<float*>(g.c) + ((size_t)cur.at.slice * g.P + cur.at.row_begin) * g.N_out, 0,
            blk.store ? cur.at.rows * g.N_out * 4 : 0, 0x00027000);
#pragma unroll
        for (int m = 0; m < MB; m++) {
          if (16 * m >= cur.at.rows) break;
          const int at = ((16 * m + lrow) * g.N_out + 16 * blk.out + 8 * lgrp) * 4;
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[m][0]), y, at, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[m][1]), y, at + 16, 0, 0);
        }
      }
      clear();
      cur = nxt;
      // the pair copies of the finish before this one are older than a whole
      // stage's operations
      wait_vm<St::NA + St::NS + St::NW>();
      nxt = sources(ahead, ii + 2);
      ahead = place(ii + 3);
      copy_pairs(ahead, ii + 3);
      ii++;
    };
    // stages in turn, the slots with them, straight across items
    for (int kt = 0;;) {
      stage(kt, slot0, slot1, w[0], swn[0]);
      if (++kt == nk) {
        finish();
        kt = 0;
        if (ii == n_items) break;
      }
      stage(kt, slot1, slot0, w[D - 1], swn[D - 1]);
      if (++kt == nk) {
        finish();
        kt = 0;
        if (ii == n_items) break;
      }
    }
    // the trailing re-loads still write this workgroup's LDS: let them land
    wait_vm<0>();
  };
  if (g.header[kHdrMaxExpertTiles] > 1) body(std::false_type{});
  else body(std::true_type{});
}

template <int MB, int G, int GS, bool GATEUP>
static hipError_t launch_mx4_strip_t(const moe_host::Mx4Args& a, int grid, hipStream_t s) {
  hipLaunchKernelGGL((mx4_strip_kernel<MB, G, GS, mx4_stages_ahead(MB, G, GS), GATEUP>), dim3(grid),
                     dim3(kMx4Waves * 64), 0, s, a);
  return hipGetLastError();
}

// Groups a stage: four to six units where the reduction divides into them
// (shorter stages leave too little in flight; Qwen2-57B-shaped slice, T = 1024,
// down over five units on 160-row tiles, one stage instead of five: 39.0 -> 36.3
// us).  Taller tiles have no registers for the longer stages, the gate-up, whose
// sources and epilogue take more, from 160 rows on, the down from 192.
static int mx4_stage_groups(int mb, int K, bool gateup) {
  const int units = K / 128;
  const bool room = mb <= (gateup ? 8 : 10);
  if (units % 4 == 0) return 1;
  if (units % 2 == 0) return room && units % 6 == 0 ? 3 : 1;
  if (room && units % 5 == 0) return 5;
  return units % 3 == 0 ? 3 : 1;
}

static int mx4_strip_stages(int mb, int K, bool gateup) { return K / 128 / mx4_group(K) / mx4_stage_groups(mb, K, gateup); }

template <int MB, bool GATEUP>
static hipError_t launch_mx4_strip_g(const moe_host::Mx4Args& a, int grid, hipStream_t s) {
  const int G = mx4_group(a.K), GS = mx4_stage_groups(MB, a.K, GATEUP);
  if (G == 4) return launch_mx4_strip_t<MB, 4, 1, GATEUP>(a, grid, s);
  if constexpr (MB <= (GATEUP ? 8 : 10)) {
    if (G == 2 && GS == 3) return launch_mx4_strip_t<MB, 2, 3, GATEUP>(a, grid, s);
    if (GS == 5) return launch_mx4_strip_t<MB, 1, 5, GATEUP>(a, grid, s);
  }
  if (G == 2) return launch_mx4_strip_t<MB, 2, 1, GATEUP>(a, grid, s);
  if (GS == 3) return launch_mx4_strip_t<MB, 1, 3, GATEUP>(a, grid, s);
  return launch_mx4_strip_t<MB, 1, 1, GATEUP>(a, grid, s);
}

}  // namespace moe

namespace moe_host {

int mx4_down_stages(int mb, int K) { return moe::mx4_strip_stages(mb, K, false); }

hipError_t launch_mx4_strip(const Mx4Args& a, bool gateup, int mb, int grid, hipStream_t s) {
  if (a.K % 128 || a.N_out % 128 || a.w_rows != (gateup ? 2 : 1) * a.N_out) return hipErrorInvalidValue;
  if (a.split < 1 || (gateup && a.split > 1) || moe::mx4_strip_stages(mb, a.K, gateup) % a.split) return hipErrorInvalidValue;
#define MOE_MX4_CASE(M) \
  if (mb == M) return gateup ? moe::launch_mx4_strip_g<M, true>(a, grid, s) : moe::launch_mx4_strip_g<M, false>(a, grid, s);
  MOE_MX4_CASE(4) MOE_MX4_CASE(6) MOE_MX4_CASE(8) MOE_MX4_CASE(10) MOE_MX4_CASE(12)
#undef MOE_MX4_CASE
  return hipErrorInvalidValue;
}

}  // namespace moe_host
