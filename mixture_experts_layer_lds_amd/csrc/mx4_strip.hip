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
//    codes go to one of two LDS slots by direct global->LDS copies spread over
//    the waves, while the other slot is multiplied.
//  * The wave's weights of a unit are loaded into the registers that the
//    multiplication of the same unit of the stage before has just left, so a
//    whole stage (8 KiB a wave at four units, 64 KiB a CU) stays in flight at
//    the cost of one stage of registers, and the copies and loads run straight
//    across work items.
//  * Gate-up epilogue: 32 columns of h are one MXFP4 block a row, held by two
//    neighbouring waves; they exchange the rows' largest magnitudes through
//    LDS and write codes and scale codes in the blocks that the down GEMM
//    copies as contiguous chunks.  Down writes bf16 rows, 16 bytes a lane.
//
// Every wave issues the same number of vector-memory operations a stage
// (copies past the tile's chunks repeat an earlier one, bytes and place), so
// the wait at the head of a stage is an exact count.
#include "lds_dma.h"
#include "mx4_epilogue.h"

namespace moe {

constexpr int kMx4Waves = 8;

template <int MB, int G, int GS>
struct Mx4Stage {
  static constexpr int U = G * GS;                                   // units
  static constexpr int NA = (MB * U + kMx4Waves - 1) / kMx4Waves;    // token chunks a wave copies
  static constexpr int NS = (MB * GS + kMx4Waves - 1) / kMx4Waves;   // scale chunks
  static constexpr int NW = 2 * U + 2 * GS;                          // weight loads of a wave
  static constexpr int kTokens = MB * U * 1024;
  static constexpr int kSlot = kTokens + MB * GS * 256;
  static constexpr int kLds = 2 * kSlot + kMx4Waves * MB * 16 * 4;
};

template <int MB, int G, int GS>
struct Mx4Item {
  using St = Mx4Stage<MB, G, GS>;
  int ti, row_begin, rows;
  int blk0;                        // gate-up: first of the 32-column pair's blocks; down: the wave's first block
  bool store;                      // the wave's columns exist (down: H may end inside a strip)
  const char* abase;               // of the offsets a[] (and, down, s[]): uniform
  uint32_t a[St::NA], s[St::NS];   // this lane's byte offsets
  const char* b[2];                // the wave's weight blocks: uniform
};

template <int MB, int G, int GS, bool GATEUP>
__device__ __forceinline__ Mx4Item<MB, G, GS> mx4_item(const moe_host::Mx4Args& g, int item, int n_strips, int wave,
                                                       int lane) {
  using St = Mx4Stage<MB, G, GS>;
  Mx4Item<MB, G, GS> it;
  const int units = g.K / 128;
  const uint32_t block_bytes = (uint32_t)units * kMx4Unit;
  it.ti = item / n_strips;
  const int nt = item - it.ti * n_strips;   // the strips of one tile side by side: they meet its token rows in L2
  const moe_task_t task = load_task_scalar(g.tasks + it.ti);
  it.row_begin = task.row_begin;
  it.rows = task.rows;
  // x codes take at most 2^31 bytes (T H / 2), a task's blocks of h far less:
  // 32-bit offsets from a uniform base
  it.abase = static_cast<const char*>(g.a) + (GATEUP ? 0 : (size_t)it.ti * MB * block_bytes);
  // row blocks past the tile, and rows past it inside the last block, re-read
  // the tile's first row (gate-up) or block: valid, never stored
#pragma unroll
  for (int i = 0; i < St::NA; i++) {
    const int c = (wave + kMx4Waves * i) % (MB * St::U);   // chunk: row block c / U, unit c % U
    const int rb = c / St::U, u = c % St::U;
    const bool in = rb * 16 < task.rows;
    if constexpr (GATEUP) {
      const int crow = tok_copy_row(lane);
      const i32x16_t sp = load16_scalar(g.sorted_pairs + task.row_begin + (in ? rb * 16 : 0));
      const int p = in && rb * 16 + crow < task.rows ? pick16(sp, crow) : sp[0];
      it.a[i] = (uint32_t)(p / g.topk) * (uint32_t)(g.K / 2) + u * 64 + 16 * tok_copy_piece(lane);
    } else {
      it.a[i] = (in ? rb : 0) * block_bytes + u / G * (G * kMx4Unit) + u % G * 1024 + 16 * lane;
    }
  }
#pragma unroll
  for (int i = 0; i < St::NS; i++) {
    const int c = (wave + kMx4Waves * i) % (MB * GS);      // row block c / GS, group c % GS
    const int rb = c / GS, j = c % GS;
    const bool in = rb * 16 < task.rows;
    if constexpr (GATEUP) {
      const int lrow = lane & 15;
      const i32x16_t sp = load16_scalar(g.sorted_pairs + task.row_begin + (in ? rb * 16 : 0));
      const int p = in && rb * 16 + lrow < task.rows ? spread16(sp, lane) : sp[0];
      it.s[i] = (uint32_t)(p / g.topk) * (uint32_t)(g.K / 32) + 4 * G * j + (((lane >> 4) * G) & ~3);
    } else {
      it.s[i] = (in ? rb : 0) * block_bytes + j * (G * kMx4Unit) + G * 1024 + ((lane * G) & ~3);
    }
  }
  int b0, b1;
  if constexpr (GATEUP) {
    it.blk0 = 8 * nt + (wave & ~1);   // 128 h columns a strip, 32 a pair of waves
    b0 = it.blk0 + (wave & 1);
    b1 = b0 + g.N_out / 16;
    it.store = true;
  } else {
    it.blk0 = 16 * nt + 2 * wave;
    it.store = it.blk0 < g.N_out / 16;
    b0 = it.store ? it.blk0 : 0;
    b1 = b0 + 1;
  }
  const char* B = static_cast<const char*>(g.b) + (size_t)task.expert * (g.w_rows / 16) * block_bytes;
  it.b[0] = B + (size_t)b0 * block_bytes;
  it.b[1] = B + (size_t)b1 * block_bytes;
  return it;
}

template <int MB, int G, int GS, bool GATEUP>
__global__ void __launch_bounds__(kMx4Waves * 64, 1)
mx4_strip_kernel(moe_host::Mx4Args g) {
  using St = Mx4Stage<MB, G, GS>;
  using It = Mx4Item<MB, G, GS>;
  constexpr int U = St::U;
  static_assert(MB % 4 == 0, "row blocks are read four at a time");
  static_assert(St::NW < 64, "vmcnt range");
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  uint32_t* amax = reinterpret_cast<uint32_t*>(lds + 2 * St::kSlot);   // [wave][16 MB rows]
  const int lane = threadIdx.x & 63;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int num_tasks = min(g.header[kHdrNumTasks], g.max_tasks);
  const int n_strips = GATEUP ? g.N_out / 128 : (g.N_out + 255) / 256;
  const int total = num_tasks * n_strips;
  const int nk = g.K / 128 / U;   // stages per item
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
    It cur = mx4_item<MB, G, GS, GATEUP>(g, vid, n_strips, wave, lane);
    It nxt = cur;   // past the last item its own first stage again: valid, never used
    if (n_items > 1) nxt = mx4_item<MB, G, GS, GATEUP>(g, vid + gs, n_strips, wave, lane);

    auto issue_tokens = [&](bool in_cur, int kt, char* slot) __attribute__((always_inline)) {
      const size_t at = GATEUP ? (size_t)kt * (U * 64) : (size_t)kt * (U * kMx4Unit);
      const char* as = (in_cur ? cur.abase : nxt.abase) + at;
      const char* ss = GATEUP ? reinterpret_cast<const char*>(g.a_sc) + (size_t)kt * (4 * U) : as;
#pragma unroll
      for (int i = 0; i < St::NA; i++)
        dma16(as + (in_cur ? cur.a[i] : nxt.a[i]), slot + ((wave + kMx4Waves * i) % (MB * U)) * 1024);
#pragma unroll
      for (int i = 0; i < St::NS; i++)
        dma4(ss + (in_cur ? cur.s[i] : nxt.s[i]), slot + St::kTokens + ((wave + kMx4Waves * i) % (MB * GS)) * 256);
    };
    u32x4 w[U][2];
    uint32_t sw[GS][2];
    auto load_unit = [&](const char* b0, const char* b1, int u) __attribute__((always_inline)) {
      const int at = u / G * (G * kMx4Unit) + u % G * 1024;
      const u32x4* p0 = reinterpret_cast<const u32x4*>(b0 + at + wlane);
      const u32x4* p1 = reinterpret_cast<const u32x4*>(b1 + at + wlane);
      w[u][0] = NT_B ? __builtin_nontemporal_load(p0) : *p0;
      w[u][1] = NT_B ? __builtin_nontemporal_load(p1) : *p1;
      if (u % G == G - 1) {   // the group's scale codes with its last unit
        const uint32_t* q0 = reinterpret_cast<const uint32_t*>(b0 + u / G * (G * kMx4Unit) + slane);
        const uint32_t* q1 = reinterpret_cast<const uint32_t*>(b1 + u / G * (G * kMx4Unit) + slane);
        sw[u / G][0] = NT_B ? __builtin_nontemporal_load(q0) : *q0;
        sw[u / G][1] = NT_B ? __builtin_nontemporal_load(q1) : *q1;
      }
    };
    // The empty asm statements keep the copies ahead of the weights in issue
    // order, which the vmcnt count relies on.
    issue_tokens(true, 0, lds);
    __asm__ volatile("" ::: "memory");
#pragma unroll
    for (int u = 0; u < U; u++) load_unit(cur.b[0], cur.b[1], u);
    __asm__ volatile("" ::: "memory");

    int par = 0;   // LDS slot of the stage
    for (int ii = 0; ii < n_items; ii++) {
      f32x4 acc[MB][2];
#pragma unroll
      for (int m = 0; m < MB; m++) acc[m][0] = acc[m][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

      for (int kt = 0; kt < nk; kt++, par ^= 1) {
        // the stage's copies have landed in this wave (only its weights were
        // issued after them), then in every wave
        __asm__ volatile("" ::: "memory");
        wait_vm<St::NW>();
        barrier_nofence();
        // the next stage into the slot that every wave had read before the barrier
        const bool in_cur = kt + 1 < nk;
        const int kn = in_cur ? kt + 1 : 0;
        issue_tokens(in_cur, kn, lds + (par ^ 1) * St::kSlot);
        __asm__ volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        const char* b0 = (in_cur ? cur.b[0] : nxt.b[0]) + (size_t)kn * (U * kMx4Unit);
        const char* b1 = (in_cur ? cur.b[1] : nxt.b[1]) + (size_t)kn * (U * kMx4Unit);
        const char* sb = lds + par * St::kSlot;
        const uint32_t* sc = reinterpret_cast<const uint32_t*>(sb + St::kTokens);
        // four row blocks at a time, their fragments read while the previous
        // four are multiplied; the scheduling barriers keep the compiler from
        // reading more of them ahead than there are registers for
        u32x4 t[2][4];
        uint32_t st[MB];
        auto read4 = [&](u32x4 (&to)[4], int step) __attribute__((always_inline)) {
#pragma unroll
          for (int i = 0; i < 4; i++)
            to[i] = *reinterpret_cast<const u32x4*>(sb + ((step % (MB / 4) * 4 + i) * U + step / (MB / 4)) * 1024 + aoff);
        };
        read4(t[0], 0);
#pragma unroll
        for (int j = 0; j < GS; j++) {
#pragma unroll
          for (int m = 0; m < MB; m++) st[m] = sc[64 * (m * GS + j) + lane] >> ash;
          mx4_units<G>([&](auto uu) {
            constexpr int V = decltype(uu)::value;
            const int un = j * G + V;
#pragma unroll
            for (int mc = 0; mc < MB / 4; mc++) {
              const int step = un * (MB / 4) + mc;
              if (step + 1 < U * (MB / 4)) read4(t[(step + 1) & 1], step + 1);
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int i = 0; i < 4; i++) {
                mfma_mx4<V>(acc[4 * mc + i][0], w[un][0], t[step & 1][i], sw[j][0] >> bsh, st[4 * mc + i]);
                mfma_mx4<V>(acc[4 * mc + i][1], w[un][1], t[step & 1][i], sw[j][1] >> bsh, st[4 * mc + i]);
              }
              __builtin_amdgcn_sched_barrier(0);
            }
            load_unit(b0, b1, un);   // of the next stage
            __builtin_amdgcn_sched_barrier(0);
          });
        }
      }

      if constexpr (GATEUP) {
        // h = SiLU(gate) * up in place of the gate sums; the row's largest
        // magnitude over this wave's 16 columns to LDS
#pragma unroll
        for (int m = 0; m < MB; m++) {
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            acc[m][0][i] = silu_f32(acc[m][0][i]) * acc[m][1][i];
            mx = max(mx, abs_bits(acc[m][0][i]));
          }
          mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
          mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
          if (lgrp == 0) amax[(wave * MB + m) * 16 + lrow] = mx;
        }
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the writes are in LDS
        barrier_nofence();
        // (the next write of `amax` comes after the barriers of the next item's stages)
#pragma unroll
        for (int m = 0; m < MB; m++) {
          const uint32_t mx = max(amax[(wave * MB + m) * 16 + lrow], amax[((wave ^ 1) * MB + m) * 16 + lrow]);
          const uint32_t code = mx4_scale_code(mx);
          const uint32_t w4 = mx4_encode4(acc[m][0], code);
          if (16 * m + lrow < cur.rows) {
            const Mx4Out o = mx4_out(g.c, (size_t)cur.ti * MB + m, cur.blk0 / 2, units2, G2);
            *reinterpret_cast<uint16_t*>(o.codes + 16 * lrow + 4 * lgrp + 2 * (wave & 1)) = (uint16_t)w4;
            if (lgrp == 0 && (wave & 1) == 0) o.scale[lrow * o.G] = (char)code;
          }
        }
      } else {
#pragma unroll
        for (int m = 0; m < MB; m++) {
          if (16 * m + lrow < cur.rows && cur.store) {
            u32x4 v;
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = bf16_pair(acc[m][i >> 1][2 * (i & 1)], acc[m][i >> 1][2 * (i & 1) + 1]);
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.c) + (size_t)(cur.row_begin + 16 * m + lrow) * g.N_out +
                                      16 * cur.blk0 + 8 * lgrp) = v;
          }
        }
      }
      cur = nxt;
      if (ii + 2 < n_items) nxt = mx4_item<MB, G, GS, GATEUP>(g, vid + (ii + 2) * gs, n_strips, wave, lane);
    }
    // the trailing re-loads still write this workgroup's LDS: let them land
    wait_vm<0>();
  };
  if (g.header[kHdrMaxExpertTiles] > 1) body(std::false_type{});
  else body(std::true_type{});
}

template <int MB, int G, int GS, bool GATEUP>
static hipError_t launch_mx4_strip_t(const moe_host::Mx4Args& a, int grid, hipStream_t s) {
  constexpr int lds_bytes = Mx4Stage<MB, G, GS>::kLds;
  static_assert(lds_bytes <= 160 * 1024, "LDS of a CU");
  // (an attribute of the function on the current device; set before every launch)
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx4_strip_kernel<MB, G, GS, GATEUP>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, lds_bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((mx4_strip_kernel<MB, G, GS, GATEUP>), dim3(grid), dim3(kMx4Waves * 64), lds_bytes, s, a);
  return hipGetLastError();
}

// Stages of four to six units where the reduction divides into them: shorter
// ones leave too little in flight.
template <int MB, bool GATEUP>
static hipError_t launch_mx4_strip_g(const moe_host::Mx4Args& a, int grid, hipStream_t s) {
  const int units = a.K / 128;
  if (units % 4 == 0) return launch_mx4_strip_t<MB, 4, 1, GATEUP>(a, grid, s);
  if constexpr (MB <= 8) {   // 192 rows: two slots of six units do not fit, five spill registers
    if (units % 6 == 0) return launch_mx4_strip_t<MB, 2, 3, GATEUP>(a, grid, s);
    if (units % 10 == 5) return launch_mx4_strip_t<MB, 1, 5, GATEUP>(a, grid, s);
  }
  if (units % 2 == 0) return launch_mx4_strip_t<MB, 2, 1, GATEUP>(a, grid, s);
  if (units % 3 == 0) return launch_mx4_strip_t<MB, 1, 3, GATEUP>(a, grid, s);
  return launch_mx4_strip_t<MB, 1, 1, GATEUP>(a, grid, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_mx4_strip(const Mx4Args& a, bool gateup, int mb, int grid, hipStream_t s) {
  if (a.K % 128 || a.N_out % 128 || a.w_rows != (gateup ? 2 : 1) * a.N_out) return hipErrorInvalidValue;
#define MOE_MX4_CASE(M) \
  if (mb == M) return gateup ? moe::launch_mx4_strip_g<M, true>(a, grid, s) : moe::launch_mx4_strip_g<M, false>(a, grid, s);
  MOE_MX4_CASE(4) MOE_MX4_CASE(8) MOE_MX4_CASE(12)
#undef MOE_MX4_CASE
  return hipErrorInvalidValue;
}

}  // namespace moe_host
