// MXFP4 grouped GEMM for few rows per expert (decode and small batches),
// and the down GEMM with the top-k sum of a single token.
//
// Same pipeline role as stream_gemm.hip (HPC-Ops x SGLang blog, section
// "MoE": gate-up reads tokens through the route index; a persistent grid
// consumes the per-tile task map; the activation follows the gate-up GEMM).
// What bounds it is the weight stream: at one to sixteen rows an expert
// every weight byte (17/32 a value with its scale) meets a few rows.
//
//  * Work item = (task tile of 16 MB rows, 64 weight rows).  Gate-up: the two
//    16-row blocks of 32 gate rows and the two of the matching up rows, so the
//    item holds 32 columns of h, one MXFP4 block of its rows, and writes h as
//    codes: no fp32 or bf16 h in memory and no requantisation launch.  Down:
//    64 columns.
//  * A workgroup of W waves takes one item; wave w reduces every W-th group of
//    units.  The weights are the first MFMA operand (16 weight rows), the
//    tokens the second (16 columns), so a lane ends up with eight consecutive
//    output columns of one token row: its codes are one dword, its fp32 sums
//    two 16-byte stores.
//  * The group's weights (4 blocks x 1 KiB a unit) and scale codes (one dword
//    a lane for all its units) go straight to registers, non-temporal, one
//    group ahead of the one that is multiplied, the next item's first group
//    ahead of the epilogue (Qwen3-30B-A3B-shaped T = 64 41.5 -> 39.8 us a
//    layer, Mixtral-8x7B-shaped 145 -> 140, DeepSeek-V3-shaped T = 16 384 ->
//    380).
//  * The waves' sums meet in LDS and are added in ascending wave order.
//
// Measured, gate-up / down in us (TB/s of weights with their scale codes):
// DeepSeek-V3-shaped T = 16 251 (6.5) / 125 (6.5), T = 64 517 (6.7) / 276
// (6.3); Mixtral-8x7B-shaped T = 16 79 (6.3) / 42 (6.0); Qwen3-30B-A3B-shaped
// T = 64 19.7 (4.2) / 13.2 (3.2), too short to reach the full rate.  One token,
// DeepSeek-V3-shaped: 20.5 (6.1) and, with the top-k sum, 14.3 (4.4).
#include "decode_route.h"
#include "lds_dma.h"
#include "mx4_epilogue.h"

namespace moe {

constexpr int kMx4NB = 4;   // 16-row weight blocks per item

// A lane's scale codes of a group, as the low bytes of a dword: its piece at
// byte G * lane of the block's scale area.
template <int G>
__device__ __forceinline__ const char* mx4_piece(const char* area, int lane) {
  return area + ((lane * G) & ~3);
}
template <int G>
__device__ __forceinline__ int mx4_piece_shift(int lane) {
  return 8 * ((lane * G) & 3);
}

template <int MB, int W, int G, bool GATEUP>
__global__ void __launch_bounds__(W * 64)
mx4_stream_kernel(moe_host::Mx4Args g) {
  __shared__ f32x4 red[W][MB][kMx4NB][64];
  const int lane = threadIdx.x & 63;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int num_tasks = min(g.header[kHdrNumTasks], g.max_tasks);
  const int n_groups = g.N_out / (GATEUP ? 32 : 64);   // items per task
  const int total = num_tasks * n_groups;
  const int units = g.K / 128, ngrp = units / G;
  const char* __restrict__ A = static_cast<const char*>(g.a);
  const char* __restrict__ B = static_cast<const char*>(g.b);
  const size_t block_bytes = (size_t)units * kMx4Unit;
  const size_t expert_bytes = (size_t)(g.w_rows / 16) * block_bytes;
  // the down GEMM's group size, in which h is stored
  const int units2 = g.N_out / 128, G2 = units2 % 4 == 0 ? 4 : (units2 % 2 == 0 ? 2 : 1);

  // XCD-aware numbering: consecutive items (the column groups of one task)
  // on the workgroups of one XCD, sharing the task's token rows in L2.
  const int gs = gridDim.x;
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8;
  const int per_xcd = gs / 8, extra = gs % 8;
  const int vid = (xcd < extra ? xcd * (per_xcd + 1) : extra * (per_xcd + 1) + (xcd - extra) * per_xcd) + slot;

  if (vid >= total) return;
  struct Stage {
    u32x4 w[G][kMx4NB], t[G][MB];
    uint32_t sw[kMx4NB], st[MB];
  };
  Stage s0, s1;
  const char* bp[kMx4NB];
  // 16-row weight blocks: gate 0, gate 1, up 0, up 1, or four of the output
  auto blocks = [&](int expert, int cg) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < kMx4NB; q++) {
      const int blk = GATEUP ? (q & 1) + 2 * cg + (q >> 1) * (g.N_out / 16) : 4 * cg + q;
      bp[q] = B + (size_t)expert * expert_bytes + (size_t)blk * block_bytes;
    }
  };
  auto load_weights = [&](Stage& f, int grp) __attribute__((always_inline)) {
    const size_t at = (size_t)grp * (G * kMx4Unit);
#pragma unroll
    for (int q = 0; q < kMx4NB; q++)
      f.sw[q] = __builtin_nontemporal_load(
          reinterpret_cast<const uint32_t*>(mx4_piece<G>(bp[q] + at + G * 1024, lane)));
#pragma unroll
    for (int u = 0; u < G; u++)
#pragma unroll
      for (int q = 0; q < kMx4NB; q++)
        f.w[u][q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bp[q] + at + u * 1024 + 16 * lane));
  };
  const int n = ngrp > wave ? (ngrp - wave + W - 1) / W : 0;   // groups of this wave
  int item = vid, ti = item / n_groups;
  moe_task_t task = load_task_scalar(g.tasks + ti);
  blocks(task.expert, item - ti * n_groups);
  // an item's first weights are loaded before the (dependent) look-up of its
  // token rows, and from the second item on while the one before is finished
  if (n > 0) load_weights(s0, wave);
  for (;;) {
    const int cg = item - ti * n_groups;
    const int next = item + gs, next_ti = next < total ? next / n_groups : ti;
    // token rows: rows past the tile re-read its first row (a valid address
    // whose products land only in columns that are never stored)
    const char *ap[MB], *asp[MB];
#pragma unroll
    for (int b = 0; b < MB; b++) {
      const int rb = b * 16 < task.rows ? b : 0;
      if constexpr (GATEUP) {
        const i32x16_t sp = load16_scalar(g.sorted_pairs + task.row_begin + rb * 16);
        const int p = rb * 16 + lrow < task.rows ? spread16(sp, lane) : sp[0];
        const size_t row = (size_t)(p / g.topk);
        ap[b] = A + row * (g.K / 2) + 16 * lgrp;
        asp[b] = reinterpret_cast<const char*>(g.a_sc) + row * (g.K / 32) + ((lgrp * G) & ~3);
      } else {
        ap[b] = A + ((size_t)ti * MB + rb) * block_bytes + 16 * lane;
        asp[b] = mx4_piece<G>(A + ((size_t)ti * MB + rb) * block_bytes + G * 1024, lane);
      }
    }
    const int ash = GATEUP ? 8 * ((lgrp * G) & 3) : mx4_piece_shift<G>(lane);
    const int bsh = mx4_piece_shift<G>(lane);

    auto load_tokens = [&](Stage& f, int grp) __attribute__((always_inline)) {
      const size_t at = (size_t)grp * (G * kMx4Unit);
#pragma unroll
      for (int b = 0; b < MB; b++)
        f.st[b] = *reinterpret_cast<const uint32_t*>(asp[b] + (GATEUP ? (size_t)grp * (4 * G) : at));
#pragma unroll
      for (int u = 0; u < G; u++)
#pragma unroll
        for (int b = 0; b < MB; b++)
          f.t[u][b] = *reinterpret_cast<const u32x4*>(
              ap[b] + (GATEUP ? (size_t)(grp * G + u) * 64 : at + u * 1024));
    };
    auto load = [&](Stage& f, int grp) __attribute__((always_inline)) {
      load_tokens(f, grp);
      load_weights(f, grp);
    };
    f32x4 acc[MB][kMx4NB];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int q = 0; q < kMx4NB; q++) acc[m][q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto compute = [&](const Stage& f) __attribute__((always_inline)) {
      mx4_units<G>([&](auto u) {
        constexpr int U = decltype(u)::value;
#pragma unroll
        for (int b = 0; b < MB; b++)
#pragma unroll
          for (int q = 0; q < kMx4NB; q++)
            mfma_mx4<U>(acc[b][q], f.w[U][q], f.t[U][b], f.sw[q] >> bsh, f.st[b] >> ash);
      });
    };
    // Groups wave, wave + W, ...: no load sits under a condition inside the
    // loop, so each multiply waits for exactly its own group while the next
    // one is in flight.
    if (n > 0) load_tokens(s0, wave);
    const moe_task_t next_task = load_task_scalar(g.tasks + next_ti);
    if (n > 0) {
      int i = 0;
      for (; i + 2 < n; i += 2) {
        load(s1, wave + (i + 1) * W);
        compute(s0);
        load(s0, wave + (i + 2) * W);
        compute(s1);
      }
      if (i + 1 < n) {
        load(s1, wave + (i + 1) * W);
        compute(s0);
        compute(s1);
      } else {
        compute(s0);
      }
    }

    if (next < total) {
      blocks(next_task.expert, next - next_ti * n_groups);
      if (n > 0) load_weights(s0, wave);
    }
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int q = 0; q < kMx4NB; q++) red[wave][m][q][lane] = acc[m][q];
    __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the sums are in LDS
    barrier_nofence();

    // Epilogue of row block m by wave m % W: lane holds token row lane % 16
    // and, of block q, output columns 8 (lane / 16) + 4 (q % 2) + i of its 32.
    for (int m = wave; m < MB; m += W) {
      f32x4 tot[kMx4NB];
#pragma unroll
      for (int q = 0; q < kMx4NB; q++) {
        tot[q] = red[0][m][q][lane];
#pragma unroll
        for (int s = 1; s < W; s++) tot[q] += red[s][m][q][lane];
      }
      const int rr = m * 16 + lrow;
      if constexpr (GATEUP) {
        float h[8];
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
          h[i] = mx4_silu(tot[i >> 2][i & 3]) * tot[2 + (i >> 2)][i & 3];
          mx = max(mx, abs_bits(h[i]));
        }
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
        mx = max(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
        const uint32_t code = mx4_scale_code(mx);
        const uint32_t w8 = mx4_encode8(h, code);
        if (rr < task.rows) {
          const Mx4Out o = mx4_out(g.c, (size_t)ti * MB + m, cg, units2, G2);
          *reinterpret_cast<uint32_t*>(o.codes + 16 * lrow + 4 * lgrp) = w8;
          if (lgrp == 0) o.scale[lrow * o.G] = (char)code;
        }
      } else if (rr < task.rows) {
        // fp32: the row is a term of the token's weighted sum, which rounds once
        float* y = static_cast<float*>(g.c) + (size_t)(task.row_begin + rr) * g.N_out + 64 * cg + 8 * lgrp;
#pragma unroll
        for (int q = 0; q < kMx4NB; q++) *reinterpret_cast<f32x4*>(y + 32 * (q >> 1) + 4 * (q & 1)) = tot[q];
      }
    }
    if (next >= total) break;
    __builtin_amdgcn_s_waitcnt(0xC07F);   // this wave's reads of LDS are done
    barrier_nofence();                    // LDS free for the next item
    item = next;
    ti = next_ti;
    task = next_task;
  }
}

// Down GEMM and top-k weighted sum of a single token in one launch:
// out[c] = sum over the token's rows of w_r (h_r . W2[e_r][c]).  One
// workgroup of W waves per 16 output columns; the groups of all the token's
// experts form one list, cut into equal runs, one a wave.  At the end of each
// expert's run a lane weights the column of the product that is its row
// (rows outside the task are dropped by a select, whatever they hold), and
// the rows' and waves' sums meet at the end: no partial rows in memory, no
// further launch.
template <int W, int G>
__global__ void __launch_bounds__(W * 64)
mx4_down_reduce_kernel(moe_host::Mx4Args g) {
  __shared__ f32x4 red[W][4];
  __shared__ moe_task_t tk[kMaxTopK];
  const int lane = threadIdx.x & 63;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (threadIdx.x < kMaxTopK && (int)threadIdx.x < g.max_tasks) tk[threadIdx.x] = g.tasks[threadIdx.x];
  const int nt = min(min(g.header[kHdrNumTasks], g.max_tasks), kMaxTopK);
  const i32x16_t sp = load16_scalar(g.sorted_pairs);
  __syncthreads();

  const int units = g.K / 128, ngrp = units / G;
  const size_t block_bytes = (size_t)units * kMx4Unit;
  const size_t expert_bytes = (size_t)(g.w_rows / 16) * block_bytes;
  const char* __restrict__ A = static_cast<const char*>(g.a);
  const char* __restrict__ B = static_cast<const char*>(g.b) + (size_t)blockIdx.x * block_bytes;
  const int total = nt * ngrp;
  const int per = (total + W - 1) / W;
  const int first = min(total, wave * per), n = min(total, first + per) - first;
  const int sh = mx4_piece_shift<G>(lane);

  struct Stage {
    u32x4 w[G], t[G];
    uint32_t sw, st;
  };
  auto load = [&](Stage& f, int i) __attribute__((always_inline)) {
    const int t = i / ngrp;
    const size_t at = (size_t)(i - t * ngrp) * (G * kMx4Unit);
    const char* bp = B + (size_t)__builtin_amdgcn_readfirstlane(tk[t].expert) * expert_bytes + at;
    const char* ap = A + (size_t)t * block_bytes + at;   // the task's one 16-row block
    f.sw = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(mx4_piece<G>(bp + G * 1024, lane)));
    f.st = *reinterpret_cast<const uint32_t*>(mx4_piece<G>(ap + G * 1024, lane));
#pragma unroll
    for (int u = 0; u < G; u++) {
      f.w[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(bp + u * 1024 + 16 * lane));
      f.t[u] = *reinterpret_cast<const u32x4*>(ap + u * 1024 + 16 * lane);
    }
  };
  f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f}, sum = acc;
  auto compute = [&](const Stage& f, int i) __attribute__((always_inline)) {
    mx4_units<G>([&](auto u) {
      constexpr int U = decltype(u)::value;
      mfma_mx4<U>(acc, f.w[U], f.t[U], f.sw >> sh, f.st >> sh);
    });
    const int t = i / ngrp;
    if (i + 1 == first + n || (i + 1) % ngrp == 0) {   // the task's last group of this wave
      const moe_task_t task = tk[t];
      const bool in = lrow < task.rows;
      const float w = g.topk_w[in ? pick16(sp, (task.row_begin + lrow) & 15) : 0];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        sum[j] += in ? w * acc[j] : 0.0f;
        acc[j] = 0.0f;
      }
    }
  };
  if (n > 0) {
    Stage s0, s1;
    load(s0, first);
    int i = 0;
    for (; i + 2 < n; i += 2) {
      load(s1, first + i + 1);
      compute(s0, first + i);
      load(s0, first + i + 2);
      compute(s1, first + i + 1);
    }
    if (i + 1 < n) {
      load(s1, first + i + 1);
      compute(s0, first + i);
      compute(s1, first + i + 1);
    } else {
      compute(s0, first + i);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; j++)
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) sum[j] += __shfl_xor(sum[j], o, 64);
  if (lrow == 0) red[wave][lgrp] = sum;
  __syncthreads();
  if (threadIdx.x < 4) {
    f32x4 v = red[0][threadIdx.x];
#pragma unroll
    for (int w = 1; w < W; w++) v += red[w][threadIdx.x];
    const int col = 32 * (blockIdx.x / 2) + 8 * threadIdx.x + 4 * (blockIdx.x % 2);
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(g.c) + col) =
        u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  }
}

template <int MB, int W, bool GATEUP>
static hipError_t launch_mx4_stream_t(const moe_host::Mx4Args& a, int grid, hipStream_t s) {
  switch (mx4_group(a.K)) {
    case 4: hipLaunchKernelGGL((mx4_stream_kernel<MB, W, 4, GATEUP>), dim3(grid), dim3(W * 64), 0, s, a); break;
    case 2: hipLaunchKernelGGL((mx4_stream_kernel<MB, W, 2, GATEUP>), dim3(grid), dim3(W * 64), 0, s, a); break;
    default: hipLaunchKernelGGL((mx4_stream_kernel<MB, W, 1, GATEUP>), dim3(grid), dim3(W * 64), 0, s, a); break;
  }
  return hipGetLastError();
}

template <int MB, int W>
static hipError_t launch_mx4_stream_w(const moe_host::Mx4Args& a, bool gateup, int grid, hipStream_t s) {
  return gateup ? launch_mx4_stream_t<MB, W, true>(a, grid, s) : launch_mx4_stream_t<MB, W, false>(a, grid, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_mx4_stream(const Mx4Args& a, bool gateup, int mb, int waves, int grid, hipStream_t s) {
  if (a.K % 128 || a.N_out % 128 || a.w_rows != (gateup ? 2 : 1) * a.N_out) return hipErrorInvalidValue;
#define MOE_MX4_CASE(M, Wv) \
  if (mb == M && waves == Wv) return moe::launch_mx4_stream_w<M, Wv>(a, gateup, grid, s);
  MOE_MX4_CASE(1, 1) MOE_MX4_CASE(1, 2) MOE_MX4_CASE(1, 4) MOE_MX4_CASE(1, 8)
  MOE_MX4_CASE(2, 1) MOE_MX4_CASE(2, 2) MOE_MX4_CASE(2, 4) MOE_MX4_CASE(2, 8)
#undef MOE_MX4_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_mx4_down_reduce(const Mx4Args& a, hipStream_t s) {
  if (a.K % 128 || a.N_out % 128 || a.w_rows != a.N_out || a.topk > moe::kMaxTopK) return hipErrorInvalidValue;
  const dim3 grid(a.N_out / 16);
  switch (moe::mx4_group(a.K)) {
    case 4: hipLaunchKernelGGL((moe::mx4_down_reduce_kernel<8, 4>), grid, dim3(512), 0, s, a); break;
    case 2: hipLaunchKernelGGL((moe::mx4_down_reduce_kernel<8, 2>), grid, dim3(512), 0, s, a); break;
    default: hipLaunchKernelGGL((moe::mx4_down_reduce_kernel<8, 1>), grid, dim3(512), 0, s, a); break;
  }
  return hipGetLastError();
}

}  // namespace moe_host
