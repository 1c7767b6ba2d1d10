// The LDS-tile kernel of the linear layers and their gradients (linear.h).
//
//  * A persistent grid goes over items (expert, tile of m, tile of c).  Which
//    rows an expert has is known on the device only: every workgroup counts the
//    experts' tiles from expert_offsets when it starts, and the grid depends on
//    the sizes alone.  Neighbouring items share an operand's tile; workgroups
//    are renumbered so that an XCD takes a run of them.
//  * A stage is KG sub-steps of 64 q of both operands, copied straight to LDS
//    while the stage before is multiplied.  Rows behind an expert's last, and q
//    behind the end, are outside the copy's buffer range and come as zeros.
//  * Sums are fp32; bias, activation, residual and the one rounding happen on
//    the accumulators.
#pragma once

#include "linear.h"

namespace moe {

constexpr int kXcds = 8;

// Workgroups are dealt to the XCDs in turn: renumber them so that each XCD has a run.
__device__ __forceinline__ int xcd_order(int b, int G) {
  const int xcd = b % kXcds, slot = b / kXcds;
  const int per = G / kXcds, extra = G % kXcds;
  return (xcd < extra ? xcd * (per + 1) : extra * (per + 1) + (xcd - extra) * per) + slot;
}

// Every vector-memory and LDS operation of this wave is done.
__device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(0x0070); }

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Rows [begin, end) of expert e, kept inside [0, rows): a routing buffer that
// does not belong to these sizes cannot lead an access out of bounds.
struct RowRange {
  int begin, end;
};
__device__ __forceinline__ RowRange expert_rows(const moe_host::LinearArgs& g, int e) {
  if (!g.expert_offsets) return {0, g.rows};
  const int a = min(max(g.expert_offsets[e], 0), g.rows);
  return {a, min(max(g.expert_offsets[e + 1], a), g.rows)};
}

// first[e]: the first item of expert e, first[E] their number; wave 0 fills it.
template <int BM>
__device__ __forceinline__ void count_items(const moe_host::LinearArgs& g, int tiles_c, int* first, int lane) {
  int n[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const int e = lane * 8 + i;
    n[i] = 0;
    if (e < g.E) {
      const RowRange r = expert_rows(g, e);
      n[i] = (r.end - r.begin + BM - 1) / BM * tiles_c;
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
    if (lane * 8 + i <= g.E) first[lane * 8 + i] = before;
    before += n[i];
  }
}

// The expert of an item: the last whose first item is not behind it.
__device__ __forceinline__ int find_expert(const int* first, int E, int item, int lane) {
  int n = 0;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    n += __popcll(__ballot(e < E && first[e] <= item));
  }
  return n - 1;
}

template <typename Elem, LinearOp OP, typename S>
__global__ void __launch_bounds__(S::kThreads, 2)
linear_tile_kernel(moe_host::LinearArgs g) {
  constexpr bool TR = OP == kGradW, TC = OP != kForward;
  constexpr int BM = S::BM, BC = S::BC, KG = S::KG, MB = S::MB, CB = S::CB;
  typedef OperandTile<TR, BM> TileR;
  typedef OperandTile<TC, BC> TileC;
  static_assert(KG * TileR::kCopies % S::kWaves == 0 && KG * TileC::kCopies % S::kWaves == 0, "whole copies a wave");
  constexpr int NR = KG * TileR::kCopies / S::kWaves, NC = KG * TileC::kCopies / S::kWaves;
  __shared__ __attribute__((aligned(1024))) char lds[S::kLds];
  int* const first = reinterpret_cast<int*>(lds + S::kStage * S::kStages);

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  const int kg = wave / (S::WM * S::WC), wm = wave / S::WC % S::WM, wc = wave % S::WC;

  const bool gated = OP == kForward && g.act == MOE_ACT_SWIGLU;
  const int N = g.N, K = g.K;
  const int width_c = OP == kForward ? (gated ? N / 2 : N) : K;   // values of c of an output row
  const int step_c = gated ? BC / 2 : BC;                         // ... and of a tile
  const int tiles_c = (width_c + step_c - 1) / step_c;
  const int tiles_w = (N + BM - 1) / BM;                          // grad w: tiles of m
  int total;
  if constexpr (OP == kGradW) {
    total = g.E * tiles_w * tiles_c;
  } else {
    if (wave == 0) count_items<BM>(g, tiles_c, first, lane);
    __syncthreads();
    total = uniform(first[g.E]);
  }

  const int G = gridDim.x;
  for (int item = xcd_order(blockIdx.x, G); item < total; item += G) {
    // --- which tile
    int e, tiles_m, at;
    if constexpr (OP == kGradW) {
      tiles_m = tiles_w;
      e = item / (tiles_m * tiles_c);
      at = item - e * tiles_m * tiles_c;
    } else {
      e = uniform(find_expert(first, g.E, item, lane));
      at = item - uniform(first[e]);
    }
    const RowRange range = expert_rows(g, e);
    const int begin = uniform(range.begin), rows = uniform(range.end - range.begin);
    if constexpr (OP != kGradW) tiles_m = (rows + BM - 1) / BM;
    // tiles of m in groups of up to 8, c by c: a run of items is a block of both
    const int group = 8 * tiles_c, m_group = at / group;
    const int ms = min(8, tiles_m - m_group * 8), in_group = at - m_group * group;
    const int tc = in_group / ms, tm = m_group * 8 + in_group - tc * ms;
    const int m0 = tm * BM, c0 = tc * step_c;

    // --- where the operands are
    const int Q = OP == kForward ? K : OP == kGradX ? N : rows;
    const int steps = (Q + kStepQ * KG - 1) / (kStepQ * KG);
    const char* baseR;
    const char* baseC;
    uint32_t bytesR = 0, bytesC = 0;   // of the operands that are contiguous in q
    size_t ldR, ldC;                   // bytes a row in memory
    if constexpr (OP == kGradW) {
      ldR = (size_t)N * 2, ldC = (size_t)K * 2;
      baseR = static_cast<const char*>(g.rows_in) + (size_t)begin * ldR + m0 * 2;
      baseC = static_cast<const char*>(g.x) + (size_t)begin * ldC + c0 * 2;
    } else {
      ldR = (size_t)Q * 2, ldC = (size_t)K * 2;
      baseR = static_cast<const char*>(g.rows_in) + (size_t)(begin + m0) * ldR;
      bytesR = (uint32_t)(min(rows - m0, BM) * ldR);
      const char* w = static_cast<const char*>(g.w) + (size_t)e * N * ldC;
      if constexpr (OP == kForward) {
        baseC = w + (size_t)c0 * ldC;
        bytesC = (uint32_t)((size_t)(N - c0) * ldC);
      } else {
        baseC = w + (size_t)c0 * 2;
      }
    }
    baseR = uniform_ptr(baseR);
    baseC = uniform_ptr(baseC);
    // a lane's offset of each of its copies, but for the stage's
    uint32_t offR[NR], offC[NC];
#pragma unroll
    for (int j = 0; j < NR; j++) {
      const int id = j * S::kWaves + wave, sub = id / TileR::kCopies, i = id % TileR::kCopies;
      const int row = TileR::copy_row(i, lane) + (TR ? sub * kStepQ : 0);
      offR[j] = (uint32_t)(row * ldR) + TileR::copy_byte(i, lane) + (TR ? 0 : sub * 128);
    }
#pragma unroll
    for (int j = 0; j < NC; j++) {
      const int id = j * S::kWaves + wave, sub = id / TileC::kCopies, i = id % TileC::kCopies;
      int row = TileC::copy_row(i, lane) + (TC ? sub * kStepQ : 0);
      // gate and up rows alternate, 16 by 16, so that a wave has both of a column
      if (gated) row = (row / 32) * 16 + row % 16 + ((row / 16) % 2) * (N / 2);
      offC[j] = (uint32_t)(row * ldC) + TileC::copy_byte(i, lane) + (TC ? 0 : sub * 128);
    }

    auto copy = [&](int step) {
      char* const stage = lds + (step % S::kStages) * S::kStage;
      const int q0 = step * kStepQ * KG;
      const bool tail = q0 + kStepQ * KG > Q;
      const int left = min(Q - q0, kStepQ * KG);
      auto one = [&](auto tile, bool trans, int j, const char* base, uint32_t bytes, size_t ld, int skip, uint32_t off, int part) {
        typedef decltype(tile) T;
        const int id = j * S::kWaves + wave, sub = id / T::kCopies, i = id % T::kCopies;
        char* const dst = stage + sub * S::kSub + part + i * 1024;
        if (trans) {
          range_dma16(range_rsrc(base + (size_t)q0 * ld, (uint32_t)(left * ld) - skip), off, 0, dst);
        } else {
          const int q = q0 * 2 + sub * 128 + T::copy_byte(i, lane);
          range_dma16(range_rsrc(base, bytes), tail && q >= Q * 2 ? kOutside : off, q0 * 2, dst);
        }
      };
#pragma unroll
      for (int j = 0; j < NR; j++) one(TileR{}, TR, j, baseR, bytesR, ldR, m0 * 2, offR[j], 0);
#pragma unroll
      for (int j = 0; j < NC; j++) one(TileC{}, TC, j, baseC, bytesC, ldC, c0 * 2, offC[j], BM * 128);
    };

    f32x4 acc[CB][MB];
#pragma unroll
    for (int c = 0; c < CB; c++)
#pragma unroll
      for (int m = 0; m < MB; m++) acc[c][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float colsum[MB];   // grad w: sums of dy over the rows, the bias's gradient
#pragma unroll
    for (int m = 0; m < MB; m++) colsum[m] = 0.0f;
    const bool with_bias = OP == kGradW && g.dbias && tc == 0 && wc == 0;
    const bool busy = OP == kGradW || m0 + wm * MB * 16 < rows;   // whether the wave has rows

    if (steps > 0) copy(0);
    for (int step = 0; step < steps; step++) {
      wait_all();          // this stage's copies, and the LDS reads of the one before
      barrier_nofence();
      if (step + 1 < steps) copy(step + 1);
      if (busy) {
        const char* const stage = lds + (step % S::kStages) * S::kStage + kg * S::kSub;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          u32x4 a[CB], b[MB];
#pragma unroll
          for (int c = 0; c < CB; c++) a[c] = TileC::fragment(stage + BM * 128, wc * CB + c, h, lane);
#pragma unroll
          for (int m = 0; m < MB; m++) b[m] = TileR::fragment(stage, wm * MB + m, h, lane);
#pragma unroll
          for (int m = 0; m < MB; m++)
#pragma unroll
            for (int c = 0; c < CB; c++) acc[c][m] = Elem::mfma(a[c], b[m], acc[c][m]);
          if (with_bias) {
#pragma unroll
            for (int m = 0; m < MB; m++) {
              float v[8];
              Elem::Row::unpack(b[m], v);
#pragma unroll
              for (int i = 0; i < 8; i++) colsum[m] += v[i];
            }
          }
        }
      }
    }
    wait_all();
    barrier_nofence();   // the stages are free again

    // --- the groups' sums, in ascending order
    if constexpr (KG > 1) {
      f32x4* const part = reinterpret_cast<f32x4*>(lds);
      float* const part_sum = reinterpret_cast<float*>(lds + (KG - 1) * S::WM * S::WC * CB * MB * 1024);
      const int w = wave % (S::WM * S::WC);
      static_assert((KG - 1) * S::WM * S::WC * MB * (CB * 1024 + 256) <= S::kStage * S::kStages, "partial sums fit");
      if (kg > 0) {
#pragma unroll
        for (int c = 0; c < CB; c++)
#pragma unroll
          for (int m = 0; m < MB; m++)
            part[((((kg - 1) * S::WM * S::WC + w) * CB + c) * MB + m) * 64 + lane] = acc[c][m];
#pragma unroll
        for (int m = 0; m < MB; m++) part_sum[(((kg - 1) * S::WM * S::WC + w) * MB + m) * 64 + lane] = colsum[m];
      }
      __syncthreads();
      if (kg == 0) {
        for (int k = 0; k < KG - 1; k++) {
#pragma unroll
          for (int c = 0; c < CB; c++)
#pragma unroll
            for (int m = 0; m < MB; m++)
              acc[c][m] += part[(((k * S::WM * S::WC + w) * CB + c) * MB + m) * 64 + lane];
#pragma unroll
          for (int m = 0; m < MB; m++) colsum[m] += part_sum[((k * S::WM * S::WC + w) * MB + m) * 64 + lane];
        }
      }
      __syncthreads();
      if (kg > 0) continue;
    }

    // --- epilogue: lane holds c = 4 (lane / 16) + 0..3 of row lane % 16 of every block
    typedef typename Elem::Row::elem elem;
    const int lm = lane & 15, lc = 4 * (lane >> 4);
    if constexpr (OP == kGradW) {
#pragma unroll
      for (int m = 0; m < MB; m++) {
        const int n = m0 + (wm * MB + m) * 16 + lm;
        if (n >= N) continue;
        const size_t row = ((size_t)e * N + n) * K;
#pragma unroll
        for (int c = 0; c < CB; c++) {
          const int k = c0 + (wc * CB + c) * 16 + lc;
          if (k >= K) continue;
          if (g.out_fp32) {
            f32x4* const p = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + row + k);
            *p = g.accumulate ? *p + acc[c][m] : acc[c][m];
          } else {
            u32x2* const p = reinterpret_cast<u32x2*>(static_cast<elem*>(g.out) + row + k);
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (g.accumulate) Elem::unpack4(*p, v);
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] += acc[c][m][i];
            *p = Elem::pack4(v);
          }
        }
      }
      if (with_bias) {
#pragma unroll
        for (int m = 0; m < MB; m++) {
          float s = colsum[m];
          s += __shfl_xor(s, 16, 64);
          s += __shfl_xor(s, 32, 64);
          const int n = m0 + (wm * MB + m) * 16 + lm;
          if (lane >= 16 || n >= N) continue;
          const size_t at_n = (size_t)e * N + n;
          if (g.out_fp32) {
            float* const p = static_cast<float*>(g.dbias) + at_n;
            *p = g.accumulate ? *p + s : s;
          } else {
            elem* const p = static_cast<elem*>(g.dbias) + at_n;
            *p = Elem::round(g.accumulate ? Elem::widen(*p) + s : s);
          }
        }
      }
    } else {
      if (!busy) continue;
      if (gated) {
        if constexpr (OP == kForward) {
#pragma unroll
          for (int m = 0; m < MB; m++) {
            const int r = m0 + (wm * MB + m) * 16 + lm;
            if (r >= rows) continue;
            const size_t row = begin + r;
#pragma unroll
            for (int c = 0; c < CB / 2; c++) {
              const int n = c0 + (wc * CB / 2 + c) * 16 + lc;
              if (n >= width_c) continue;
              float gate[4], up[4], y[4];
#pragma unroll
              for (int i = 0; i < 4; i++) gate[i] = acc[2 * c][m][i], up[i] = acc[2 * c + 1][m][i];
              if (g.bias) {
                const elem* const b = static_cast<const elem*>(g.bias) + (size_t)e * N + n;
                float v[4];
                Elem::unpack4(*reinterpret_cast<const u32x2*>(b), v);
#pragma unroll
                for (int i = 0; i < 4; i++) gate[i] += v[i];
                Elem::unpack4(*reinterpret_cast<const u32x2*>(b + N / 2), v);
#pragma unroll
                for (int i = 0; i < 4; i++) up[i] += v[i];
              }
              if (g.z_out) {
                elem* const z = static_cast<elem*>(g.z_out) + row * N + n;
                *reinterpret_cast<u32x2*>(z) = Elem::pack4(gate);
                *reinterpret_cast<u32x2*>(z + N / 2) = Elem::pack4(up);
              }
#pragma unroll
              for (int i = 0; i < 4; i++) y[i] = silu(gate[i]) * up[i];
              const size_t o = row * width_c + n;
              if (g.residual) {
                float v[4];
                Elem::unpack4(*reinterpret_cast<const u32x2*>(static_cast<const elem*>(g.residual) + o), v);
#pragma unroll
                for (int i = 0; i < 4; i++) y[i] += v[i];
              }
              *reinterpret_cast<u32x2*>(static_cast<elem*>(g.out) + o) = Elem::pack4(y);
            }
          }
        }
        continue;
      }
#pragma unroll
      for (int m = 0; m < MB; m++) {
        const int r = m0 + (wm * MB + m) * 16 + lm;
        if (r >= rows) continue;
        const size_t row = begin + r;
#pragma unroll
        for (int c = 0; c < CB; c++) {
          const int n = c0 + (wc * CB + c) * 16 + lc;
          if (n >= width_c) continue;
          float v[4], y[4];
#pragma unroll
          for (int i = 0; i < 4; i++) v[i] = acc[c][m][i];
          const size_t o = row * width_c + n;
          if constexpr (OP == kForward) {
            if (g.bias) {
              float b[4];
              Elem::unpack4(*reinterpret_cast<const u32x2*>(static_cast<const elem*>(g.bias) + (size_t)e * N + n), b);
#pragma unroll
              for (int i = 0; i < 4; i++) v[i] += b[i];
            }
            if (g.z_out) *reinterpret_cast<u32x2*>(static_cast<elem*>(g.z_out) + o) = Elem::pack4(v);
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = activate(v[i], g.act);
            if (g.residual) {
              float b[4];
              Elem::unpack4(*reinterpret_cast<const u32x2*>(static_cast<const elem*>(g.residual) + o), b);
#pragma unroll
              for (int i = 0; i < 4; i++) y[i] += b[i];
            }
            *reinterpret_cast<u32x2*>(static_cast<elem*>(g.out) + o) = Elem::pack4(y);
          } else if (g.act == MOE_ACT_SWIGLU) {
            const size_t oz = row * 2 * width_c + n;
            const elem* const z = static_cast<const elem*>(g.z_in) + oz;
            float gate[4], up[4];
            Elem::unpack4(*reinterpret_cast<const u32x2*>(z), gate);
            Elem::unpack4(*reinterpret_cast<const u32x2*>(z + width_c), up);
#pragma unroll
            for (int i = 0; i < 4; i++) {
              y[i] = v[i] * silu(gate[i]);
              v[i] = v[i] * up[i] * silu_slope(gate[i]);
            }
            elem* const out = static_cast<elem*>(g.out) + oz;
            *reinterpret_cast<u32x2*>(out) = Elem::pack4(v);
            *reinterpret_cast<u32x2*>(out + width_c) = Elem::pack4(y);
          } else {
            if (g.act != MOE_ACT_NONE) {
              float z[4];
              Elem::unpack4(*reinterpret_cast<const u32x2*>(static_cast<const elem*>(g.z_in) + o), z);
#pragma unroll
              for (int i = 0; i < 4; i++) v[i] *= act_slope(z[i], g.act);
            }
            *reinterpret_cast<u32x2*>(static_cast<elem*>(g.out) + o) = Elem::pack4(v);
          }
        }
      }
    }
  }
}

// A persistent grid for at most `items` items, `occupancy` workgroups a CU.
template <typename Elem, LinearOp OP, typename S>
static hipError_t launch_linear_tile(const moe_host::LinearArgs& a, long items, int cus, hipStream_t s) {
  constexpr int kOccupancy = S::kLds <= 80 * 1024 && S::kThreads <= 256 ? 2 : 1;
  const long grid = items < (long)cus * kOccupancy ? items : (long)cus * kOccupancy;
  if (grid <= 0) return hipSuccess;
  hipLaunchKernelGGL((linear_tile_kernel<Elem, OP, S>), dim3((unsigned)grid), dim3(S::kThreads), 0, s, a);
  return hipGetLastError();
}

// Tiles of BM rows that `rows` rows of E experts can need at most.
static inline long max_tiles(const moe_host::LinearArgs& a, int BM) {
  return a.expert_offsets ? a.rows / BM + (a.rows < a.E ? a.rows : a.E) : (a.rows + BM - 1) / BM;
}

}  // namespace moe
