// The forward product (linear.h) of few rows per expert: bound by the stream
// of the weights.
//
// An item is NB blocks of 16 weight rows (SwiGLU: gate and up rows in turn) and a
// tile of 16 MB rows.  The four waves of a workgroup, one a CU, take the item's
// chunks of 64 q in turn and add their sums at the end.  Every wave has a ring
// of NS chunks of its own in LDS, which direct copies fill ahead of the
// multiplications, on from item to item, and waits for its own copies alone:
// the waves meet once an item.  NS is what LDS holds, so that a CU has 48 to 96 KiB
// of weights on their way.
//
// Measured (us; TB/s of weights): one row of 7168 with 4096 gate and up rows 12.5
// (4.7; on the 128-row tiles 68; its first weights arrive some 3 us after the start),
// one token on eight experts of the same 82 (5.7), 16 tokens 295 (6.3), two experts
// of 28672 x 4096 at one row 81 (5.8).  The read of a large buffer reaches 7.0.
#include "linear_tile.h"

namespace moe {

constexpr int kStreamWaves = 4;

template <int NB_, int MB_, int NS_>
struct StreamShape {
  static constexpr int NB = NB_, MB = MB_, NS = NS_;
  static constexpr int kSlot = (NB + MB) * 2048;
  static constexpr int kRing = NS * kSlot;
  // sums of a wave: rows of 16 NB, padded by four against bank conflicts
  static constexpr int kPitch = NB * 16 + 4;
  static constexpr int kPart = MB * 16 * kPitch * 4;
  static constexpr int kLds = kStreamWaves * (kRing + 2 * kPart) + 3 * 4 * (kMaxExperts + 1);
  static_assert(kLds <= 160 * 1024, "one workgroup's LDS");
};

template <typename Elem, typename S>
__global__ void __launch_bounds__(kStreamWaves * 64, 1)
linear_stream_kernel(moe_host::LinearArgs g) {
  constexpr int NB = S::NB, MB = S::MB, NS = S::NS, BM = MB * 16;
  typedef OperandTile<false, 16> Block;
  constexpr int COPIES = (NB + MB) * Block::kCopies;
  __shared__ __attribute__((aligned(1024))) char lds[S::kLds];
  Experts* const experts = reinterpret_cast<Experts*>(lds + kStreamWaves * (S::kRing + 2 * S::kPart));
  float* const parts = reinterpret_cast<float*>(lds + kStreamWaves * S::kRing);

  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6);
  char* const ring = lds + wave * S::kRing;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(lds_void*)lds + wave * S::kRing;
  const bool gated = g.act == MOE_ACT_SWIGLU;
  const int N = g.N, K = g.K;
  const int width = gated ? N / 2 : N, step_c = gated ? NB * 8 : NB * 16;
  const int tiles_c = (width + step_c - 1) / step_c;
  if (wave == 0) count_items(g, experts, lane, [&](int rows) { return (rows + BM - 1) / BM * tiles_c; });
  __syncthreads();
  const int total = uniform(experts->first[g.E]);
  const int G = gridDim.x;
  const int chunks = (K + kStepQ - 1) / kStepQ;
  const int mine = (chunks - wave + kStreamWaves - 1) / kStreamWaves;   // this wave's, of every item

  struct Tile {
    int e, begin, rows, c0;
  };
  // an expert's tiles of m take a tile of its weights one after another
  auto decode = [&](int item) {
    Tile t;
    t.e = find_expert(experts, g.E, item, lane);
    const int at = item - uniform(experts->first[t.e]);
    const int begin = uniform(experts->rows[t.e].begin), rows = uniform(experts->rows[t.e].end) - begin;
    const int tiles_m = (rows + BM - 1) / BM, tc = at / tiles_m, m0 = (at - tc * tiles_m) * BM;
    t.begin = begin + m0;
    t.rows = min(rows - m0, BM);
    t.c0 = tc * step_c;
    return t;
  };

  // --- the copies: of chunk `from_chunk` (counted in the wave's own) of item from_item
  int from_item = 0, from_chunk = 0;
  const char* base_x = nullptr;
  const char* base_w = nullptr;
  uint32_t bytes_x = 0, bytes_w = 0;
  uint32_t off_w[NB * Block::kCopies], off_x[MB * Block::kCopies];
  const size_t ld = (size_t)K * 2;
  const int byte = Block::copy_byte(0, lane);   // the same in every copy: eight rows each
#pragma unroll
  for (int j = 0; j < MB * Block::kCopies; j++) off_x[j] = (uint32_t)((j * 8 + lane / 8) * ld) + byte;
#pragma unroll
  for (int j = 0; j < NB * Block::kCopies; j++) {
    const int b = j / Block::kCopies, r = Block::copy_row(j % Block::kCopies, lane);
    const int row = gated ? b / 2 * 16 + r + (b % 2) * (N / 2) : b * 16 + r;
    off_w[j] = (uint32_t)(row * ld) + byte;
  }
  auto enter = [&](int item) {
    from_item = item;
    from_chunk = 0;
    if (item >= total) return;
    const Tile t = decode(item);
    base_x = static_cast<const char*>(g.rows_in) + (size_t)t.begin * ld;
    bytes_x = (uint32_t)(t.rows * ld);
    base_w = static_cast<const char*>(g.w) + ((size_t)t.e * N + t.c0) * ld;
    bytes_w = (uint32_t)((size_t)(N - t.c0) * ld);
  };
  // The copies of the next chunk into the ring's slot `slot`; behind the last one copies of nothing.
  auto copy = [&](int slot) {
    if (from_chunk == mine) enter(from_item + G);
    const bool any = from_item < total;
    const auto rx = range_rsrc(uniform_ptr(base_x), uniform(any ? bytes_x : 0));
    const auto rw = range_rsrc(uniform_ptr(base_w), uniform(any ? bytes_w : 0));
    const int q2 = any ? (from_chunk * kStreamWaves + wave) * kStepQ * 2 : 0;   // within the range, also where that is nothing
    const bool inside = q2 + byte < K * 2;   // no q behind the end
    char* const at = ring + slot * S::kSlot;
#pragma unroll
    for (int j = 0; j < NB * Block::kCopies; j++) range_dma16(rw, inside ? off_w[j] : kOutside, q2, at + j * 1024);
#pragma unroll
    for (int j = 0; j < MB * Block::kCopies; j++) range_dma16(rx, inside ? off_x[j] : kOutside, q2, at + NB * 2048 + j * 1024);
    from_chunk++;
  };

  int item = xcd_order(blockIdx.x, G);
  if (item >= total) return;
  if (mine > 0) {
    enter(item);
#pragma unroll
    for (int s = 0; s < NS; s++) copy(s);
  }
  const uint32_t place = Block::lane_place(0, lane);
  int slot = 0;
  for (int turn = 0; item < total; item += G, turn ^= 1) {
    f32x4 acc[NB][MB];
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int m = 0; m < MB; m++) acc[b][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < mine; i++) {
      wait_but<(NS - 1) * COPIES>();
      __asm__ volatile("" ::: "memory");
      u32x4 w[2][NB], x[2][MB];
      const uint32_t at = ring0 + slot * S::kSlot + place;
#pragma unroll
      for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int b = 0; b < NB; b++) w[h][b] = Block::fragment(at, b, h);
#pragma unroll
        for (int m = 0; m < MB; m++) x[h][m] = Block::fragment(at, NB + m, h);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);   // the slot is read (lgkmcnt alone)
      __asm__ volatile("" ::: "memory");
      copy(slot);
      slot = slot == NS - 1 ? 0 : slot + 1;
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
          for (int b = 0; b < NB; b++) acc[b][m] = Elem::mfma(w[h][b], x[h][m], acc[b][m]);
    }
    // --- the waves' sums, in ascending order; two sets of places, so that one meeting is enough
    float* const part = parts + turn * (kStreamWaves * S::kPart / 4);
#pragma unroll
    for (int b = 0; b < NB; b++)
#pragma unroll
      for (int m = 0; m < MB; m++)
        *reinterpret_cast<f32x4*>(part + wave * (S::kPart / 4) + (m * 16 + (lane & 15)) * S::kPitch + b * 16 + 4 * (lane >> 4)) = acc[b][m];
    __builtin_amdgcn_s_waitcnt(0xC07F);
    barrier_nofence();
    const Tile d = decode(item);
    auto sum8 = [&](int row, int c, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = 0.0f;
#pragma unroll
      for (int q = 0; q < kStreamWaves; q++) {
        const float* const p = part + q * (S::kPart / 4) + row * S::kPitch + c;
        const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] += a[i], v[4 + i] += b[i];
      }
    };
    const int per_row = step_c / 8;
    for (int u = threadIdx.x; u < BM * per_row; u += kStreamWaves * 64) {
      const int row = u / per_row, c = u % per_row * 8, n = d.c0 + c;
      if (row >= d.rows || n >= width) continue;
      float v[8];
      if (gated) {
        float up[8];
        sum8(row, c / 16 * 32 + c % 16, v);
        sum8(row, c / 16 * 32 + 16 + c % 16, up);
        forward_out<Elem>(g, d.e, (size_t)d.begin + row, n, v, up);
      } else {
        sum8(row, c, v);
        forward_out<Elem>(g, d.e, (size_t)d.begin + row, n, v);
      }
    }
  }
  wait_all();   // no copy may reach LDS that is another workgroup's by then
}

template <typename Elem, typename S>
static hipError_t launch_stream(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  const int width = a.act == MOE_ACT_SWIGLU ? a.N / 2 : a.N, step = a.act == MOE_ACT_SWIGLU ? S::NB * 8 : S::NB * 16;
  const long items = max_tiles(a, S::MB * 16) * ((width + step - 1) / step);
  const long grid = items < cus ? items : cus;
  hipLaunchKernelGGL((linear_stream_kernel<Elem, S>), dim3((unsigned)grid), dim3(kStreamWaves * 64), 0, s, a);
  return hipGetLastError();
}

template <typename Elem>
static hipError_t stream(const moe_host::LinearArgs& a, int nb, int mb, int cus, hipStream_t s) {
  if (mb == 2) return launch_stream<Elem, StreamShape<2, 2, 3>>(a, cus, s);
  if (nb == 1) return launch_stream<Elem, StreamShape<1, 1, 7>>(a, cus, s);
  if (nb == 2) return launch_stream<Elem, StreamShape<2, 1, 5>>(a, cus, s);
  return launch_stream<Elem, StreamShape<4, 1, 3>>(a, cus, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear_stream(const LinearArgs& a, int row_type, int nb, int mb, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::stream<moe::ElemBf16>(a, nb, mb, cus, s) : moe::stream<moe::ElemFp16>(a, nb, mb, cus, s);
}

}  // namespace moe_host
