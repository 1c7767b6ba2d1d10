// Forward products of rows with their experts' matrices, and the gradient of
// the rows (linear_tile.h).
#include "linear_tile.h"

namespace moe {

typedef LinearShape<256, 256, 2, 4, 1, 2> Tile256;
typedef LinearShape<128, 128, 2, 2, 1, 2> Tile128;

// Rows of an expert that has any, were they spread evenly.
static int mean_rows(const moe_host::LinearArgs& a) {
  return a.expert_offsets ? (a.rows + a.E - 1) / a.E : a.rows;
}
static long blocks(long n, long size) { return (n + size - 1) / size; }

// Whether tiles of 256 x 256, one workgroup a CU, take fewer rounds of the chip
// than those of 128 x 128, two a CU, which do 0.8 of their work in the same time.
static bool large_tiles(const moe_host::LinearArgs& a, int width, int cus) {
  const int groups = a.expert_offsets ? (a.rows < a.E ? a.rows : a.E) : 1, mean = mean_rows(a);
  const long large = groups * blocks(mean, 256) * blocks(width, 256), small = groups * blocks(mean, 128) * blocks(width, 128);
  return blocks(large, cus) * 1.6 <= blocks(small, 2 * cus);
}

template <typename Elem>
static hipError_t forward(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  const bool gated = a.act == MOE_ACT_SWIGLU;
  if (large_tiles(a, a.N, cus)) {
    const long tiles_c = gated ? blocks(a.N / 2, 128) : blocks(a.N, 256);
    return launch_linear_tile<Elem, kForward, Tile256>(a, max_tiles(a, 256) * tiles_c, cus, s);
  }
  const long tiles_c = gated ? blocks(a.N / 2, 64) : blocks(a.N, 128);
  return launch_linear_tile<Elem, kForward, Tile128>(a, max_tiles(a, 128) * tiles_c, cus, s);
}

template <typename Elem>
static hipError_t grad_x(moe_host::LinearArgs a, int cus, hipStream_t s) {
  const size_t z = a.act == MOE_ACT_NONE ? 1 : a.act == MOE_ACT_SWIGLU ? 4 : 2;   // dx, and z as wide
  a.stream_out = past_caches(2 * ((size_t)a.rows * (a.N + z * a.K) + (size_t)a.E * a.N * a.K));
  if (large_tiles(a, a.K, cus))
    return launch_linear_tile<Elem, kGradX, Tile256>(a, max_tiles(a, 256) * blocks(a.K, 256), cus, s);
  return launch_linear_tile<Elem, kGradX, Tile128>(a, max_tiles(a, 128) * blocks(a.K, 128), cus, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  // few rows an expert: the weights' stream, on as many columns a workgroup as leave every CU one
  const int mean = moe::mean_rows(a);
  if (mean <= 32) {
    const int groups = a.expert_offsets ? (a.rows < a.E ? a.rows : a.E) : 1, mb = mean <= 16 ? 1 : 2;
    const int least = a.act == MOE_ACT_SWIGLU ? 2 : 1;
    int nb = mb == 2 ? 2 : 4;
    while (nb > least && groups * moe::blocks(a.N, 16 * nb) < cus) nb /= 2;
    return launch_linear_stream(a, row_type, nb, nb == 1 ? 1 : mb, cus, s);
  }
  return row_type == MOE_ROW_BF16 ? moe::forward<moe::ElemBf16>(a, cus, s) : moe::forward<moe::ElemFp16>(a, cus, s);
}

hipError_t launch_linear_grad_x(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_x<moe::ElemBf16>(a, cus, s) : moe::grad_x<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
