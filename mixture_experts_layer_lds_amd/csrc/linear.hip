// Forward products of rows with their experts' matrices, and the gradient of
// the rows (linear_tile.h).
#include "linear_tile.h"

namespace moe {

typedef LinearShape<256, 256, 2, 4, 1, 2> Tile128;

template <typename Elem>
static hipError_t forward(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  const bool gated = a.act == MOE_ACT_SWIGLU;
  const long tiles_c = gated ? (a.N / 2 + 127) / 128 : (a.N + 255) / 256;
  return launch_linear_tile<Elem, kForward, Tile128>(a, max_tiles(a, 256) * tiles_c, cus, s);
}

template <typename Elem>
static hipError_t grad_x(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  return launch_linear_tile<Elem, kGradX, Tile128>(a, max_tiles(a, 256) * ((a.K + 255) / 256), cus, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::forward<moe::ElemBf16>(a, cus, s) : moe::forward<moe::ElemFp16>(a, cus, s);
}

hipError_t launch_linear_grad_x(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_x<moe::ElemBf16>(a, cus, s) : moe::grad_x<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
