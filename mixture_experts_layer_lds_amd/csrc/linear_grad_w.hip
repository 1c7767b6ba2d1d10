// Gradient of the experts' matrices and biases (linear_tile.h).
#include "linear_tile.h"

namespace moe {

typedef LinearShape<256, 256, 2, 4, 1, 2> Tile128;

template <typename Elem>
static hipError_t grad_w(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  const long items = (long)a.E * ((a.N + 255) / 256) * ((a.K + 255) / 256);
  return a.dbias ? launch_linear_tile<Elem, kGradW, Tile128, true>(a, items, cus, s)
                 : launch_linear_tile<Elem, kGradW, Tile128, false>(a, items, cus, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear_grad_w(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_w<moe::ElemBf16>(a, cus, s) : moe::grad_w<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
