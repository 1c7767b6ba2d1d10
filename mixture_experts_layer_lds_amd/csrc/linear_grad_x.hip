// Gradient of the rows, or of the pre-activation that they come from (linear_tile.h).
#include "linear_tile.h"

namespace moe {

template <typename Elem>
static hipError_t grad_x(moe_host::LinearArgs a, int cus, hipStream_t s) {
  const size_t z = a.act == MOE_ACT_NONE ? 1 : a.act == MOE_ACT_SWIGLU ? 4 : 2;   // dx, and z as wide
  a.stream_out = past_caches(2 * ((size_t)a.rows * (a.N + z * a.K) + (size_t)a.E * a.N * a.K));
  return with_shape<true>(grad_x_tile(sizes_of(a), cus), [&](auto shape) {
    typedef decltype(shape) S;
    return launch_linear_tile<Elem, kGradX, S>(a, max_tiles(a, S::BM) * blocks(a.K, S::BC), cus, s);
  });
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear_grad_x(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_x<moe::ElemBf16>(a, cus, s) : moe::grad_x<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
