// Gradient of the experts' matrices and biases (linear_tile.h).
#include "linear_tile.h"

namespace moe {

template <typename Elem>
static hipError_t grad_w(moe_host::LinearArgs a, int cus, hipStream_t s) {
  a.stream_out = past_caches(2 * (size_t)a.rows * (a.N + a.K) + (size_t)a.E * a.N * a.K * (a.out_fp32 ? 4 : 2));
  return with_shape<false>(grad_w_tile(sizes_of(a), cus), [&](auto shape) {
    typedef decltype(shape) S;
    const long items = a.E * blocks(a.N, S::BM) * blocks(a.K, S::BC);
    return a.dbias ? launch_linear_tile<Elem, kGradW, S, true>(a, items, cus, s)
                   : launch_linear_tile<Elem, kGradW, S, false>(a, items, cus, s);
  });
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear_grad_w(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_w<moe::ElemBf16>(a, cus, s) : moe::grad_w<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
