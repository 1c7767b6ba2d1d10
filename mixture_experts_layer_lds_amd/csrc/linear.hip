// Forward products of rows with their experts' matrices (linear_tile.h; few rows
// an expert: linear_stream.hip).
#include "linear_tile.h"

namespace moe {

template <typename Elem>
static hipError_t forward(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  return with_shape<true>(forward_tile(sizes_of(a), cus), [&](auto shape) {
    typedef decltype(shape) S;
    const long tiles_c = a.act == MOE_ACT_SWIGLU ? blocks(a.N / 2, S::BC / 2) : blocks(a.N, S::BC);
    return launch_linear_tile<Elem, kForward, S>(a, max_tiles(a, S::BM) * tiles_c, cus, s);
  });
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  const moe::StreamItem few = moe::stream_item(moe::sizes_of(a), cus);
  if (few.nb) return launch_linear_stream(a, row_type, few.nb, few.mb, cus, s);
  return row_type == MOE_ROW_BF16 ? moe::forward<moe::ElemBf16>(a, cus, s) : moe::forward<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
