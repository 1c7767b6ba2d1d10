// Forward products of rows with their experts' matrices (linear_tile.h; few rows
// an expert: linear_stream.hip).
#include "linear_tile.h"

namespace moe {

template <typename Elem>
static hipError_t forward(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  return with_shape(used_groups(a), mean_rows(a), a.expert_offsets != nullptr, a.N, a.K, cus, [&](auto shape) {
    typedef decltype(shape) S;
    const long tiles_c = a.act == MOE_ACT_SWIGLU ? blocks(a.N / 2, S::BC / 2) : blocks(a.N, S::BC);
    return launch_linear_tile<Elem, kForward, S>(a, max_tiles(a, S::BM) * tiles_c, cus, s);
  });
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  // few rows an expert: the weights' stream.  Of items of 4, 2 or 1 blocks of weight
  // rows those that take least: the rounds over the CUs, times the blocks and a
  // third of one for the rows' copies and the waves' meeting (2 experts of 28672 x
  // 4096, one row each: 94 us on 4 blocks, 3.5 rounds, 81 on 2, 7 rounds)
  const int mean = moe::mean_rows(a);
  if (mean <= 32) {
    const int mb = mean <= 16 ? 1 : 2, least = mb == 2 || a.act == MOE_ACT_SWIGLU ? 2 : 1;
    int nb = 2;
    long best = -1;
    for (int n = mb == 2 ? 2 : 4; n >= least; n /= 2) {
      const long cost = moe::blocks(moe::used_groups(a) * moe::blocks(a.N, 16 * n), cus) * (3 * n + 1);
      if (best < 0 || cost < best) best = cost, nb = n;
    }
    return launch_linear_stream(a, row_type, nb, mb, cus, s);
  }
  return row_type == MOE_ROW_BF16 ? moe::forward<moe::ElemBf16>(a, cus, s) : moe::forward<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
