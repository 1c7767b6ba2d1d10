// Forward products of rows with their experts' matrices (linear_tile.h; few rows
// an expert: linear_stream.hip).
#include "linear_tile.h"

namespace moe {

template <typename Elem>
static hipError_t forward(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  return with_shape<true>(used_groups(a), mean_rows(a), a.expert_offsets != nullptr, a.N, a.K, cus, [&](auto shape) {
    typedef decltype(shape) S;
    const long tiles_c = a.act == MOE_ACT_SWIGLU ? blocks(a.N / 2, S::BC / 2) : blocks(a.N, S::BC);
    return launch_linear_tile<Elem, kForward, S>(a, max_tiles(a, S::BM) * tiles_c, cus, s);
  });
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  // Few rows an expert: the weights' stream, on tiles of 16 or 32 rows.  Experts'
  // rows spread, and one with a row more than the tile reads its weights again, so
  // theirs go to half the rows that plain ones do (us, gate-up and down of the layer,
  // on 16, on 32 and on the large tiles: 8 of 32 experts of 7168 x 2048, 64 tokens, 16
  // rows an expert 337 + 176, 312 + 175, 309 + 220; 128 tokens - , 470 + 214, 313 + 223;
  // 64 skewed experts of 3584 x 640, 128 tokens 110 + 63, 108 + 69, 138 + 58).
  // Of items of 4, 2 or 1 blocks of weight rows those that take least: the rounds over
  // the CUs, times the blocks and a third of one for the rows' copies and the waves'
  // meeting (2 experts of 28672 x 4096, one row each: 94 us on 4 blocks, 3.5 rounds, 81
  // on 2, 7 rounds)
  const int mean = moe::mean_rows(a), of_one = a.expert_offsets ? 8 : 16;
  if (mean <= 2 * of_one) {
    const int mb = mean <= of_one ? 1 : 2, least = mb == 2 || a.act == MOE_ACT_SWIGLU ? 2 : 1;
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
