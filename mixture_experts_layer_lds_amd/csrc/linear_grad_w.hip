// Gradient of the experts' matrices and biases (linear_tile.h).
#include "linear_tile.h"

namespace moe {

typedef LinearShape<256, 256, 2, 4, 1, 2> Tile256;
typedef LinearShape<128, 128, 2, 2, 1, 2> Tile128;

template <typename Elem, typename S>
static hipError_t grad_w(const moe_host::LinearArgs& a, int cus, hipStream_t s) {
  const long items = (long)a.E * ((a.N + S::BM - 1) / S::BM) * ((a.K + S::BC - 1) / S::BC);
  return a.dbias ? launch_linear_tile<Elem, kGradW, S, true>(a, items, cus, s)
                 : launch_linear_tile<Elem, kGradW, S, false>(a, items, cus, s);
}

template <typename Elem>
static hipError_t grad_w(moe_host::LinearArgs a, int cus, hipStream_t s) {
  a.stream_out = past_caches(2 * (size_t)a.rows * (a.N + a.K) + (size_t)a.E * a.N * a.K * (a.out_fp32 ? 4 : 2));
  auto blocks = [](long n, long size) { return (n + size - 1) / size; };
  const long large = a.E * blocks(a.N, 256) * blocks(a.K, 256), small = a.E * blocks(a.N, 128) * blocks(a.K, 128);
  return blocks(large, cus) * 1.6 <= blocks(small, 2 * cus) ? grad_w<Elem, Tile256>(a, cus, s) : grad_w<Elem, Tile128>(a, cus, s);
}

}  // namespace moe

namespace moe_host {

hipError_t launch_linear_grad_w(const LinearArgs& a, int row_type, int cus, hipStream_t s) {
  return row_type == MOE_ROW_BF16 ? moe::grad_w<moe::ElemBf16>(a, cus, s) : moe::grad_w<moe::ElemFp16>(a, cus, s);
}

}  // namespace moe_host
