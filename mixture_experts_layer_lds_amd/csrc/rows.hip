// Token rows to expert order and back, and their gradients (HPC-Ops x SGLang
// blog, section "MoE", routing & index build: the route index names, for
// every token-expert pair, its row in the expert-sorted order).
//
// Pair p = t * k + j stands at sorted row r = pair_pos[p] when its id is
// valid (r < expert_offsets[E]):
//   to experts   rows[r] = w[p] tokens[t]
//   to tokens    tokens[t] = sum_j w[p] rows[r]
// Each is the other's gradient with respect to the rows; the gradient of
// the weights is dw[p] = <rows[r], tokens[t]>, with dw[p] = 0 for a dropped
// pair.  All of them are bound by the rows' bytes, so every kernel reads
// each row once: a thread holds 16 bytes of its token in registers and goes
// through the token's k pairs.  Sums run in fp32 in ascending j and are
// rounded once; rows behind the last valid one are not written.
//
// Measured: 8192 tokens of 7168 bf16 values, top-8, to experts 187 us (5.7
// TB/s of rows read and written), to tokens 192 (5.5), the gradients with the
// weights' 202 (to tokens, 5.8) and 392 (to experts, which writes the rows it
// also reads, 5.1); the router's gradient of 8192 tokens by 256 experts 7.7.
//
// A position outside [0, valid) counts as dropped, so a routing buffer that
// does not belong to these sizes cannot lead a row access out of bounds.
#include "rows.h"

namespace moe {

constexpr int kMoveThreads = 256;

// The k pairs of token t: sorted row (-1: dropped) and weight.
template <int KM>
__device__ __forceinline__ void pair_rows(const moe_host::RowMoveArgs& g, int t, int (&row)[KM], float (&w)[KM]) {
  const int valid = min(g.expert_offsets[g.E], g.T * g.k);
#pragma unroll
  for (int j = 0; j < KM; j++) {
    const int p = t * g.k + (j < g.k ? j : g.k - 1);
    const int r = g.pair_pos[p];
    w[j] = g.w ? g.w[p] : 1.0f;
    row[j] = j < g.k && (unsigned)r < (unsigned)valid ? r : -1;
  }
}

template <typename R, int KM>
__global__ void __launch_bounds__(kMoveThreads)
rows_to_experts_kernel(moe_host::RowMoveArgs g) {
  typedef typename R::elem elem;
  constexpr int N = R::kVec;
  const int t = blockIdx.x;
  const int c = (blockIdx.y * kMoveThreads + threadIdx.x) * N;
  if (c >= g.H) return;
  float v[N];
  row_load<R>(static_cast<const elem*>(g.tokens) + (size_t)t * g.H + c, v);
  int row[KM];
  float w[KM];
  pair_rows<KM>(g, t, row, w);
  elem* out = static_cast<elem*>(g.out) + c;
#pragma unroll
  for (int j = 0; j < KM; j++) {
    if (row[j] < 0) continue;
    float o[N];
#pragma unroll
    for (int i = 0; i < N; i++) o[i] = w[j] * v[i];
    __builtin_nontemporal_store(R::pack(o), reinterpret_cast<u32x4*>(out + (size_t)row[j] * g.H));
  }
}

// O: the type of the token rows (the rows' own, or bf16 for fp32 rows).
template <typename R, typename O, int KM>
__global__ void __launch_bounds__(kMoveThreads)
rows_to_tokens_kernel(moe_host::RowMoveArgs g) {
  typedef typename R::elem elem;
  constexpr int N = R::kVec;
  const int t = blockIdx.x;
  const int c = (blockIdx.y * kMoveThreads + threadIdx.x) * N;
  if (c >= g.H) return;
  int row[KM];
  float w[KM];
  pair_rows<KM>(g, t, row, w);
  const elem* rows = static_cast<const elem*>(g.rows) + c;
  // every row's load ahead of the first use; a dropped pair's is of row 0 and
  // takes no part (a load under a condition would wait for the ones before it)
  u32x4 raw[KM];
#pragma unroll
  for (int j = 0; j < KM; j++)
    raw[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(rows + (size_t)max(row[j], 0) * g.H));
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; i++) acc[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < KM; j++) {
    float v[N];
    R::unpack(raw[j], v);
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = row[j] < 0 ? acc[i] : acc[i] + w[j] * v[i];
  }
  typename O::elem* out = static_cast<typename O::elem*>(g.out) + (size_t)t * g.H + c;
  if constexpr (O::kVec == N) row_store<O>(out, acc);
  else *reinterpret_cast<u32x2*>(out) = u32x2{bf16_pair(acc[0], acc[1]), bf16_pair(acc[2], acc[3])};
}

// The gradients with the weights': WPT waves a token.  TO_TOKENS (the
// gradient of dispatch): out[t] = sum_j w rows[r]; else (of combine)
// out[r] = w tokens[t].  Both: dw[p] = <rows[r], tokens[t]>, a lane's columns
// in ascending order, then over the lanes and waves.
template <typename R, int KM, int WPT, bool TO_TOKENS>
__global__ void __launch_bounds__(WPT < 4 ? kMoveThreads : WPT * 64)
rows_grad_kernel(moe_host::RowMoveArgs g) {
  typedef typename R::elem elem;
  constexpr int N = R::kVec;
  constexpr int TPB = WPT < 4 ? 4 / WPT : 1;   // tokens a workgroup
  __shared__ float part[WPT * TPB][KM];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t = blockIdx.x * TPB + wave / WPT;   // waves past the last token have no columns
  const int H = t < g.T ? g.H : 0;
  int row[KM];
  float w[KM], dot[KM];
  pair_rows<KM>(g, min(t, g.T - 1), row, w);
#pragma unroll
  for (int j = 0; j < KM; j++) dot[j] = 0.0f;
  const elem* rows = static_cast<const elem*>(g.rows);
  elem* out = static_cast<elem*>(g.out);
  for (int c = ((wave % WPT) * 64 + lane) * N; c < H; c += WPT * 64 * N) {
    u32x4 raw[KM];
#pragma unroll
    for (int j = 0; j < KM; j++)
      raw[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(rows + (size_t)max(row[j], 0) * g.H + c));
    float x[N], acc[N];
    row_load<R>(static_cast<const elem*>(g.tokens) + (size_t)t * g.H + c, x);
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < KM; j++) {
      if (row[j] < 0) continue;
      float v[N];
      R::unpack(raw[j], v);
#pragma unroll
      for (int i = 0; i < N; i++) {
        dot[j] += v[i] * x[i];
        if constexpr (TO_TOKENS) acc[i] += w[j] * v[i];
        else v[i] = w[j] * x[i];
      }
      if constexpr (!TO_TOKENS)
        __builtin_nontemporal_store(R::pack(v), reinterpret_cast<u32x4*>(out + (size_t)row[j] * g.H + c));
    }
    if constexpr (TO_TOKENS) row_store<R>(out + (size_t)t * g.H + c, acc);
  }
#pragma unroll
  for (int j = 0; j < KM; j++)
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot[j] += __shfl_xor(dot[j], o, 64);
  if constexpr (WPT > 1) {
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < KM; j++) part[wave][j] = dot[j];
    }
    __syncthreads();
    const int j = (wave % WPT) * 64 + lane;   // of the token's threads
    if (t < g.T && j < g.k) {
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < WPT; q++) s += part[wave / WPT * WPT + q][j];
      g.dw[(size_t)t * g.k + j] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < KM; j++)
      if (lane == 0 && t < g.T && j < g.k) g.dw[(size_t)t * g.k + j] = dot[j];
  }
}

// d(logits) of the router's softmax top-k (router.hip) from d(topk_w), a wave
// a token.  With p the softmax over the E scores and s = sum_j w_j dw_j over
// the token's k chosen experts:
//   renormalised   dl[e] = w_j (dw_j - s) for the chosen e = e_j, else 0
//   otherwise      dl[e] = [e = e_j] w_j dw_j - p[e] s
// The n_shared columns behind the k have constant weights and pass no
// gradient.  The scores and their gradient are read and written once.
template <bool RENORM>
__global__ void __launch_bounds__(256)
router_topk_grad_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                        const float* __restrict__ w, const float* __restrict__ dw, int T, int E, int k, int ncol,
                        float* __restrict__ dl) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= T) return;
  // lane j < k holds the j-th chosen expert
  const size_t at = (size_t)t * ncol + (lane < k ? lane : 0);
  const int id = ids[at];
  const float wj = lane < k ? w[at] : 0.0f, dj = lane < k ? dw[at] : 0.0f;
  constexpr int NE = 4;   // E <= 256: experts a lane
  float l[NE];
  if constexpr (!RENORM) {
#pragma unroll
    for (int q = 0; q < NE; q++) {
      const int e = q * 64 + lane;
      l[q] = e < E ? logits[(size_t)t * E + e] : 0.0f;
    }
  }
  float s = lane < k ? wj * dj : 0.0f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  s = __shfl(s, 0, 64);   // k <= 16: the first 16 lanes' sum
  const float up = RENORM ? wj * (dj - s) : wj * dj;
  float g[NE];
#pragma unroll
  for (int q = 0; q < NE; q++) g[q] = 0.0f;
  if constexpr (!RENORM) {
    // softmax over the E scores; a NaN score counts as -infinity, as in the choice
    float m = -__builtin_inff();
#pragma unroll
    for (int q = 0; q < NE; q++) {
      l[q] = q * 64 + lane < E && l[q] == l[q] ? l[q] : -__builtin_inff();
      m = __builtin_fmaxf(m, l[q]);
    }
    m = wave_max(m);
    float z = 0.0f;
#pragma unroll
    for (int q = 0; q < NE; q++) {
      l[q] = l[q] == -__builtin_inff() ? 0.0f : expf(l[q] - m);
      z += l[q];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) z += __shfl_xor(z, o, 64);
    const float c = s / z;
#pragma unroll
    for (int q = 0; q < NE; q++) g[q] = l[q] == 0.0f ? 0.0f : -l[q] * c;
  }
  for (int j = 0; j < k; j++) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float u = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(up), j));
#pragma unroll
    for (int q = 0; q < NE; q++) g[q] += e == q * 64 + lane ? u : 0.0f;
  }
#pragma unroll
  for (int q = 0; q < NE; q++) {
    const int e = q * 64 + lane;
    if (e < E) dl[(size_t)t * E + e] = g[q];
  }
}

// f(KM) for the next instance of k pairs.  The places past k load row 0 and drop
// it: to tokens, T = 4096, 7168 bf16 values, k = 6 and 10 reach 4.9 TB/s where 8
// and 16 reach 5.2 and 5.4 (half of eight pairs dropped: 4.5).
template <typename F>
static hipError_t with_pairs(int k, F&& f) {
  if (k <= 2) return f(std::integral_constant<int, 2>{});
  if (k <= 4) return f(std::integral_constant<int, 4>{});
  if (k <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace moe

namespace moe_host {

hipError_t launch_rows_to_experts(const RowMoveArgs& a, int row_type, hipStream_t s) {
  return moe::with_row_type(row_type, [&](auto r) {
    const dim3 grid(a.T, (a.H / decltype(r)::kVec + moe::kMoveThreads - 1) / moe::kMoveThreads);
    return moe::with_pairs(a.k, [&](auto km) {
      hipLaunchKernelGGL((moe::rows_to_experts_kernel<decltype(r), decltype(km)::value>), grid,
                         dim3(moe::kMoveThreads), 0, s, a);
      return hipGetLastError();
    });
  });
}

// rows of type R, token rows of type O
template <typename R, typename O>
static hipError_t launch_rows_to_tokens_t(const RowMoveArgs& a, hipStream_t s) {
  const dim3 grid(a.T, (a.H / R::kVec + moe::kMoveThreads - 1) / moe::kMoveThreads);
  return moe::with_pairs(a.k, [&](auto km) {
    hipLaunchKernelGGL((moe::rows_to_tokens_kernel<R, O, decltype(km)::value>), grid, dim3(moe::kMoveThreads), 0, s, a);
    return hipGetLastError();
  });
}

hipError_t launch_rows_to_tokens(const RowMoveArgs& a, int row_type, hipStream_t s) {
  return moe::with_row_type(row_type, [&](auto r) { return launch_rows_to_tokens_t<decltype(r), decltype(r)>(a, s); });
}

hipError_t launch_rows_to_bf16_tokens(const RowMoveArgs& a, hipStream_t s) {
  return launch_rows_to_tokens_t<moe::RowFp32, moe::RowBf16>(a, s);
}

hipError_t launch_rows_grad(const RowMoveArgs& a, bool to_tokens, int row_type, hipStream_t s) {
  return moe::with_row_type(row_type, [&](auto r) {
    return moe::with_pairs(a.k, [&](auto km) {
      using R = decltype(r);
      constexpr int KM = decltype(km)::value;
      // waves a token by its 1 KiB runs: one or two for as many (of combine,
      // 8192 tokens of 512 bf16 values, top-8, on one, two and four waves 32, 35
      // and 48 us), four for longer rows, and sixteen for up to 512 tokens, where
      // four leave compute units idle (7168 values, four against sixteen waves:
      // T = 256 21.1 / 17.5, 512 30.0 / 28.7, 768 40.8 / 44.2, 4096 196 / 202)
      const int runs = (a.H / R::kVec + 63) / 64;
      auto launch = [&](auto wpt) {
        constexpr int W = decltype(wpt)::value, tpb = W < 4 ? 4 / W : 1;
        const dim3 grid((a.T + tpb - 1) / tpb), block(W < 4 ? moe::kMoveThreads : W * 64);
        if (to_tokens) hipLaunchKernelGGL((moe::rows_grad_kernel<R, KM, W, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((moe::rows_grad_kernel<R, KM, W, false>), grid, block, 0, s, a);
      };
      if (runs <= 1) launch(std::integral_constant<int, 1>{});
      else if (runs <= 2) launch(std::integral_constant<int, 2>{});
      else if (runs >= 8 && a.T <= 512) launch(std::integral_constant<int, 16>{});
      else launch(std::integral_constant<int, 4>{});
      return hipGetLastError();
    });
  });
}

hipError_t launch_router_topk_grad(const float* logits, const int32_t* ids, const float* w, const float* dw, int T,
                                   int E, int k, bool renorm, int n_shared, float* dl, hipStream_t s) {
  const dim3 grid((T + 3) / 4);
  if (renorm)
    hipLaunchKernelGGL(moe::router_topk_grad_kernel<true>, grid, dim3(256), 0, s, logits, ids, w, dw, T, E, k,
                       k + n_shared, dl);
  else
    hipLaunchKernelGGL(moe::router_topk_grad_kernel<false>, grid, dim3(256), 0, s, logits, ids, w, dw, T, E, k,
                       k + n_shared, dl);
  return hipGetLastError();
}

}  // namespace moe_host
