// MXFP4 quantisation of rows, its inverse, and the one-time weight pre-pack
// (SGLang tuning guide, block shapes: gfx95 devices keep MX's [1, 32]
// blocks; the format and its rounding are in mx4.h).
//
// Both passes go over 16 bytes of row values a lane at a time (eight 16-bit or
// four 32-bit values), so that a wave's loads and stores of rows are whole
// 1 KiB runs, and a 32-value block lies on four or eight neighbouring lanes,
// which exchange its largest magnitude in two or three steps.  Every value is
// read once and nothing is kept: the passes are bound by their bytes.  Large
// ones take four runs a wave, all loads ahead of the first use: 131072 x 7168
// fp32 values in 709 us (6.0 TB/s) and back in 786 (5.4).  Rows apart take a
// 64-bit division a vector: 65536 x 3584 bf16 values 104 us (5.7 TB/s), 97 where
// they follow one another.
#include "decode_route.h"
#include "route_group.h"
#include "mx4.h"
#include "rows.h"

namespace moe {

constexpr int kMx4Threads = 256;

// Eight values -> the lane's four code bytes and the block's scale code.
__device__ __forceinline__ uint32_t mx4_quant8(const float (&v)[8], uint32_t& code) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) m = max(m, abs_bits(v[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
  code = mx4_scale_code(m);
  return mx4_encode8(v, code);
}

// The vector (16 bytes of row values) that lane and step u of this thread
// take: a wave's UN runs are consecutive.
template <int UN>
__device__ __forceinline__ size_t mx4_vector(int u) {
  return (((size_t)blockIdx.x * (kMx4Threads / 64) + (threadIdx.x >> 6)) * UN + u) * 64 + (threadIdx.x & 63);
}

// rows x cols values -> codes [rows][cols/2] and scale codes [rows][cols/32],
// row-major.  FLAT: rows follow one another; else row_stride elements apart.
template <typename R, int UN, bool FLAT>
__global__ void __launch_bounds__(kMx4Threads)
mx4_quantize_kernel(const typename R::elem* __restrict__ x, size_t nvec, uint32_t vec_per_row, size_t row_stride,
                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int N = R::kVec, LB = 32 / N;   // values a lane, lanes a block
  u32x4 raw[UN];
#pragma unroll
  for (int u = 0; u < UN; u++) {
    size_t i = mx4_vector<UN>(u);
    i = i < nvec ? i : 0;
    size_t at = i * N;
    if constexpr (!FLAT) {
      const size_t row = i / vec_per_row;
      at = row * row_stride + (i - row * vec_per_row) * N;
    }
    raw[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + at));
  }
#pragma unroll
  for (int u = 0; u < UN; u++) {
    const size_t i = mx4_vector<UN>(u);
    if (i >= nvec) continue;   // whole blocks: nvec is a multiple of LB
    float v[N];
    R::unpack(raw[u], v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; j++) m = max(m, abs_bits(v[j]));
#pragma unroll
    for (int o = 1; o < LB; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    const uint32_t code = mx4_scale_code(m);
    if constexpr (N == 8) reinterpret_cast<uint32_t*>(codes)[i] = mx4_encode8(v, code);
    else reinterpret_cast<uint16_t*>(codes)[i] = (uint16_t)mx4_encode4(f32x4{v[0], v[1], v[2], v[3]}, code);
    if (threadIdx.x % LB == 0) scales[i / LB] = (uint8_t)code;
  }
}

// codes and scale codes -> values.
template <typename R, int UN>
__global__ void __launch_bounds__(kMx4Threads)
mx4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, size_t nvec,
                      typename R::elem* __restrict__ out) {
  constexpr int N = R::kVec, LB = 32 / N;
  uint32_t c[UN], sc[UN];
#pragma unroll
  for (int u = 0; u < UN; u++) {
    size_t i = mx4_vector<UN>(u);
    i = i < nvec ? i : 0;
    if constexpr (N == 8) c[u] = reinterpret_cast<const uint32_t*>(codes)[i];
    else c[u] = reinterpret_cast<const uint16_t*>(codes)[i];
    sc[u] = scales[i / LB];
  }
#pragma unroll
  for (int u = 0; u < UN; u++) {
    const size_t i = mx4_vector<UN>(u);
    if (i >= nvec) continue;
    const float scale = sc[u] == 255u ? __uint_as_float(0x7fc00000u) : mx4_scale_value(sc[u]);
    float v[N];
#pragma unroll
    for (int j = 0; j < N; j++) {
      const uint32_t n = (c[u] >> (4 * j)) & 15u, m = n & 7u;
      // magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6 as floats, from the code's exponent and mantissa bits
      const float mag = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
      v[j] = __uint_as_float(__float_as_uint(mag) | ((n & 8u) << 28)) * scale;
    }
    __builtin_nontemporal_store(R::pack(v), reinterpret_cast<u32x4*>(out + i * N));
  }
}

// x [T][H] bf16 -> codes [T][H/2] row-major, scale codes [T][H/128/G][4][G]
// (a lane of the product takes the G codes of its 32-value column in one
// load); vector i, eight values.
__device__ __forceinline__ void mx4_quant_x(const uint16_t* __restrict__ x, uint32_t i, uint32_t vec_per_row, int G,
                                            uint32_t* __restrict__ xq, uint8_t* __restrict__ sx) {
  float v[8];
  row_load<RowBf16>(x + (size_t)i * 8, v);
  uint32_t code;
  xq[i] = mx4_quant8(v, code);
  if ((threadIdx.x & 3) == 0) {
    const uint32_t row = i / vec_per_row, b = (i - row * vec_per_row) / 4;   // block of the row
    const uint32_t unit = b / 4, kb = b % 4, grp = unit / G, u = unit % G;
    sx[(size_t)row * (vec_per_row / 4) + grp * 4 * G + kb * G + u] = (uint8_t)code;
  }
}

// ROUTE (at most 64 pairs): workgroup 0 also does the routing build.
template <bool ROUTE>
__global__ void __launch_bounds__(kMx4Threads)
mx4_quant_x_kernel(const uint16_t* __restrict__ x, uint32_t nvec, uint32_t vec_per_row, int G,
                   uint32_t* __restrict__ xq, uint8_t* __restrict__ sx, moe_host::DecodeRouteOut route, int P) {
  if constexpr (ROUTE) {
    if (blockIdx.x == 0) {
      const int lane = threadIdx.x & 63;
      const DecodeRoute rt = decode_route(route.ids, P, route.E, route.block_m, lane);
      decode_route_write(rt, route, P, threadIdx.x, kMx4Threads, lane, threadIdx.x >> 6);
    }
  }
  const uint32_t i = blockIdx.x * kMx4Threads + threadIdx.x;
  if (i < nvec) mx4_quant_x(x, i, vec_per_row, G, xq, sx);   // whole blocks: nvec % 16 == 0
}

// Up to kOneGroupPairs pairs: workgroup 0 does the routing build, the others
// the codes, which do not depend on it.  One launch instead of two: the build
// takes about 5 us whatever the batch, the codes 4 (Qwen3-30B-A3B-shaped layer,
// T = 64: 46.0 -> 44.4 us, DeepSeek-V3-shaped 816 -> 814).
__global__ void __launch_bounds__(kRouteThreads)
mx4_route_quant_kernel(const uint16_t* __restrict__ x, uint32_t nvec, uint32_t vec_per_row, int G,
                       uint32_t* __restrict__ xq, uint8_t* __restrict__ sx, moe_host::DecodeRouteOut o, int P) {
  if (blockIdx.x == 0) {
    route_one_group(o.ids, P, o.E, o.block_m, o.max_tasks, o.header, o.expert_offsets, o.sorted_pairs, o.pair_pos,
                    o.tasks);
    return;
  }
  const uint32_t i = (blockIdx.x - 1) * kRouteThreads + threadIdx.x;
  if (i < nvec) mx4_quant_x(x, i, vec_per_row, G, xq, sx);
}

// Row-major codes and scale codes -> blocks of 16 rows x G units (mx4.h).
// Block b of an expert holds rows 32 (b / 2) + 8 g + 4 (b % 2) + i in its
// row 4 g + i: the product then leaves a lane four consecutive output
// columns, and with the neighbouring block eight.  One thread a 16-byte
// piece of codes.
__global__ void __launch_bounds__(256)
mx4_pack_kernel(const u32x4* __restrict__ codes, const uint8_t* __restrict__ scales, size_t pieces, int units,
                int G, char* __restrict__ packed) {
  for (size_t p = (size_t)blockIdx.x * 256 + threadIdx.x; p < pieces; p += (size_t)gridDim.x * 256) {
    const int lane = (int)(p % 64);
    const size_t chunk = p / 64;
    const int unit = (int)(chunk % units);
    const size_t blk = chunk / units;   // over all experts
    const int m = lane & 15, kb = lane >> 4;
    const size_t row = 32 * (blk / 2) + 8 * (m >> 2) + 4 * (blk % 2) + (m & 3);
    char* base = packed + (blk * units + unit / G * G) * kMx4Unit;
    const int u = unit % G;
    *reinterpret_cast<u32x4*>(base + u * 1024 + 16 * lane) = codes[(row * units + unit) * 4 + kb];
    base[G * 1024 + lane * G + u] = (char)scales[(row * units + unit) * 4 + kb];
  }
}

}  // namespace moe

namespace moe_host {

// Workgroups of a grid-stride pass over n items: at most sixteen per compute
// unit (of 256), fewer when there is less to do.
static unsigned pass_grid(size_t n) {
  const size_t b = (n + 255) / 256;
  return (unsigned)(b < 4096 ? b : 4096);
}

// f(UN) with the workgroups of a pass over nvec vectors: four runs a wave from
// 4 MiB of them on (131072 x 7168 bf16, one run against four: back 521 / 395 us,
// the quantiser 390 / 404; at 2^18 vectors and up to 2^20 both within a launch's
// spread, and fewer vectors would leave compute units idle).
template <typename F>
static hipError_t mx4_pass(size_t nvec, F&& f) {
  const size_t per = moe::kMx4Threads;
  if (nvec >= (size_t)1 << 18) return f(std::integral_constant<int, 4>{}, dim3((unsigned)((nvec + 4 * per - 1) / (4 * per))));
  return f(std::integral_constant<int, 1>{}, dim3((unsigned)((nvec + per - 1) / per)));
}

hipError_t launch_mx4_quantize(const void* x, int row_type, size_t rows, int cols, size_t row_stride, uint8_t* codes,
                               uint8_t* scales, hipStream_t s) {
  return moe::with_row_type(row_type, [&](auto r) {
    using R = decltype(r);
    const uint32_t per_row = cols / R::kVec;
    const size_t nvec = rows * (size_t)per_row;
    const typename R::elem* p = static_cast<const typename R::elem*>(x);
    return mx4_pass(nvec, [&](auto un, dim3 grid) {
      constexpr int UN = decltype(un)::value;
      if (row_stride == (size_t)cols)
        hipLaunchKernelGGL((moe::mx4_quantize_kernel<R, UN, true>), grid, dim3(moe::kMx4Threads), 0, s, p, nvec,
                           per_row, row_stride, codes, scales);
      else
        hipLaunchKernelGGL((moe::mx4_quantize_kernel<R, UN, false>), grid, dim3(moe::kMx4Threads), 0, s, p, nvec,
                           per_row, row_stride, codes, scales);
      return hipGetLastError();
    });
  });
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, const uint8_t* scales, size_t rows, int cols, int row_type,
                                 void* out, hipStream_t s) {
  return moe::with_row_type(row_type, [&](auto r) {
    using R = decltype(r);
    const size_t nvec = rows * (size_t)(cols / R::kVec);
    return mx4_pass(nvec, [&](auto un, dim3 grid) {
      hipLaunchKernelGGL((moe::mx4_dequantize_kernel<R, decltype(un)::value>), grid, dim3(moe::kMx4Threads), 0, s,
                         codes, scales, nvec, static_cast<typename R::elem*>(out));
      return hipGetLastError();
    });
  });
}

int mx4_route_pairs() { return moe::kOneGroupPairs; }

hipError_t launch_mx4_quant_x(const uint16_t* x, int T, int H, uint8_t* xq, uint8_t* sx, hipStream_t s,
                              const DecodeRouteOut* route, int P) {
  if (route && (P > moe::kOneGroupPairs || !route->ids)) return hipErrorInvalidValue;
  const uint32_t nvec = (uint32_t)T * (uint32_t)(H / 8);   // T * H <= 2^32
  const dim3 grid((nvec + moe::kMx4Threads - 1) / moe::kMx4Threads);
  const DecodeRouteOut ro = route ? *route : DecodeRouteOut{};
  uint32_t* q = reinterpret_cast<uint32_t*>(xq);
  if (route && P > moe::kDecodeRoutePairs)
    hipLaunchKernelGGL(moe::mx4_route_quant_kernel, dim3(1 + (nvec + moe::kRouteThreads - 1) / moe::kRouteThreads),
                       dim3(moe::kRouteThreads), 0, s, x, nvec, (uint32_t)(H / 8), moe::mx4_group(H), q, sx, ro, P);
  else if (route)
    hipLaunchKernelGGL(moe::mx4_quant_x_kernel<true>, grid, dim3(moe::kMx4Threads), 0, s, x, nvec, (uint32_t)(H / 8),
                       moe::mx4_group(H), q, sx, ro, P);
  else
    hipLaunchKernelGGL(moe::mx4_quant_x_kernel<false>, grid, dim3(moe::kMx4Threads), 0, s, x, nvec, (uint32_t)(H / 8),
                       moe::mx4_group(H), q, sx, ro, P);
  return hipGetLastError();
}

hipError_t launch_mx4_pack(const uint8_t* codes, const uint8_t* scales, int E, int rows, int cols, void* packed,
                           hipStream_t s) {
  const size_t pieces = (size_t)E * rows * (cols / 32);
  hipLaunchKernelGGL(moe::mx4_pack_kernel, dim3(pass_grid(pieces)), dim3(256), 0, s,
                     reinterpret_cast<const moe::u32x4*>(codes), scales, pieces, cols / 128, moe::mx4_group(cols),
                     static_cast<char*>(packed));
  return hipGetLastError();
}

}  // namespace moe_host
