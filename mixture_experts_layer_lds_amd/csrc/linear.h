// Matrix products of rows with the experts' matrices, and their gradients, on
// LDS tiles: what linear.hip, linear_stream.hip, linear_grad_x.hip and
// linear_grad_w.hip share.
//
// Every product is D[m][c] = sum over q of R[m][q] C[c][q], c the contiguous
// index of D.  The MFMA takes C as its rows and R as its columns, so that a
// lane holds four neighbouring values of a row of D.
//
//               m         c              q           R            C
//   forward     row       column n       k           x[m][q]      w[c][q]
//   grad x      row       column k       n           dy[m][q]     w[q][c]
//   grad w      n         k              row         dy[q][m]     x[q][c]
//
// An operand that is contiguous in q stands in LDS as rows of 64 q (128 bytes),
// one that is not as rows of c or m, q by q, read with the transposing LDS read.
#pragma once

#include "act.h"
#include "lds_dma.h"

namespace moe {

enum LinearOp { kForward, kGradX, kGradW };

struct ElemBf16 {
  typedef RowBf16 Row;
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ u32x2 pack4(const float (&v)[4]) {
    return u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  }
  static __device__ __forceinline__ void unpack4(const u32x2& q, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint16_t round(float v) { return (uint16_t)bf16_pair(v, 0.0f); }
  static __device__ __forceinline__ float widen(uint16_t v) { return bf16_bits_to_f32(v); }
};

struct ElemFp16 {
  typedef RowFp16 Row;
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  static __device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ u32x2 pack4(const float (&v)[4]) {
    return __builtin_bit_cast(u32x2, f16x4{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]});
  }
  static __device__ __forceinline__ void unpack4(const u32x2& q, float (&v)[4]) {
    const f16x4 h = __builtin_bit_cast(f16x4, q);
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = (float)h[i];
  }
  static __device__ __forceinline__ _Float16 round(float v) { return (_Float16)v; }
  static __device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
};

// A buffer offset that is out of every range (they end at 2^31) and stays so with the
// stage's added: the copy writes zeros.
constexpr uint32_t kOutside = 0x80000000u;

// A buffer of `bytes` from base: copies from behind it write zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_rsrc(const char* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ void range_dma16(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff, char* dst) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, off, soff, 0, 0);
}

constexpr int kStepQ = 64;   // q of a sub-step, and of a chunk of the streamed weights: 128 bytes

// One operand's tile in LDS: TILE values of m or c by kStepQ of q.
//
// TRANS false: TILE rows of 128 bytes, piece p (16 bytes) of row r at place
// p ^ (r % 8).  A copy instruction takes 8 rows.  A fragment (row lane % 16,
// piece lane / 16 of the 64-byte half) is one ds_read_b128.
//
// TRANS true: 64 rows (q) of TILE values; block b (16 values, 32 bytes) of row
// q at place b ^ f(q), f the row's two low bits and its bit 3 (64 values: its
// bits 1 and 3; 32: bit 3), so that the eight rows which half a wave reads at once stand
// in different banks.  A fragment is two ds_read_b64_tr_b16: 16 lanes read four
// rows of a block and get four q of their own column each.
template <bool TRANS, int TILE>
struct OperandTile {
  static constexpr int kBytes = TILE * kStepQ * 2;
  static constexpr int kCopies = kBytes / 1024;                    // wave instructions
  static constexpr int kPitch = TRANS ? TILE * 2 : kStepQ * 2;     // bytes a row
  static constexpr int kRowsACopy = 1024 / kPitch;

  static __device__ __forceinline__ int swizzle(int q) {
    return TILE >= 128 ? (q & 3) | ((q >> 3) & 1) << 2 : TILE == 64 ? ((q >> 1) & 1) | ((q >> 3) & 1) << 1 : (q >> 3) & 1;
  }
  // The row of the tile that a lane of copy i takes, and its byte in that row.
  static __device__ __forceinline__ int copy_row(int i, int lane) { return i * kRowsACopy + lane / (kPitch / 16); }
  static __device__ __forceinline__ int copy_byte(int i, int lane) {
    const int p = lane % (kPitch / 16);
    if constexpr (TRANS) return (((p >> 1) ^ swizzle(copy_row(i, lane))) << 5) | (p & 1) << 4;
    return (p ^ (lane >> 3)) * 16;   // copy_row % 8 is lane / 8
  }
  // A lane's place in the fragments of the wave's first block, and the fragment
  // of its block `block` for the 32 q of half h, `at` being that place in the
  // stage.  The wave's blocks are `first` with the bits of `block` set, which
  // are none of first's.
  static __device__ __forceinline__ uint32_t lane_place(int first, int lane) {
    const int g = lane >> 4;
    if constexpr (!TRANS) return (first * 16 + (lane & 15)) * 128 + ((g ^ (lane & 7)) << 4);
    const int q = 8 * g + ((lane & 15) >> 2);
    return q * kPitch + (((first & 7) ^ swizzle(q)) << 5) + ((first & ~7) << 5) + 8 * (lane & 3);
  }
  static __device__ __forceinline__ u32x4 fragment(uint32_t at, int block, int h) {
    if constexpr (!TRANS) {
      typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
      return *reinterpret_cast<lds_u32x4*>((at ^ (h << 6)) + block * 2048);
    } else {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
      const uint32_t p = (at ^ ((block & 7) << 5)) + ((block & ~7) << 5) + h * 32 * kPitch;
      const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(p)));
      const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(p + 4 * kPitch)));
      return u32x4{a[0], a[1], c[0], c[1]};
    }
  }
};

// A tile of BM by BC, WM by WC waves, KG groups of them that take the
// sub-steps of a stage in turn and add their sums at the end; NS stages in LDS.
template <int BM_, int BC_, int WM_, int WC_, int KG_, int NS_>
struct LinearShape {
  static constexpr int BM = BM_, BC = BC_, WM = WM_, WC = WC_, KG = KG_, kStages = NS_;
  static constexpr int kWaves = WM * WC * KG, kThreads = kWaves * 64;
  static constexpr int MB = BM / WM / 16, CB = BC / WC / 16;   // 16 x 16 blocks of a wave
  static constexpr int MB0 = (MB + 1) / 2;                     // ... of m in the first part of its operand
  static constexpr int kRows0 = MB0 * WM * 16, kRows1 = BM - kRows0;
  static constexpr int kSub = (BM + BC) * kStepQ * 2;          // bytes of a sub-step
  static constexpr int kStage = kSub * KG;
  static constexpr int kRanges = 3 * 4 * (kMaxExperts + 1);    // first item and rows of every expert
  static constexpr int kScratch = 2048;                        // of a wave: 16 rows of 128 bytes, or its columns in 64 bits
  static constexpr int kSpare = 1024;                          // where copies go that a wave has too many
  static constexpr int kLds = kStage * kStages + kRanges + kSpare + kWaves * kScratch;
  // workgroups that share a CU's LDS, and the waves on a SIMD that they make
  static constexpr int kOccupancy = kLds <= 80 * 1024 && kThreads <= 256 ? 2 : 1;
  static constexpr int kWavesASimd = kOccupancy * kWaves / 4;
};

}  // namespace moe
