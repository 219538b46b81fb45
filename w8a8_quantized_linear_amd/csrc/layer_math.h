// Device arithmetic that the kernels of norms, rotary positions and block scales share.
#pragma once

#include "epilogue_math.h"
#include "quant_math.h"

namespace w8a8 {
namespace lm {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// The value of another lane of the row of 16: i ^ 1, i ^ 2, i ^ 3, 7 - i of its eight, 15 - i, i ^ 8.
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kHalfMirror = 0x141, kMirror = 0x140, kXor8 = 0x128;

// The larger of two values; a NaN where one is (fmaxf gives the other one): what a scale is made of, so that a NaN shows in
// all that the scale multiplies.  (One instruction for three values, as for fmaxf.)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Maximum (as larger()) and sum over the 16 lanes of a row, the same in all of them.
__device__ __forceinline__ float max16(float v) {
  v = larger(v, qm::dpp_move<kXor1>(v));
  v = larger(v, qm::dpp_move<kXor2>(v));
  v = larger(v, qm::dpp_move<kHalfMirror>(v));
  return larger(v, qm::dpp_move<kMirror>(v));
}
__device__ __forceinline__ float sum16(float v) {
  v += qm::dpp_move<kXor1>(v);
  v += qm::dpp_move<kXor2>(v);
  v += qm::dpp_move<kHalfMirror>(v);
  return v + qm::dpp_move<kMirror>(v);
}

// And over the wave: the swaps exchange odd rows of 16 (the upper half) of one copy with even rows (the lower half)
// of the other.
__device__ __forceinline__ float max64(float v) {
  v = max16(v);
  uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = larger(__uint_as_float(a[0]), __uint_as_float(a[1]));
  u = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return larger(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum64(float v) {
  v = sum16(v);
  uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  u = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ void widen8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = qm::bf16lo(v[i]);
    f[2 * i + 1] = qm::bf16hi(v[i]);
  }
}
__device__ __forceinline__ u32x4 narrow8(const float (&f)[8]) {
  return u32x4{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3]), bf16x2_rne(f[4], f[5]), bf16x2_rne(f[6], f[7])};
}

// E4M3 codes of eight values that carry the scale's pre-factor: the nearest to fl32(v / s) within +-448, the sign of
// v on a zero (all codes +0 where the scale is zero or a NaN).
__device__ __forceinline__ u32x2 e4m3_codes8(const float (&v)[8], const qm::QuotientScale& q) {
  const uint32_t keep = q.s > 0.0f ? ~0u : 0u;
  u32x2 out;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      t[e] = fminf(fmaxf(__builtin_copysignf(qm::quotient(v[4 * g + e], q.s, q.r), v[4 * g + e]), -448.0f), 448.0f);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
    out[g] = (uint32_t)w & keep;
  }
  return out;
}
__device__ __forceinline__ u32x2 int8_codes8(const float (&v)[8], const qm::QuotientScale& q) {
  return u32x2{qm::int8_codes4(v[0], v[1], v[2], v[3], q.s, q.r), qm::int8_codes4(v[4], v[5], v[6], v[7], q.s, q.r)};
}

// Byte of element e (a multiple of 8) of a row of codes: row-major, or packed (blocks of 32 rows x 64 bytes).
__device__ __forceinline__ int64_t code_at(int64_t row, int64_t e, int64_t K, bool packed) {
  return packed ? (row / 32 * (K / 64) + e / 64) * 2048 + row % 32 * 64 + e % 64 : row * K + e;
}

// Block id -> place in row order: consecutive ids go to the 8 XCDs in turn, so that every XCD gets a run of neighbouring
// rows, which share 128-byte lines of packed codes and of their scales.
__device__ __forceinline__ int64_t xcd_order(int64_t bid, int64_t blocks) {
  const int64_t q = blocks / 8, r = blocks % 8, xcd = bid % 8;
  return xcd * q + (xcd < r ? xcd : r) + bid / 8;
}

}  // namespace lm
}  // namespace w8a8
