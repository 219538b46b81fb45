// What the forms of the product of E4M3 codes with block scales share.
//
// The instruction (v_mfma_f32_16x16x128_f8f6f4) does not sum like fp32 throughout: measured on the device, products that
// lie 2^-13 below the largest of their group of products lose what is below that, toward zero, while groups and the
// accumulator meet in fp32.  On normal values that is 1.4e-5 of the output's rms (4e-5 with outliers twenty times as
// large), against 1.6e-3 that rounding the output to bf16 makes and about 4e-2 of quantizing both operands; widening to
// bf16 instead would sum in fp32 at half the rate.  Each block starts from zero, so that nothing is lost against the sum
// so far.
#pragma once

#include "layer_math.h"

namespace w8a8 {
namespace lm {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 128 columns of 16 weight rows and 16 tokens: lane l holds 32 columns of row l % 16 of both, l / 16 the same quarter of
// them, and gets token l % 16, weight rows 4 (l / 16) .. + 3.
__device__ __forceinline__ f32x4 mfma128(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}

// Memory from `base` on, for loads of a scalar and a 32-bit lane offset (the scalar part stays out of the lanes'
// registers). The range is left open: what is read is the caller's to keep inside.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, -1, 0x00020000);
}
// Packed rows' operand at lane offset `at` (row's place + 16 h), scalar offset `from`: columns 16 h .. + 15 and 64 + 16
// h .. + 15 of a block, so that each load of a wave is one run of 1 KiB.  (Which columns meet in which lanes is free as
// long as both operands agree.  32 columns a lane in order leave every load half of twice as many lines: 64 tokens of
// 5,120 x 34,816 took 2 to 5% longer that way.)
__device__ __forceinline__ i32x8 load_operand(Buffer p, uint32_t at, uint32_t from) {
  const u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(p, (int)at, (int)from, 0);
  const u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(p, (int)at + 2048, (int)from, 0);
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}
__device__ __forceinline__ float load_scale(Buffer p, uint32_t at, uint32_t from) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(p, (int)at, (int)from, 0));
}

// Largest of lanes l, l ^ 16, l ^ 32 and l ^ 48, as larger().
__device__ __forceinline__ float max_quarters(float v) {
  uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = larger(__uint_as_float(a[0]), __uint_as_float(a[1]));
  u = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return larger(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// Four sums of token m, rows n .. n + 3 (n % 4 == 0): the bias added, rounded once.
__device__ __forceinline__ void store_row4(f32x4 sum, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t m, int64_t n,
                                           int64_t N) {
  if (bias) {
    float b[4];
    bf16x4(*reinterpret_cast<const uint2*>(bias + n), b);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += b[e];
  }
  *reinterpret_cast<uint2*>(y + m * N + n) = make_uint2(bf16x2_rne(sum[0], sum[1]), bf16x2_rne(sum[2], sum[3]));
}

}  // namespace lm
}  // namespace w8a8
