// Product of E4M3 codes with block scales, y = x W^T + b.
//
// What it computes: y[m][n] = bf16(sum over blocks b of 128 columns of s[b][m] * sw[n / 128][b] * (sum over the block of
// q[m][k] * w[n][k]) + bias[n]): the inner sums on the E4M3 matrix instructions, the outer one in fp32.
//
// The instruction (v_mfma_f32_16x16x128_f8f6f4 and its 32x32x64 form) does not sum like fp32 throughout: measured on the
// device, products that lie 2^-13 below the largest of their group of products lose what is below that, toward zero,
// while groups and the accumulator meet in fp32.  On normal values that is 1.4e-5 of the output's rms (4e-5 with
// outliers twenty times as large), against 1.6e-3 that rounding the output to bf16 makes and about 4e-2 of quantizing
// both operands; widening to bf16 instead would sum in fp32 at half the rate.  A block starts from zero, so that nothing
// is lost against the sum so far.
#include "decode.h"
#include "layer.h"
#include "layer_math.h"

namespace w8a8 {
namespace {

using namespace lm;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// 128 columns of 16 weight rows and 16 tokens: lane l holds columns 32 (l / 16) .. + 31 of row l % 16 of both, and gets
// token l % 16, weight rows 4 (l / 16) .. + 3.
__device__ __forceinline__ f32x4 mfma128(i32x8 w, i32x8 x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 127, 0, 127);
}

// 32 bytes of a packed row: columns 128 b + 32 h ...
__device__ __forceinline__ i32x8 operand(const uint8_t* __restrict__ p, int64_t row, int64_t b, int h, int64_t K) {
  const uint8_t* at = p + code_at(row, 128 * b + 32 * h, K, true);
  i32x8 v;
  reinterpret_cast<u32x4*>(&v)[0] = *reinterpret_cast<const u32x4*>(at);
  reinterpret_cast<u32x4*>(&v)[1] = *reinterpret_cast<const u32x4*>(at + 16);
  return v;
}

// One wave for 16 tokens and 16 weight rows, operands straight from memory.
__global__ void __launch_bounds__(64)
block_gemm_simple(const uint8_t* __restrict__ q, const float* __restrict__ s, const uint8_t* __restrict__ w, const float* __restrict__ sw,
                  const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t M, int64_t N, int64_t K, int64_t first, int64_t tiles_n) {
  const int l = threadIdx.x, c = l % 16, h = l / 16;
  const int64_t tile = first + blockIdx.x, m = tile / tiles_n * 16 + c, n0 = tile % tiles_n * 16;
  const int64_t mr = min(m, M - 1), s_ld = block_scale_stride(M);
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t b = 0; b < K / kScaleBlock; ++b) {
    const f32x4 part = mfma128(operand(w, min(n0 + c, N - 1), b, h, K), operand(q, mr, b, h, K));
    const float by = s[b * s_ld + mr] * sw[n0 / kScaleBlock * (K / kScaleBlock) + b];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], by, acc[i]);
  }
  const int64_t n = n0 + 4 * h;
  if (m >= M || n >= N) return;
  if (bias) {
    float b4[4];
    bf16x4(*reinterpret_cast<const uint2*>(bias + n), b4);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] += b4[i];
  }
  *reinterpret_cast<uint2*>(y + m * N + n) = make_uint2(bf16x2_rne(acc[0], acc[1]), bf16x2_rne(acc[2], acc[3]));
}

}  // namespace

hipError_t launch_block_gemm(const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  const int64_t tiles_n = (N + 15) / 16;
  return in_launches((M + 15) / 16 * tiles_n, 1, 64, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL(block_gemm_simple, dim3((unsigned)count), dim3(64), 0, stream, q, s, w, sw, bias, y, M, N, K, first, tiles_n);
    return hipGetLastError();
  });
}

}  // namespace w8a8
