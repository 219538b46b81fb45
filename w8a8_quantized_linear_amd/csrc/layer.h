// What a decoder layer does around its projections and attention (norms, rotary positions, E4M3 products with block
// scales): host-side launch interface between the C entry points (layer_api.cpp) and the kernel sources.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace w8a8 {

// What a norm writes: bf16, or codes with one scale a token (int8, E4M3) or one for each 128 columns (E4M3).
enum class NormOut : int { kBf16 = 0, kI8 = 1, kFp8 = 2, kBlock = 3 };

// Columns of a block scale, and rows of one of a weight.
constexpr int kScaleBlock = 128;

// Row stride of the scales [K / 128][stride] that go with packed activation codes.
__host__ __device__ inline int64_t block_scale_stride(int64_t M) { return (M + 31) / 32 * 32; }

// norm.hip: h = bf16(x + residual) (x itself without one), y = h * weight / sqrt(mean(h^2) + eps).
struct Norm {
  const uint16_t* x;
  const uint16_t* residual;   // or null
  const uint16_t* weight;     // [K]
  uint16_t* h;                // or null
  void* out;                  // bf16 [M, K], or codes [M, K], row-major or packed
  float* scales;              // [M]; block scales [M, K / 128], of packed codes [K / 128][block_scale_stride(M)]
  int64_t M, K;
  float eps;
  NormOut kind;
  bool rotate, packed;        // rotate: codes of the values turned by the normalized transform in blocks of 128
};
hipError_t launch_norm(const Norm& n, hipStream_t stream);

// rope.hip: rows [seqs * tokens] of q [q_heads, dim] and k [heads, dim], out in rows of their own strides.
struct Rope {
  const uint16_t *q, *k;
  uint16_t *q_out, *k_out;
  int64_t ldq, ldk, ldq_out, ldk_out;
  const uint64_t* turns;      // [rotary / 2]
  const int32_t* lens;        // [seqs]
  int64_t seqs, tokens;
  int q_heads, heads, dim, rotary;
  bool interleaved;
  float amplitude;
};
hipError_t launch_rope(const Rope& r, hipStream_t stream);

// block_quant.hip: E4M3 codes with a scale for each 128 columns of a row, or each 128 x 128 block of a weight.
hipError_t launch_quantize_block(const uint16_t* x, int64_t M, int64_t K, bool packed, uint8_t* q, float* s, hipStream_t stream);
hipError_t launch_quantize_weight_block(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* s, hipStream_t stream);

// Packed codes and their block scales, y bf16 [M, N].  block_few.hip: where block_few_fits(), or x bf16 itself where
// block_fused_fits(); block_gemm.hip: any shape.
bool block_few_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_block_few(const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y,
                            int64_t M, int64_t N, int64_t K, hipStream_t stream);
bool block_fused_fits(int64_t M, int64_t N, int64_t K);
hipError_t launch_block_fused(const uint16_t* x, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y, int64_t M,
                              int64_t N, int64_t K, hipStream_t stream);
// Bytes of the sums that launch_block_gemm needs where it cuts K (0 elsewhere).
size_t block_gemm_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_block_gemm(const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, float* sums, hipStream_t stream);

}  // namespace w8a8
