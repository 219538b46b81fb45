// What the two forms of attention over the paged 8-bit cache share: types, the codes' conversion, the cut of a
// sequence into pieces, and where the pieces leave their partial results.
#pragma once

#include "decode.h"
#include "epilogue_math.h"

namespace w8a8 {
namespace kva {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kLazy = 8.0f;                   // log2 of how far p * scale may pass the running maximum
constexpr float kProbExp = 7.0f;                // p' < 2^(kLazy + kProbExp); f16 ends at 2^16
constexpr float kLeastLog = -90.0f;             // values' scales below 2^this count as zero
constexpr float kSumBy = 0x1p-8f;               // sums are held times this: p' / scale < 2^(15 + 90), over 2^30 tokens
                                                // 2^135, past fp32's range without it (and 2^-8 / scale keeps 13 bits
                                                // up to a scale of 2^128)
constexpr int kPiece = 128;                     // pieces of a sequence are whole multiples of this

// Tokens of each of the `splits` pieces of a sequence.
__host__ __device__ __forceinline__ int piece_of(int held, int splits) {
  return ((held + splits - 1) / splits + kPiece - 1) / kPiece * kPiece;
}

// Two f16 values 1024 + u -> u - 128, exactly: with 0x64 above it a byte u is the f16 1024 + u, and a code with its
// top bit flipped is u = code + 128.
__device__ __forceinline__ uint32_t f16_codes(uint32_t biased) {
  const f16x2 v = __builtin_bit_cast(f16x2, biased) - f16x2{(_Float16)1152.0f, (_Float16)1152.0f};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

// Four codes in memory order -> f16, two per word.
__device__ __forceinline__ void f16_word(uint32_t word, uint32_t* two) {
  word ^= 0x80808080u;
  two[0] = f16_codes(__builtin_amdgcn_perm(0x64646464u, word, 0x04010400u));
  two[1] = f16_codes(__builtin_amdgcn_perm(0x64646464u, word, 0x04030402u));
}

// Byte b of two words -> f16.
__device__ __forceinline__ uint32_t f16_bytes(uint32_t hi, uint32_t lo, int b) {
  return f16_codes(__builtin_amdgcn_perm(hi, lo, 0x0c000c00u | (4 + b) << 16 | b) ^ 0x64806480u);
}

// The power of two that brings a row of queries whose largest magnitude has these bits into [2^7, 2^8).
__device__ __forceinline__ int query_exp(uint32_t top_bits) { return min(134 - (int)(top_bits >> 23), 126); }

// The larger (sum) of lanes l and l ^ 32; of lanes l, l ^ 16, l ^ 32 and l ^ 48.  The swaps exchange the odd rows
// of 16 (the upper half) of one copy with the even rows (the lower half) of the other.
__device__ __forceinline__ float max_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float sum_halves(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float max_quarters(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return max_halves(fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
}
__device__ __forceinline__ float sum_quarters(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return sum_halves(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// Partial results of a row's pieces, for each row and piece: unnormalised outputs [dim], and maximum and sum.
struct Partial {
  float* out;
  float* stat;
  Partial from(int64_t index, int dim) const { return out ? Partial{out + index * dim, stat + 2 * index} : *this; }
};

// The part of `length` tokens that the last `tokens` of them see on average.
inline double seen_of(int64_t tokens, int64_t length) {
  return tokens < length ? 1.0 - 0.5 * (double)tokens / (double)length : 0.5;
}

// Prompt form (attention_prompt.hip): query rows of a workgroup (128 or 256) and pieces of a sequence.
struct PromptCut {
  int rows;
  int64_t splits;
};
PromptCut prompt_cut(int64_t seqs, int64_t rows, int64_t tokens, int heads, int dim, int64_t length);
template <int DIM>
hipError_t launch_prompt(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group,
                         float scale, PromptCut cut, uint16_t* y, Partial part, hipStream_t stream);

}  // namespace kva
}  // namespace w8a8
