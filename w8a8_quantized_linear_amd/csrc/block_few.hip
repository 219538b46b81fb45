// Product of E4M3 codes with block scales for few tokens: bound by the weight's bytes.
//
// What it computes: as block_gemm.hip, on the same instruction.
//
// A workgroup owns 16 RB weight rows and up to 16 TB tokens; its W waves take the blocks of 128 columns in turn, operands
// straight from memory into registers (each weight byte is used by one wave, the tokens' codes stay in the L2), D steps
// ahead.  Nothing is shared and nothing waits for another wave before the end, where the W sums meet in LDS in the order
// of the waves.  One workgroup reads all of K, so there is no second launch and no workspace for the sums.
//
// 5 tokens of 17,408 x 5,120 take 15.5 to 16.6 us (89 MB, 5.4 to 5.7 TB/s; a kernel that only reads does 5.4 over 96
// MiB), 8 of 5,120 x 34,816 31 us (5.7 TB/s): the weight's bytes are what bounds it.  A small weight is three dependent
// trips to memory and the joining of the sums: 1 token of 1,024 x 1,024 3.8 us.
//
// FUSED: x comes as bf16 and every workgroup quantizes the tokens itself, in operand layout: a lane holds a quarter of a
// block of one token.  That saves a launch (about 2 us) and costs about a thousand cycles a step, so it is for rows of
// few steps.
#include "block_choice.h"
#include "block_math.h"
#include "decode.h"
#include "layer.h"

namespace w8a8 {
namespace {

using namespace lm;

// One step of a wave: 128 columns of 16 RB weight rows and 16 TB tokens, and the scales.
template <int RB, int TB, bool FUSED>
struct Step {
  i32x8 w[RB];
  i32x8 x[FUSED ? 1 : TB];
  u32x4 raw[FUSED ? 4 : 1];
  float sx[TB], sw;
};

template <int W, int RB, int TB, int D, bool FUSED>
__global__ void __launch_bounds__(64 * W)
block_few(const uint16_t* __restrict__ xb, const uint8_t* __restrict__ q, const float* __restrict__ s, const uint8_t* __restrict__ w,
          const float* __restrict__ sw, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int M, int64_t N, int K, int64_t first) {
  static_assert(!FUSED || TB == 1, "fused: one block of tokens");
  constexpr int CB = RB * TB < 4 ? RB * TB : 4;            // 16 x 16 blocks that meet at a time
  __shared__ __attribute__((aligned(16))) f32x4 red[W][CB][64];
  const int tid = threadIdx.x, l = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = l & 15, h = l >> 4;
  const int64_t n0 = (first + blockIdx.x) * (16 * RB);
  const int blocks = K / kScaleBlock, steps = blocks > wave ? (blocks - 1 - wave) / W + 1 : 0;
  const int64_t s_ld = block_scale_stride(M);

  // 32-bit places of this lane's bytes within the workgroup's rows and the tokens, at block 0
  const int64_t row0 = n0 / 32 * 32;
  uint32_t wo[RB], qo[TB];
  uint32_t mt[TB];
  auto place = [&](int row) -> uint32_t { return (uint32_t)(row / 32) * 32 * (uint32_t)K + row % 32 * 64 + 16 * h; };
#pragma unroll
  for (int i = 0; i < RB; ++i) wo[i] = place((int)min(n0 + 16 * i + c, N - 1) - (int)row0);
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    mt[j] = (uint32_t)min(16 * j + c, M - 1);
    qo[j] = place((int)mt[j]);
  }
  const Buffer wbuf = buffer(w + row0 * K), qbuf = buffer(q), sbuf = buffer(s), xbuf = buffer(xb);
  const float* swp = sw + n0 / kScaleBlock * blocks;

  using S = Step<RB, TB, FUSED>;
  auto load = [&](S& t, int step) __attribute__((always_inline)) {
    const int b = min(wave + W * step, blocks - 1);    // (past the last step: read again, not used)
#pragma unroll
    for (int i = 0; i < RB; ++i) t.w[i] = load_operand(wbuf, wo[i], (uint32_t)b * 4096);
    if constexpr (FUSED) {
#pragma unroll
      for (int i = 0; i < 4; ++i)                           // columns 16 h .. + 15, 64 + 16 h .. + 15
        t.raw[i] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)((mt[0] * K + 16 * h + 64 * (i / 2)) * 2 + 16 * (i % 2)), b * 256, 0);
    } else {
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        t.x[j] = load_operand(qbuf, qo[j], (uint32_t)b * 4096);
        t.sx[j] = load_scale(sbuf, 4 * mt[j], (uint32_t)(b * s_ld) * 4);
      }
    }
    t.sw = swp[b];
  };

  f32x4 acc[RB][TB];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](S& t) __attribute__((always_inline)) {
    if constexpr (FUSED) {
      float v[32], m = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[8 * i + 2 * e] = qm::bf16lo(t.raw[i][e]);
          v[8 * i + 2 * e + 1] = qm::bf16hi(t.raw[i][e]);
        }
#pragma unroll
      for (int i = 0; i < 32; ++i) m = larger(m, fabsf(v[i]));
      t.sx[0] = max_quarters(m) / 448.0f;
      const qm::QuotientScale qs = qm::quotient_scale(t.sx[0]);
      qm::apply_prefactor(v, qs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float g[8] = {v[8 * i], v[8 * i + 1], v[8 * i + 2], v[8 * i + 3], v[8 * i + 4], v[8 * i + 5], v[8 * i + 6], v[8 * i + 7]};
        const u32x2 k = e4m3_codes8(g, qs);
        t.x[0][2 * i] = (int)k[0];
        t.x[0][2 * i + 1] = (int)k[1];
      }
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const float by = t.sx[j] * t.sw;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const f32x4 part = mfma128(t.w[i], t.x[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(part[e], by, acc[i][j][e]);
      }
      // (16 products at a time need more registers than there are)
      if constexpr (RB * TB > 4) __builtin_amdgcn_sched_barrier(0);
    }
  };

  S ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], d);
  int i = 0;
  for (; i + D <= steps; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(ring[d]);
      load(ring[d], i + d + D);
    }
  }
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (i + d < steps) multiply(ring[d]);

#pragma unroll
  for (int r = 0; r < RB * TB / CB; ++r) {
    if (r) __syncthreads();
#pragma unroll
    for (int b = 0; b < CB; ++b) red[wave][b][l] = acc[(r * CB + b) % RB][(r * CB + b) / RB];
    __syncthreads();
    if (tid < CB * 64) {                                   // (whole waves)
      const int at = tid / 64, b = r * CB + at, i = b % RB, j = b / RB, m = 16 * j + c;
      f32x4 sum = red[0][at][l];
#pragma unroll
      for (int v = 1; v < W; ++v) sum += red[v][at][l];
      const int64_t n = n0 + 16 * i + 4 * h;
      if (m < M && n < N) store_row4(sum, bias, y, m, n, N);
    }
  }
}

template <int W, int RB, int TB, int D, bool FUSED>
hipError_t launch(const uint16_t* x, const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y,
                  int64_t M, int64_t N, int64_t K, hipStream_t stream) {
  return in_launches((N + 16 * RB - 1) / (16 * RB), 1, 64 * W, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((block_few<W, RB, TB, D, FUSED>), dim3((unsigned)count), dim3(64 * W), 0, stream, x, q, s, w, sw, bias, y, (int)M, N,
                       (int)K, first);
    return hipGetLastError();
  });
}

}  // namespace

bool block_few_fits(int64_t M, int64_t N, int64_t K) { return block_choice::few_fits(M, N, K); }

// Weight rows of a workgroup: 16 while that gives one workgroup a CU at most (12 tokens of 4,096 x 4,096 5.7 us, 6.2
// with 32 rows; 24 tokens 5.7 and 6.6; 48 tokens 7.4 and 8.7) and, up to 16 tokens, where it gives many (8 tokens of
// 5,120 x 34,816 31.1 and 33.1 us); 32 between, where 16 leave a second round of CUs half empty (5 tokens of 17,408 x
// 5,120 22.4 and 18.6 us) and for more tokens.
hipError_t launch_block_few(const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y, int64_t M,
                            int64_t N, int64_t K, hipStream_t stream) {
  const int64_t blocks = (N + 15) / 16;
  if (M <= 16) {
    if (blocks > 256 && blocks <= 384) return launch<8, 2, 1, 2, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
    return launch<8, 1, 1, 6, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
  }
  if (M > 64) return hipErrorInvalidValue;
  if (M <= 32) {
    if (blocks <= 256) return launch<4, 1, 2, 3, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
    return launch<4, 2, 2, 3, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
  }
  if (blocks <= 256) return launch<4, 1, 4, 3, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
  return launch<4, 2, 4, 2, false>(nullptr, q, s, w, sw, bias, y, M, N, K, stream);
}

bool block_fused_fits(int64_t M, int64_t N, int64_t K) { return block_choice::fused_fits(M, N, K); }

hipError_t launch_block_fused(const uint16_t* x, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                              int64_t K, hipStream_t stream) {
  return launch<block_choice::kFusedWaves, 1, 1, 2, true>(x, nullptr, nullptr, w, sw, bias, y, M, N, K, stream);
}

}  // namespace w8a8
