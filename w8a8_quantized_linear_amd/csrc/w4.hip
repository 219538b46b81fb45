// Projections of a few tokens with 4-bit weights.
//
// What it computes: y[m][n] = bf16( sum_g s[n][g] * sum_{k in g} x[m][k] * c[n][k] + bias[n] ) with codes
// c in [-8, 7], one bf16 scale for each row and group of 32, 64 or 128 columns, bf16 activations and
// fp32 sums.  For a few tokens the weight codes are the traffic (half a byte for every 2M operations),
// so the kernel is built around one pass over them.
#include "epilogue_math.h"
#include "internal.h"

namespace w8a8 {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;          // rows of a packed block (an MFMA operand's rows)
constexpr int kCols = 128;         // columns of a packed block
constexpr int kBlockBytes = kRows * kCols / 2;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return (uint16_t)bf16x2_rne(f, 0.0f); }

// ---- quantizer: rows of w -> row-major codes and scales ------------------------
// One thread per 8 columns, group / 8 neighbouring lanes per group: s = bf16(amax / 7), codes
// RNE(w / s) clamped to +-7 (the rounded scale may be below amax / 7, by up to 2^-9 of it).
__global__ void __launch_bounds__(256)
w4_quantize_kernel(const uint16_t* __restrict__ w, int64_t chunks, int lanes, uint32_t* __restrict__ codes,
                   uint16_t* __restrict__ scales) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool live = j < chunks;
  const u32x4 raw = *reinterpret_cast<const u32x4*>(w + 8 * (live ? j : chunks - 1));
  float v[8], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(raw[i] << 16);
    v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  for (int d = 1; d < lanes; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
  const uint16_t sb = f32_to_bf16(amax / 7.0f);
  const float s = bf16_to_f32(sb);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = s > 0.0f ? fminf(fmaxf(rintf(v[i] / s), -7.0f), 7.0f) : 0.0f;
    word |= (uint32_t)((int)c + 8) << (4 * i);
  }
  if (!live) return;
  codes[j] = word;
  if (j % lanes == 0) scales[j / lanes] = sb;
}

// ---- row-major codes and scales -> the packed layout ------------------------------
// One thread per word of 8 codes: element i of the row-major word is nibble i; in the packed word the even
// elements 2p sit at bits 4p and the odd ones at 16 + 4p, so that one shift and mask give an aligned pair.
__global__ void __launch_bounds__(256)
w4_pack_codes_kernel(const uint32_t* __restrict__ codes, int64_t N, int64_t K, int64_t words, uint32_t* __restrict__ out) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= words) return;
  const int st = j % 4, r = j / 4 % 16, h = j / 64 % 4;
  const int64_t block = j / 256, kb = block % (K / kCols), n = block / (K / kCols) * kRows + r;
  uint32_t word = 0x88888888u;                 // padding rows: code 0
  if (n < N) {
    const uint32_t c = codes[(n * K + kb * kCols + st * 32 + h * 8) / 8];
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= ((c >> (4 * i)) & 15u) << (4 * (i / 2) + 16 * (i % 2));
  }
  out[j] = word;
}

__global__ void __launch_bounds__(256)
w4_pack_scales_kernel(const uint16_t* __restrict__ scales, int64_t N, int64_t groups, int64_t total,
                      uint16_t* __restrict__ out) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= total) return;
  const int64_t r = j % kRows, g = j / kRows % groups, n = j / kRows / groups * kRows + r;
  out[j] = n < N ? scales[n * groups + g] : 0;
}

// ---- the projection --------------------------------------------------------------
// Eight nibbles of a packed word -> eight bf16 values 128 + (code + 8): a bf16 between 128 and 256 has
// steps of one, so the nibble is its low mantissa bits and one and-or makes two values.
__device__ __forceinline__ bf16x8 widen(uint32_t w) {
  u32x4 v;
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = ((w >> (4 * p)) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, v);
}

// A workgroup computes RB blocks of 16 rows for 16 * MB tokens; its waves take every WAVES-th block of 128
// columns and meet in LDS.  MFMA 16x16x32: A = weights (lane 16 h + r: row r, columns 8 h .. 8 h + 7 of a
// 32-column step), B = tokens, D: lane 16 h + t holds rows 4 h .. 4 h + 3 of token t.  The offset of the
// widened codes goes out in the accumulator: a group's sum starts at -136 * sum(x), itself an MFMA with
// a constant operand that the RB row blocks share.
template <int MB, int RB, int GPB, int WAVES>
__global__ void __launch_bounds__(64 * WAVES)
w4_linear_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint16_t* __restrict__ s,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t M, int64_t N, int64_t K) {
  __shared__ f32x4 red[WAVES][RB * MB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4, t = lane & 15;
  const int64_t blocks = (N + kRows - 1) / kRows, b0 = (int64_t)blockIdx.x * RB, m0 = (int64_t)blockIdx.y * 16 * MB;
  const int kb_all = (int)(K / kCols);

  const uint16_t* xp[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) xp[mb] = x + min(m0 + 16 * mb + t, M - 1) * K + 8 * h;   // past M: row M - 1, not stored
  const uint8_t* wp[RB];
  const uint16_t* sp[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int64_t block = min(b0 + rb, blocks - 1) * kb_all;
    wp[rb] = w + block * kBlockBytes + 16 * lane;
    sp[rb] = s + block * (GPB * kRows) + 4 * h;
  }
  const u32x4 offs = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};   // -136
  const bf16x8 minus136 = __builtin_bit_cast(bf16x8, offs);

  f32x4 tot[RB][MB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) tot[rb][mb] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int kb = wave; kb < kb_all; kb += WAVES) {
    u32x4 wv[RB];
    u32x2 sv[RB][GPB];
    bf16x8 xv[4][MB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) wv[rb] = *reinterpret_cast<const u32x4*>(wp[rb] + (int64_t)kb * kBlockBytes);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int g = 0; g < GPB; ++g)
        sv[rb][g] = *reinterpret_cast<const u32x2*>(sp[rb] + (kb * GPB + g) * kRows);
#pragma unroll
    for (int st = 0; st < 4; ++st)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) xv[st][mb] = *reinterpret_cast<const bf16x8*>(xp[mb] + kb * kCols + 32 * st);
    constexpr int SPG = 4 / GPB;               // MFMA steps per group
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      f32x4 base[MB];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        base[mb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < SPG; ++st)
          base[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(minus136, xv[g * SPG + st][mb], base[mb], 0, 0, 0);
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        f32x4 acc[MB];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[mb] = base[mb];
#pragma unroll
        for (int st = 0; st < SPG; ++st) {
          const bf16x8 a = widen(wv[rb][g * SPG + st]);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xv[g * SPG + st][mb], acc[mb], 0, 0, 0);
        }
        const u32x2 sw = sv[rb][g];
        const float sc[4] = {__uint_as_float(sw[0] << 16), __uint_as_float(sw[0] & 0xffff0000u),
                             __uint_as_float(sw[1] << 16), __uint_as_float(sw[1] & 0xffff0000u)};
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[rb][mb][i] = __builtin_fmaf(sc[i], acc[mb][i], tot[rb][mb][i]);
      }
    }
  }

#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) red[wave][rb * MB + mb][lane] = tot[rb][mb];
  __syncthreads();
  for (int j = threadIdx.x; j < RB * MB * 64; j += 64 * WAVES) {
    const int rb = j / 64 / MB, mb = j / 64 % MB, l = j % 64;
    const int64_t m = m0 + 16 * mb + l % 16, n = (b0 + rb) * kRows + 4 * (l / 16);
    if (m >= M || n >= N) continue;            // N % 8 == 0: the four rows are whole or absent
    f32x4 v = red[0][rb * MB + mb][l];
#pragma unroll
    for (int wv = 1; wv < WAVES; ++wv) v += red[wv][rb * MB + mb][l];
    if (bias) {
      float bv[4];
      bf16x4(*reinterpret_cast<const uint2*>(bias + n), bv);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += bv[i];
    }
    *reinterpret_cast<u32x2*>(y + m * N + n) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  }
}

template <int MB, int RB, int WAVES>
hipError_t launch_linear(const uint16_t* x, const uint8_t* w, const uint16_t* s, const uint16_t* bias, uint16_t* y,
                         int64_t M, int64_t N, int64_t K, int group, hipStream_t stream) {
  const int64_t gx = ((N + kRows - 1) / kRows + RB - 1) / RB, gy = (M + 16 * MB - 1) / (16 * MB);
  if (gx > 0x7fffffff || gy > 65535) return hipErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)gy), block(64 * WAVES);
  if (group == 128)
    hipLaunchKernelGGL((w4_linear_kernel<MB, RB, 1, WAVES>), grid, block, 0, stream, x, w, s, bias, y, M, N, K);
  else if (group == 64)
    hipLaunchKernelGGL((w4_linear_kernel<MB, RB, 2, WAVES>), grid, block, 0, stream, x, w, s, bias, y, M, N, K);
  else
    hipLaunchKernelGGL((w4_linear_kernel<MB, RB, 4, WAVES>), grid, block, 0, stream, x, w, s, bias, y, M, N, K);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, uint8_t* codes,
                              uint16_t* scales, hipStream_t stream) {
  const int64_t chunks = N * K / 8, blocks = (chunks + 255) / 256;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(w4_quantize_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, w, chunks, group / 8,
                     reinterpret_cast<uint32_t*>(codes), scales);
  return hipGetLastError();
}

hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, int group,
                          uint8_t* codes_packed, uint16_t* scales_packed, hipStream_t stream) {
  const int64_t rows = (N + kRows - 1) / kRows * kRows, words = rows * K / 8, total = rows * (K / group);
  if ((words + 255) / 256 > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(w4_pack_codes_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, stream,
                     reinterpret_cast<const uint32_t*>(codes), N, K, words, reinterpret_cast<uint32_t*>(codes_packed));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(w4_pack_scales_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream, scales, N,
                     K / group, total, scales_packed);
  return hipGetLastError();
}

hipError_t launch_w4_linear(const uint16_t* x, const uint8_t* codes_packed, const uint16_t* scales_packed,
                            const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int group,
                            hipStream_t stream) {
  if (M <= 16) return launch_linear<1, 1, 8>(x, codes_packed, scales_packed, bias, y, M, N, K, group, stream);
  if (M <= 32) return launch_linear<2, 1, 8>(x, codes_packed, scales_packed, bias, y, M, N, K, group, stream);
  return launch_linear<4, 1, 8>(x, codes_packed, scales_packed, bias, y, M, N, K, group, stream);
}

}  // namespace w8a8
