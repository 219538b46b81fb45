// Root-mean-square norm of rows, after the residual's addition, as bf16 or in 8 bits.
//
// What it computes, for a row x of K bf16 values:
//   h = bf16(x + residual) (fp32 sum; x without a residual), written out for the next addition;
//   z = h * weight, exact in fp32 (8 + 8 bits), z rotated by the normalized transform in blocks of 128 where asked;
//   r = 1 / sqrt(mean(h^2) + eps);
//   bf16: y = bf16(z r);
//   int8, E4M3: scale (amax / 127, amax / 448) r over the row or over each 128 columns, codes of z over amax / 127
//   (448).  r is in the scale alone: it is common to a row, so codes of z are codes of y, and y is not rounded on
//   the way.  That also leaves one reduction: sum of squares and amax of z meet in one exchange.
#include "decode.h"
#include "layer.h"
#include "layer_math.h"

namespace w8a8 {
namespace {

using namespace lm;

constexpr float kInvSqrt128 = 0x1.6a09e6p-4f;   // fl32(2^-3.5)

// The normalized transform of the 128 values that 16 lanes hold, eight each in order: element bits 0 to 2 within the
// lane, 3 to 6 across.  fp32: seven additions a value, each off by half a step of a partial sum.
__device__ __forceinline__ void rotate128(float (&v)[8], int lane) {
#pragma unroll
  for (int b = 1; b < 8; b <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & b)) {
        const float p = v[j], q = v[j | b];
        v[j] = p + q;
        v[j | b] = p - q;
      }
  const float s1 = lane & 1 ? -1.0f : 1.0f, s2 = lane & 2 ? -1.0f : 1.0f, s4 = lane & 4 ? -1.0f : 1.0f, s8 = lane & 8 ? -1.0f : 1.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = __builtin_fmaf(s1, v[j], qm::dpp_move<kXor1>(v[j]));
    v[j] = __builtin_fmaf(s2, v[j], qm::dpp_move<kXor2>(v[j]));
    v[j] = __builtin_fmaf(s4, v[j], qm::dpp_move<kHalfMirror>(qm::dpp_move<kXor3>(v[j])));   // 7 - (i ^ 3) = i ^ 4
    v[j] = __builtin_fmaf(s8, v[j], qm::dpp_move<kXor8>(v[j]));
    v[j] *= kInvSqrt128;
  }
}

// A workgroup of T threads for each row; a thread holds V pieces of 8 columns, T * 8 columns apart, so that every load
// and store of a wave is one run of memory and 16 lanes hold a block of 128 columns.
template <int V, NormOut OUT, bool ROT>
__global__ void __launch_bounds__(1024)
norm_rows(Norm n, int64_t first) {
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63;
  const int64_t K = n.K, row = first + xcd_order(blockIdx.x, gridDim.x);
  const int64_t at = row * K;
  u32x4 hv[V], wv[V];
  float z[V][8];
  bool in[V];
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = (int64_t)(j * T + tid) * 8 < K;
#pragma unroll
  for (int j = 0; j < V; ++j) hv[j] = *reinterpret_cast<const u32x4*>(n.x + at + (in[j] ? (j * T + tid) * 8 : 0));
  if (n.residual) {
    u32x4 rv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) rv[j] = *reinterpret_cast<const u32x4*>(n.residual + at + (in[j] ? (j * T + tid) * 8 : 0));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float a[8], b[8];
      widen8(hv[j], a);
      widen8(rv[j], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      hv[j] = narrow8(a);
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) wv[j] = *reinterpret_cast<const u32x4*>(n.weight + (in[j] ? (j * T + tid) * 8 : 0));
  if (n.h) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (in[j]) *reinterpret_cast<u32x4*>(n.h + at + (j * T + tid) * 8) = hv[j];
  }

  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float h[8], w[8];
    widen8(hv[j], h);
    widen8(wv[j], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[i] = in[j] ? h[i] : 0.0f;                       // (16 lanes of a block of 128 are in or out together)
      sum[i & 3] = __builtin_fmaf(h[i], h[i], sum[i & 3]);
      z[j][i] = h[i] * w[i];
    }
    if constexpr (ROT) rotate128(z[j], lane);
    if constexpr (OUT == NormOut::kI8 || OUT == NormOut::kFp8) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(z[j][i]));
    }
  }
  __shared__ float red[2][16];
  float total = sum64((sum[0] + sum[1]) + (sum[2] + sum[3]));
  if constexpr (OUT == NormOut::kI8 || OUT == NormOut::kFp8) top = max64(top);
  if (T > 64) {
    if (lane == 0) {
      red[0][tid >> 6] = total;
      red[1][tid >> 6] = top;
    }
    __syncthreads();
    total = 0.0f;
    for (int w = 0; w < T >> 6; ++w) {
      total += red[0][w];
      top = fmaxf(top, red[1][w]);
    }
  }
  const float r = 1.0f / sqrtf(total / (float)K + n.eps);

  if constexpr (OUT == NormOut::kBf16) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] *= r;
      if (in[j]) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(n.out) + at + (j * T + tid) * 8) = narrow8(z[j]);
    }
  } else {
    uint8_t* q = static_cast<uint8_t*>(n.out);
    qm::QuotientScale qs;
    if constexpr (OUT != NormOut::kBlock) {
      const float s = top / (OUT == NormOut::kI8 ? 127.0f : 448.0f);
      if (tid == 0) n.scales[row] = s * r;
      qs = qm::quotient_scale(s);
    }
    const int64_t s_ld = n.packed ? block_scale_stride(n.M) : K / kScaleBlock;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t e = (int64_t)(j * T + tid) * 8;
      if constexpr (OUT == NormOut::kBlock) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(z[j][i]));
        const float s = max16(m) / 448.0f;
        qs = qm::quotient_scale(s);
        if (in[j] && (lane & 15) == 0) n.scales[n.packed ? e / kScaleBlock * s_ld + row : row * s_ld + e / kScaleBlock] = s * r;
      }
      qm::apply_prefactor(z[j], qs);
      const u32x2 c = OUT == NormOut::kI8 ? int8_codes8(z[j], qs) : e4m3_codes8(z[j], qs);
      if (in[j]) *reinterpret_cast<u32x2*>(q + code_at(row, e, K, n.packed)) = c;
    }
  }
}

template <int V>
hipError_t launch_v(const Norm& n, int T, hipStream_t stream) {
  return in_launches(n.M, 1, T, [&](int64_t first, int64_t count) {
    const dim3 grid((unsigned)count), block((unsigned)T);
    switch (n.kind) {
      case NormOut::kBf16: hipLaunchKernelGGL((norm_rows<V, NormOut::kBf16, false>), grid, block, 0, stream, n, first); break;
      case NormOut::kI8:
        if (n.rotate) hipLaunchKernelGGL((norm_rows<V, NormOut::kI8, true>), grid, block, 0, stream, n, first);
        else hipLaunchKernelGGL((norm_rows<V, NormOut::kI8, false>), grid, block, 0, stream, n, first);
        break;
      case NormOut::kFp8:
        if (n.rotate) hipLaunchKernelGGL((norm_rows<V, NormOut::kFp8, true>), grid, block, 0, stream, n, first);
        else hipLaunchKernelGGL((norm_rows<V, NormOut::kFp8, false>), grid, block, 0, stream, n, first);
        break;
      case NormOut::kBlock: hipLaunchKernelGGL((norm_rows<V, NormOut::kBlock, false>), grid, block, 0, stream, n, first); break;
    }
    return hipGetLastError();
  });
}

}  // namespace

// As few pieces a thread as fit: 12,016 x 5,120 with a residual and block scales 80.7 us with one piece in 640 threads, 87.6 with three
// in 256; 2,270 x 17,408 56.6 with three in 768, 63.1 with four in 576.  A row that is read alone and is no residual's is in flight
// for too short a time for that: 2,270 x 5,120 to E4M3 13.7 us with one piece in 640 threads, 10.6 with two in 320 (bf16, 4,000 x
// 8,192: 26.8 and 27.8).
hipError_t launch_norm(const Norm& n, hipStream_t stream) {
  const int64_t pieces = (n.K + 7) / 8;
  const int64_t most = n.residual || n.M <= 256 ? 1024 : 512;
  int64_t least = (pieces + most - 1) / most;
  if (least > 4) least = (pieces + 1023) / 1024;
  auto threads = [&](int64_t v) { return (int)(((pieces + v - 1) / v + 63) / 64 * 64); };
  if (least <= 1) return launch_v<1>(n, threads(1), stream);
  if (least <= 2) return launch_v<2>(n, threads(2), stream);
  if (least <= 3) return launch_v<3>(n, threads(3), stream);
  if (least <= 4) return launch_v<4>(n, threads(4), stream);
  if (least <= 8) return launch_v<8>(n, threads(8), stream);
  return launch_v<16>(n, threads(16), stream);
}

}  // namespace w8a8
