// Root-mean-square norm of rows, after the residual's addition, as bf16 or in 8 bits.
//
// What it computes, for a row x of K bf16 values:
//   h = bf16(x + residual) (fp32 sum; x without a residual), written out for the next addition;
//   z = h * weight, exact in fp32 (8 + 8 bits; below 2^-126 a multiple of 2^-149), z rotated by the normalized transform
//   in blocks of 128 where asked;
//   r = 1 / sqrt(mean(h^2) + eps);
//   bf16: y = bf16(z r);
//   int8, E4M3: scale (amax / 127, amax / 448) r over the row or over each 128 columns, codes of z over amax / 127
//   (448).  r is in the scale alone: it is common to a row, so codes of z are codes of y, and y is not rounded on
//   the way.  That also leaves one reduction: sum of squares and amax of z meet in one exchange.
//
// A workgroup for each row, whose pieces stay in registers between the reduction and the output: everything is read and
// written once, and that is what bounds it.  12,016 x 5,120 with a residual and block scales 77 us (433 MB, 5.6 TB/s),
// 2,270 x 5,120 to E4M3 10.0 us (35 MB, 3.5 TB/s: a CU holds six workgroups of 320 threads, 1,536 in all, so the rows take
// one and a half rounds, of which the second is half empty); a single row is a load, two exchanges and a store one behind
// the other, 2.0 us in the kernel.
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

// bf16(x + residual) of a piece of 8 columns.
__device__ __forceinline__ u32x4 sum_of(u32x4 x, u32x4 r) {
  float a[8], b[8];
  widen8(x, a);
  widen8(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] += b[i];
  return narrow8(a);
}

// z of a piece, rotated where asked; adds the squares of h to sum.  Columns past the row's end count as zeros.  (16
// lanes of a block of 128 are in or out together.)
template <bool ROT>
__device__ __forceinline__ void scaled(u32x4 h4, u32x4 w4, bool in, int lane, float (&z)[8], float (&sum)[4]) {
  float h[8], w[8];
  widen8(in ? h4 : u32x4{0, 0, 0, 0}, h);
  widen8(in ? w4 : u32x4{0, 0, 0, 0}, w);   // (both: a zero times a weight that is not finite is a NaN)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sum[i & 3] = __builtin_fmaf(h[i], h[i], sum[i & 3]);
    z[i] = h[i] * w[i];
  }
  if constexpr (ROT) rotate128(z, lane);
}

__device__ __forceinline__ float top_of(const float (&z)[8], float top) {
#pragma unroll
  for (int i = 0; i < 8; ++i) top = larger(top, fabsf(z[i]));
  return top;
}

// Sum (and maximum) over the row's waves, the same in all of them.
template <bool MAX>
__device__ __forceinline__ void meet(float& total, float& top) {
  __shared__ float red[2][16];
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  total = sum64(total);
  if constexpr (MAX) top = max64(top);
  if (waves == 1) return;
  if ((tid & 63) == 0) {
    red[0][tid >> 6] = total;
    red[1][tid >> 6] = top;
  }
  __syncthreads();
  total = 0.0f;
  for (int w = 0; w < waves; ++w) {
    total += red[0][w];
    top = larger(top, red[1][w]);
  }
}

// What a row's pieces are written with: r, and the scale of z where the row has one.
template <NormOut OUT>
struct Out {
  float r;
  qm::QuotientScale qs;
  __device__ __forceinline__ Out(const Norm& n, int64_t row, float total, float top) : r(1.0f / sqrtf(total / (float)n.K + n.eps)) {
    if constexpr (OUT == NormOut::kI8 || OUT == NormOut::kFp8) {
      float s = top / (OUT == NormOut::kI8 ? 127.0f : 448.0f);
      // int8 codes have no clamp: amax / s is 127 but for half a step of fp32.  A scale below the normal range may be off by half
      // of itself; one that was rounded down so far goes up instead (1.496 * 2^-149 became 2^-149, and amax the code -66).
      if (OUT == NormOut::kI8 && 127.25f * s < top) s += 0x1p-149f;
      if (threadIdx.x == 0) n.scales[row] = s * r;
      qs = qm::quotient_scale(s);
    }
  }
  // the piece at column e (whole rows of 16 lanes call it)
  __device__ __forceinline__ void write(const Norm& n, int64_t row, int64_t e, bool in, int lane, float (&z)[8]) {
    if constexpr (OUT == NormOut::kBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] *= r;
      if (in) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(n.out) + row * n.K + e) = narrow8(z);
    } else {
      if constexpr (OUT == NormOut::kBlock) {
        const float s = max16(top_of(z, 0.0f)) / 448.0f;
        qs = qm::quotient_scale(s);
        const int64_t s_ld = n.packed ? block_scale_stride(n.M) : n.K / kScaleBlock;
        if (in && (lane & 15) == 0) n.scales[n.packed ? e / kScaleBlock * s_ld + row : row * s_ld + e / kScaleBlock] = s * r;
      }
      qm::apply_prefactor(z, qs);
      const u32x2 c = OUT == NormOut::kI8 ? int8_codes8(z, qs) : e4m3_codes8(z, qs);
      if (in) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(n.out) + code_at(row, e, n.K, n.packed)) = c;
    }
  }
};

// A workgroup of T threads for each row; a thread holds V pieces of 8 columns, T * 8 columns apart, so that every load
// and store of a wave is one run of memory and 16 lanes hold a block of 128 columns.
template <int V, NormOut OUT, bool ROT>
__global__ void __launch_bounds__(1024)
norm_rows(Norm n, int64_t first) {
  constexpr bool TOKEN = OUT == NormOut::kI8 || OUT == NormOut::kFp8;
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63;
  const int64_t K = n.K, row = first + xcd_order(blockIdx.x, gridDim.x), at = row * K;
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
    for (int j = 0; j < V; ++j) hv[j] = sum_of(hv[j], rv[j]);
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
    scaled<ROT>(hv[j], wv[j], in[j], lane, z[j], sum);
    if constexpr (TOKEN) top = top_of(z[j], top);
  }
  float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  meet<TOKEN>(total, top);
  Out<OUT> out(n, row, total, top);
#pragma unroll
  for (int j = 0; j < V; ++j) out.write(n, row, (int64_t)(j * T + tid) * 8, in[j], lane, z[j]);
}

// Rows of more columns than a workgroup's registers hold (K > 65,536): each piece is read twice, the second time out of
// a cache. 300 x 131,072 with a residual: 81 us (3.9 TB/s of what must move); with 16 pieces a thread in norm_rows,
// which spill, 250 us.
template <NormOut OUT, bool ROT>
__global__ void __launch_bounds__(1024)
norm_wide(Norm n, int64_t first) {
  constexpr bool TOKEN = OUT == NormOut::kI8 || OUT == NormOut::kFp8;
  const int tid = threadIdx.x, T = blockDim.x, lane = tid & 63, K = (int)n.K;
  const int64_t row = first + xcd_order(blockIdx.x, gridDim.x), at = row * n.K;
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, top = 0.0f;
  auto load = [&](const uint16_t* p, int e) __attribute__((always_inline)) { return *reinterpret_cast<const u32x4*>(p + (e < K ? e : 0)); };
  for (int base = 0; base < K; base += T * 8) {
    const int e = base + tid * 8;
    u32x4 h = load(n.x + at, e);
    if (n.residual) h = sum_of(h, load(n.residual + at, e));
    if (n.h && e < K) *reinterpret_cast<u32x4*>(n.h + at + e) = h;
    float z[8];
    scaled<ROT>(h, load(n.weight, e), e < K, lane, z, sum);
    if constexpr (TOKEN) top = top_of(z, top);
  }
  float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
  meet<TOKEN>(total, top);
  Out<OUT> out(n, row, total, top);
  // h where it was written (it may have taken x's or the residual's place), by this thread itself; otherwise from x again
  for (int base = 0; base < K; base += T * 8) {
    const int e = base + tid * 8;
    u32x4 h = load((n.h ? n.h : n.x) + at, e);
    if (!n.h && n.residual) h = sum_of(h, load(n.residual + at, e));
    float z[8], again[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    scaled<ROT>(h, load(n.weight, e), e < K, lane, z, again);
    out.write(n, row, e, e < K, lane, z);
  }
}

// V pieces a thread, or norm_wide (V = 0).
template <int V, NormOut OUT, bool ROT>
hipError_t launch_kernel(const Norm& n, int T, hipStream_t stream) {
  return in_launches(n.M, 1, T, [&](int64_t first, int64_t count) {
    const dim3 grid((unsigned)count), block((unsigned)T);
    if constexpr (V == 0) hipLaunchKernelGGL((norm_wide<OUT, ROT>), grid, block, 0, stream, n, first);
    else hipLaunchKernelGGL((norm_rows<V, OUT, ROT>), grid, block, 0, stream, n, first);
    return hipGetLastError();
  });
}

template <int V>
hipError_t launch_v(const Norm& n, int T, hipStream_t stream) {
  switch (n.kind) {
    case NormOut::kBf16: return launch_kernel<V, NormOut::kBf16, false>(n, T, stream);
    case NormOut::kI8: return n.rotate ? launch_kernel<V, NormOut::kI8, true>(n, T, stream) : launch_kernel<V, NormOut::kI8, false>(n, T, stream);
    case NormOut::kFp8: return n.rotate ? launch_kernel<V, NormOut::kFp8, true>(n, T, stream) : launch_kernel<V, NormOut::kFp8, false>(n, T, stream);
    case NormOut::kBlock: return launch_kernel<V, NormOut::kBlock, false>(n, T, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

// As few pieces a thread as fit: 12,016 x 5,120 with a residual and block scales 80.7 us with one piece in 640 threads,
// 87.6 with three in 256; 2,270 x 17,408 56.6 with three in 768, 63.1 with four in 576.  Without a residual
// half the threads with twice the pieces: 2,270 x 5,120 to E4M3 10.2 us with two in 320 threads, 12.4 with one in 640; bf16 9.5 and
// 10.5; 12,016 x 8,192 bf16 70 and 75, to int8 57 and 74; 300 x 5,120 bf16 3.3 and 3.5, with block scales 4.2 and 4.0 (the one
// of 49 measured, from 300 x 5,120 to 12,016 x 8,192, that loses).  Eight pieces, of which the block-scaled form spills three
// registers, still are the faster form: 300 x 65,536 with a residual 30.4 us, 32.4 in norm_wide.
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
  return launch_v<0>(n, 1024, stream);
}

}  // namespace w8a8
