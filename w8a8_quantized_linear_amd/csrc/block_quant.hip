// E4M3 codes with block scales: one for each 128 columns of an activation's row, one for each 128 x 128 block of a
// weight.  scale = amax / 448, code = the nearest E4M3 value to x / scale; a block of zeros has scale 0 and codes 0, one with
// a NaN a NaN for its scale.
#include "decode.h"
#include "layer.h"
#include "layer_math.h"

namespace w8a8 {
namespace {

using namespace lm;

constexpr int kThreads = 256;   // of the weight's quantizer

// A workgroup of T threads for each row, V pieces of 8 columns a thread, T * 8 columns apart, so that 16 lanes hold a
// block of 128: two bytes read and one written a value, nothing shared between waves.  (Threads dealt over rows and
// columns alike need a division each, which takes longer than the rest for few rows: 5 x 17,408 5.0 us, 3.6 this way.)
// Bound by memory for many rows, 4,000 x 16,384 37.6 us (5.2 TB/s), and by three dependent steps for few.
template <int V>
__global__ void __launch_bounds__(1024)
quantize_block(const uint16_t* __restrict__ x, int64_t M, int K, bool packed, uint8_t* __restrict__ q, float* __restrict__ s_out, int64_t first) {
  const int tid = threadIdx.x, T = blockDim.x;
  const int64_t row = first + xcd_order(blockIdx.x, gridDim.x), at = row * K;
  u32x4 raw[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * T + tid) * 8;
    raw[j] = *reinterpret_cast<const u32x4*>(x + at + (e < K ? e : 0));
  }
  const int64_t s_ld = packed ? block_scale_stride(M) : K / kScaleBlock;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = (j * T + tid) * 8;
    float v[8], m = 0.0f;
    widen8(raw[j], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = larger(m, fabsf(v[i]));
    const float s = max16(m) / 448.0f;
    const qm::QuotientScale qs = qm::quotient_scale(s);
    qm::apply_prefactor(v, qs);
    const u32x2 c = e4m3_codes8(v, qs);
    if (e >= K) continue;                            // (16 lanes together: K is a multiple of 128)
    if ((tid & 15) == 0) s_out[packed ? e / kScaleBlock * s_ld + row : row * s_ld + e / kScaleBlock] = s;
    *reinterpret_cast<u32x2*>(q + code_at(row, e, K, packed)) = c;
  }
}

// A workgroup for each 128 x 128 block: thread t holds rows t / 16 + 16 i, columns 8 (t % 16).
__global__ void __launch_bounds__(kThreads)
quantize_weight_block(const uint16_t* __restrict__ w, int64_t N, int64_t K, uint8_t* __restrict__ q, float* __restrict__ s_out, int64_t first) {
  const int64_t block = first + blockIdx.x, per_row = K / kScaleBlock;
  const int64_t n0 = block / per_row * kScaleBlock + threadIdx.x / 16, k0 = block % per_row * kScaleBlock + threadIdx.x % 16 * 8;
  float v[8][8], m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    widen8(*reinterpret_cast<const u32x4*>(w + min(n0 + 16 * i, N - 1) * K + k0), v[i]);    // (past N: the last row again)
#pragma unroll
    for (int e = 0; e < 8; ++e) m = larger(m, fabsf(v[i][e]));
  }
  __shared__ float red[kThreads / 64];
  m = max64(m);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = m;
  __syncthreads();
  const float s = larger(larger(red[0], red[1]), larger(red[2], red[3])) / 448.0f;
  const qm::QuotientScale qs = qm::quotient_scale(s);
  if (threadIdx.x == 0) s_out[block] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    qm::apply_prefactor(v[i], qs);
    if (n0 + 16 * i < N) *reinterpret_cast<u32x2*>(q + (n0 + 16 * i) * K + k0) = e4m3_codes8(v[i], qs);
  }
}

}  // namespace

hipError_t launch_quantize_block(const uint16_t* x, int64_t M, int64_t K, bool packed, uint8_t* q, float* s, hipStream_t stream) {
  // (From 257 rows on, up to 16,384 columns, at most 512 threads with more pieces each, so beyond 4,096 columns two where one would
  // do in up to 1,024: 12,016 x 5,120 36 us, 42 with one, 2,270 x 8,192 13.7 and 14.5; but 1,502 x 5,120 7.4 and 6.8, 300 x 5,120
  // 3.3 and 3.2.)
  const int pieces = (int)(K / 8), most = M <= 256 || pieces > 2048 ? 1024 : 512, least = (pieces + most - 1) / most;
  auto run = [&](auto kernel, int v) {
    const int T = ((pieces + v - 1) / v + 63) / 64 * 64;
    return in_launches(M, 1, T, [&](int64_t first, int64_t count) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)count), dim3((unsigned)T), 0, stream, x, M, (int)K, packed, q, s, first);
      return hipGetLastError();
    });
  };
  if (least <= 1) return run(quantize_block<1>, 1);
  if (least <= 2) return run(quantize_block<2>, 2);
  if (least <= 3) return run(quantize_block<3>, 3);
  if (least <= 4) return run(quantize_block<4>, 4);
  if (least <= 8) return run(quantize_block<8>, 8);
  return run(quantize_block<16>, 16);
}

hipError_t launch_quantize_weight_block(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* s, hipStream_t stream) {
  const int64_t blocks = (N + kScaleBlock - 1) / kScaleBlock * (K / kScaleBlock);
  return in_launches(blocks, 1, kThreads, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL(quantize_weight_block, dim3((unsigned)count), dim3(kThreads), 0, stream, w, N, K, q, s, first);
    return hipGetLastError();
  });
}

}  // namespace w8a8
