// Host side of the entry points for norms, rotary positions and E4M3 projections with block scales: argument checks and
// dispatch, in the order of the other entry points -- shapes and scalar arguments, then (if there is anything to do)
// pointers and alignment, then the device.
#include "w8a8.h"

#include <cmath>

#include "entry.h"
#include "layer.h"

namespace {

using w8a8::align256;
using w8a8::aligned16;
using w8a8::check_device;
using w8a8::kScaleBlock;
using w8a8::launched;
using w8a8::NormOut;

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxValues = (int64_t)1 << 42;

w8a8_status norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int rot_block, uint16_t* h,
                 void* out, float* scales, int64_t M, int64_t K, NormOut kind, bool packed, hipStream_t stream) {
  const int64_t unit = kind == NormOut::kBlock ? kScaleBlock : packed ? 64 : kind == NormOut::kBf16 ? 8 : 32;
  if (M < 0 || M > kMaxRows || K < unit || K > W8A8_MAX_K || K % unit != 0) return W8A8_ERR_BAD_SHAPE;
  if (rot_block != 0 && rot_block != 128) return W8A8_ERR_BAD_ARGUMENT;
  if (rot_block == 128 && K % 128 != 0) return W8A8_ERR_BAD_SHAPE;
  if (!std::isfinite(eps) || !(eps > 0.0f)) return W8A8_ERR_BAD_ARGUMENT;
  if (M == 0) return W8A8_OK;
  if (!x || !weight || !out || (kind != NormOut::kBf16 && !scales)) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(h) || !aligned16(out) || !aligned16(scales))
    return W8A8_ERR_MISALIGNED;
  const w8a8_status st = check_device();
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_norm({x, residual, weight, h, out, scales, M, K, eps, kind, rot_block == 128, packed}, stream));
}

w8a8_status quantize_block(const uint16_t* x, int64_t M, int64_t K, bool packed, uint8_t* q, float* s, hipStream_t stream) {
  if (M < 0 || K < kScaleBlock || K > W8A8_MAX_K || K % kScaleBlock != 0 || M > kMaxValues / K) return W8A8_ERR_BAD_SHAPE;
  if (M == 0) return W8A8_OK;
  if (!x || !q || !s) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(q) || !aligned16(s)) return W8A8_ERR_MISALIGNED;
  const w8a8_status st = check_device();
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_quantize_block(x, M, K, packed, q, s, stream));
}

w8a8_status check_block_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 0 || M > ((int64_t)1 << 30) || N < 1 || N > ((int64_t)1 << 28) - 32 || N % 8 != 0) return W8A8_ERR_BAD_SHAPE;
  if (K < kScaleBlock || K > W8A8_MAX_K || K % kScaleBlock != 0 || M > ((int64_t)1 << 40) / N) return W8A8_ERR_BAD_SHAPE;
  return W8A8_OK;
}

// And with x [M, K] to quantize.
w8a8_status check_linear_shape(int64_t M, int64_t N, int64_t K) {
  const w8a8_status st = check_block_shape(M, N, K);
  return st == W8A8_OK && M > kMaxValues / K ? W8A8_ERR_BAD_SHAPE : st;
}

// The packed codes of M tokens and their scales in a workspace.
size_t code_bytes(int64_t M, int64_t K) {
  const size_t rows = (size_t)w8a8::block_scale_stride(M);
  return align256(rows * (size_t)K) + align256((size_t)(K / kScaleBlock) * rows * sizeof(float));
}

bool ld_ok(int64_t ld, int64_t least) { return ld >= least && ld % 8 == 0 && ld <= ((int64_t)1 << 40); }

}  // namespace

extern "C" {

w8a8_status w8a8_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, uint16_t* h,
                         uint16_t* y, int64_t M, int64_t K, hipStream_t stream) {
  return norm(x, residual, weight, eps, 0, h, y, nullptr, M, K, NormOut::kBf16, false, stream);
}
w8a8_status w8a8_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, int rot_block,
                                  uint16_t* h, int8_t* q, float* s_tok, int64_t M, int64_t K, hipStream_t stream) {
  return norm(x, residual, weight, eps, rot_block, h, q, s_tok, M, K, NormOut::kI8, false, stream);
}
w8a8_status w8a8_rmsnorm_quantize_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                         int rot_block, uint16_t* h, int8_t* q_packed, float* s_tok, int64_t M, int64_t K,
                                         hipStream_t stream) {
  return norm(x, residual, weight, eps, rot_block, h, q_packed, s_tok, M, K, NormOut::kI8, true, stream);
}
w8a8_status w8a8_rmsnorm_quantize_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                      int rot_block, uint16_t* h, uint8_t* q, float* s_tok, int64_t M, int64_t K,
                                      hipStream_t stream) {
  return norm(x, residual, weight, eps, rot_block, h, q, s_tok, M, K, NormOut::kFp8, false, stream);
}
w8a8_status w8a8_rmsnorm_quantize_fp8_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                             int rot_block, uint16_t* h, uint8_t* q_packed, float* s_tok, int64_t M,
                                             int64_t K, hipStream_t stream) {
  return norm(x, residual, weight, eps, rot_block, h, q_packed, s_tok, M, K, NormOut::kFp8, true, stream);
}
w8a8_status w8a8_rmsnorm_quantize_block(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                        uint16_t* h, uint8_t* q, float* s, int64_t M, int64_t K, hipStream_t stream) {
  return norm(x, residual, weight, eps, 0, h, q, s, M, K, NormOut::kBlock, false, stream);
}
w8a8_status w8a8_rmsnorm_quantize_block_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                               uint16_t* h, uint8_t* q_packed, float* s, int64_t M, int64_t K,
                                               hipStream_t stream) {
  return norm(x, residual, weight, eps, 0, h, q_packed, s, M, K, NormOut::kBlock, true, stream);
}

w8a8_status w8a8_rope(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const uint64_t* turns, int64_t rotary,
                      int interleaved, float amplitude, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t q_heads,
                      int64_t heads, int64_t dim, uint16_t* q_out, int64_t ldq_out, uint16_t* k_out, int64_t ldk_out,
                      hipStream_t stream) {
  if (seqs < 0 || seqs > W8A8_KV_MAX_SEQS || tokens < 0 || tokens > W8A8_KV_MAX_TOKENS || seqs * tokens >= kMaxRows)
    return W8A8_ERR_BAD_SHAPE;
  if (q_heads < 1 || q_heads > W8A8_KV_MAX_HEADS || heads < 0 || heads > W8A8_KV_MAX_HEADS) return W8A8_ERR_BAD_SHAPE;
  if (dim < 16 || dim > 256 || dim % 16 != 0 || rotary < 16 || rotary > dim || rotary % 16 != 0) return W8A8_ERR_BAD_SHAPE;
  if (!ld_ok(ldq, q_heads * dim) || !ld_ok(ldq_out, q_heads * dim)) return W8A8_ERR_BAD_SHAPE;
  if (heads && (!ld_ok(ldk, heads * dim) || !ld_ok(ldk_out, heads * dim))) return W8A8_ERR_BAD_SHAPE;
  if (!std::isfinite(amplitude)) return W8A8_ERR_BAD_ARGUMENT;
  if (seqs == 0 || tokens == 0) return W8A8_OK;
  if ((q == q_out && ldq != ldq_out) || (heads && k == k_out && ldk != ldk_out)) return W8A8_ERR_BAD_ARGUMENT;
  if (!q || !q_out || !turns || !lens || (heads && (!k || !k_out))) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(q) || !aligned16(q_out) || !aligned16(turns) || !aligned16(lens) || (heads && (!aligned16(k) || !aligned16(k_out))))
    return W8A8_ERR_MISALIGNED;
  const w8a8_status st = check_device();
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_rope({q, k, q_out, k_out, ldq, ldk, ldq_out, ldk_out, turns, lens, seqs, tokens, (int)q_heads,
                                     (int)heads, (int)dim, (int)rotary, interleaved != 0, amplitude}, stream));
}

int64_t w8a8_block_scale_stride(int64_t M) { return M <= 0 || M > kMaxValues ? 0 : w8a8::block_scale_stride(M); }

w8a8_status w8a8_quantize_act_block(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* s, hipStream_t stream) {
  return quantize_block(x, M, K, false, q, s, stream);
}
w8a8_status w8a8_quantize_act_block_packed(const uint16_t* x, int64_t M, int64_t K, uint8_t* q_packed, float* s,
                                           hipStream_t stream) {
  return quantize_block(x, M, K, true, q_packed, s, stream);
}

w8a8_status w8a8_quantize_weight_block(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* s, hipStream_t stream) {
  if (N < 0 || K < kScaleBlock || K > W8A8_MAX_K || K % kScaleBlock != 0 || N > kMaxValues / K) return W8A8_ERR_BAD_SHAPE;
  if (N == 0) return W8A8_OK;
  if (!w || !q || !s) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(w) || !aligned16(q) || !aligned16(s)) return W8A8_ERR_MISALIGNED;
  const w8a8_status st = check_device();
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_quantize_weight_block(w, N, K, q, s, stream));
}

size_t w8a8_fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M <= 0 || check_block_shape(M, N, K) != W8A8_OK ? 0 : align256(w8a8::block_gemm_workspace(M, N, K));
}

w8a8_status w8a8_fp8_block_gemm_packed(const uint8_t* q_packed, const float* s, const uint8_t* w_packed, const float* s_w,
                                       const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_block_shape(M, N, K);
  if (st != W8A8_OK) return st;
  if (M == 0) return W8A8_OK;
  const size_t need = w8a8_fp8_block_gemm_workspace_bytes(M, N, K);
  if (workspace_bytes < need) return W8A8_ERR_BAD_ARGUMENT;
  if (!q_packed || !s || !w_packed || !s_w || !y || (need && !workspace)) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(q_packed) || !aligned16(s) || !aligned16(w_packed) || !aligned16(s_w) || !aligned16(bias) || !aligned16(y) ||
      (need && !aligned16(workspace)))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  return launched(w8a8::launch_block_gemm(q_packed, s, w_packed, s_w, bias, y, M, N, K, static_cast<float*>(workspace), stream));
}

size_t w8a8_fp8_block_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return M <= 0 || check_linear_shape(M, N, K) != W8A8_OK ? 0 : code_bytes(M, K) + w8a8_fp8_block_gemm_workspace_bytes(M, N, K);
}

w8a8_status w8a8_fp8_block_linear_packed(const uint16_t* x, const uint8_t* w_packed, const float* s_w, const uint16_t* bias,
                                         uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_linear_shape(M, N, K);
  if (st != W8A8_OK) return st;
  if (M == 0) return W8A8_OK;
  if (workspace_bytes < w8a8_fp8_block_workspace_bytes(M, N, K)) return W8A8_ERR_BAD_ARGUMENT;
  if (!x || !w_packed || !s_w || !y || !workspace) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(w_packed) || !aligned16(s_w) || !aligned16(bias) || !aligned16(y) || !aligned16(workspace))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  if (w8a8::block_fused_fits(M, N, K)) return launched(w8a8::launch_block_fused(x, w_packed, s_w, bias, y, M, N, K, stream));
  uint8_t* q = static_cast<uint8_t*>(workspace);
  float* s = reinterpret_cast<float*>(q + align256((size_t)w8a8::block_scale_stride(M) * (size_t)K));
  st = launched(w8a8::launch_quantize_block(x, M, K, true, q, s, stream));
  if (st != W8A8_OK) return st;
  return launched(w8a8::launch_block_gemm(q, s, w_packed, s_w, bias, y, M, N, K, reinterpret_cast<float*>(q + code_bytes(M, K)), stream));
}

}  // extern "C"
