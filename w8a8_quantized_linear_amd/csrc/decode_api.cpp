// Host side of the few-token entry points declared in include/w8a8.h (4-bit weights, the paged 8-bit cache and
// attention over it): argument checks and dispatch, in the order of the other entry points -- shapes and scalar
// arguments, then (if there is anything to do) pointers and alignment, then the device.
#include "w8a8.h"

#include <cmath>

#include "decode.h"
#include "entry.h"

namespace {

using w8a8::align256;
using w8a8::aligned16;
using w8a8::check_device;
using w8a8::launched;

constexpr int64_t kMaxRows = (int64_t)1 << 30;

bool group_ok(int group) { return group == 32 || group == 64 || group == 128; }

w8a8_status check_w4_shape(int64_t N, int64_t K, int group) {
  if (N < 0 || N > kMaxRows || K < 128 || K > W8A8_MAX_K || K % 128 != 0) return W8A8_ERR_BAD_SHAPE;
  return group_ok(group) ? W8A8_OK : W8A8_ERR_BAD_ARGUMENT;
}

w8a8_status check_cache_shape(int64_t seqs, int64_t heads, int64_t dim, int64_t page, int64_t pages, int64_t width) {
  if (seqs < 0 || seqs > W8A8_KV_MAX_SEQS || heads < 1 || heads > W8A8_KV_MAX_HEADS) return W8A8_ERR_BAD_SHAPE;
  if ((dim != 64 && dim != 128) || (page != 16 && page != 32 && page != 64 && page != 128)) return W8A8_ERR_BAD_SHAPE;
  if (pages < 1 || pages > 0x7fffffff || width < 1 || width > W8A8_KV_MAX_LENGTH / page) return W8A8_ERR_BAD_SHAPE;
  return W8A8_OK;
}

bool ld_ok(int64_t ld, int64_t least) { return ld >= least && ld % 8 == 0 && ld <= ((int64_t)1 << 40); }

}  // namespace

extern "C" {

size_t w8a8_w4_code_bytes(int64_t N, int64_t K) {
  if (N <= 0 || K <= 0 || N > kMaxRows || K > W8A8_MAX_K) return 0;
  return (size_t)((N + 15) / 16 * 16) * (size_t)(K / 2);
}

size_t w8a8_w4_scale_bytes(int64_t N, int64_t K, int group) {
  if (N <= 0 || K <= 0 || N > kMaxRows || K > W8A8_MAX_K || !group_ok(group)) return 0;
  return (size_t)((N + 15) / 16 * 16) * (size_t)(K / group) * sizeof(uint16_t);
}

size_t w8a8_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || M > W8A8_W4_MAX_M || N > kMaxRows || K > W8A8_MAX_K) return 0;
  const int splits = w8a8::w4_splits(N, K);
  const int64_t tokens = M < w8a8::kSplitTokens ? M : w8a8::kSplitTokens;
  return splits == 1 ? 0 : align256((size_t)splits * (size_t)tokens * (size_t)N * sizeof(float));
}

w8a8_status w8a8_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, uint8_t* codes, uint16_t* scales,
                             hipStream_t stream) {
  w8a8_status st = check_w4_shape(N, K, group);
  if (st != W8A8_OK) return st;
  if (N == 0) return W8A8_OK;
  if (!w || !codes || !scales) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(w) || !aligned16(codes) || !aligned16(scales)) return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  return launched(w8a8::launch_w4_quantize(w, N, K, group, codes, scales, stream));
}

w8a8_status w8a8_w4_pack(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, int group,
                         uint8_t* codes_packed, uint16_t* scales_packed, hipStream_t stream) {
  w8a8_status st = check_w4_shape(N, K, group);
  if (st != W8A8_OK) return st;
  if (N == 0) return W8A8_OK;
  if (!codes || !scales || !codes_packed || !scales_packed) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(codes_packed) || !aligned16(scales_packed))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  return launched(w8a8::launch_w4_pack(codes, scales, N, K, group, codes_packed, scales_packed, stream));
}

w8a8_status w8a8_w4_linear(const uint16_t* x, const uint8_t* codes_packed, const uint16_t* scales_packed,
                           const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int group,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_w4_shape(N, K, group);
  if (st != W8A8_OK) return st;
  if (M < 0 || M > W8A8_W4_MAX_M || N < 1 || N % 8 != 0 || N > W8A8_W4_MAX_N) return W8A8_ERR_BAD_SHAPE;
  if (M > ((int64_t)1 << 40) / N) return W8A8_ERR_BAD_SHAPE;
  if (M == 0) return W8A8_OK;
  const size_t need = w8a8_w4_workspace_bytes(M, N, K);
  if (workspace_bytes < need) return W8A8_ERR_BAD_ARGUMENT;
  if (!x || !codes_packed || !scales_packed || !y || (need && !workspace)) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(x) || !aligned16(codes_packed) || !aligned16(scales_packed) || !aligned16(y) || (bias && !aligned16(bias)) ||
      (need && !aligned16(workspace)))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  return launched(w8a8::launch_w4_linear(x, codes_packed, scales_packed, bias, y, M, N, K, group, workspace, stream));
}

w8a8_status w8a8_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, int8_t* k_codes,
                           float* k_scale, int8_t* v_codes, float* v_scale, int64_t pages, const int32_t* table,
                           int64_t width, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t heads,
                           int64_t dim, int64_t page, hipStream_t stream) {
  w8a8_status st = check_cache_shape(seqs, heads, dim, page, pages, width);
  if (st != W8A8_OK) return st;
  if (tokens < 0 || tokens > W8A8_KV_MAX_TOKENS) return W8A8_ERR_BAD_SHAPE;
  if (!ld_ok(ldk, heads * dim) || !ld_ok(ldv, heads * dim)) return W8A8_ERR_BAD_SHAPE;
  const int64_t blocks = ((tokens + page - 2) / page + 1) * heads * 2;       // workgroups of a sequence
  if (seqs * blocks > 0x7fffffff || blocks > w8a8::most_blocks(256)) return W8A8_ERR_BAD_SHAPE;
  if (seqs == 0 || tokens == 0) return W8A8_OK;
  if (!k || !v || !k_codes || !k_scale || !v_codes || !v_scale || !table || !lens) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(k_scale) || !aligned16(v_codes) ||
      !aligned16(v_scale) || !aligned16(table) || !aligned16(lens))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  const w8a8::KvCache c{k_codes, v_codes, k_scale, v_scale, table, lens, pages, width, (int)heads, (int)dim, (int)page};
  return launched(w8a8::launch_kv_append(c, k, ldk, v, ldv, seqs, tokens, stream));
}

w8a8_status w8a8_kv_read(const int8_t* k_codes, const float* k_scale, const int8_t* v_codes, const float* v_scale,
                         int64_t pages, const int32_t* table, int64_t width, const int32_t* lens, int64_t seqs,
                         int64_t length, int64_t heads, int64_t dim, int64_t page, uint16_t* k, uint16_t* v,
                         hipStream_t stream) {
  w8a8_status st = check_cache_shape(seqs, heads, dim, page, pages, width);
  if (st != W8A8_OK) return st;
  if (length < 0 || length > W8A8_KV_MAX_LENGTH) return W8A8_ERR_BAD_SHAPE;
  if (seqs > 0 && length > (((int64_t)0x7fffffff << 8) / (heads * (dim / 8))) / seqs) return W8A8_ERR_BAD_SHAPE;
  if (length > 2048 / dim * w8a8::most_blocks(256)) return W8A8_ERR_BAD_SHAPE;
  if (seqs == 0 || length == 0) return W8A8_OK;
  if (!k || !v || !k_codes || !k_scale || !v_codes || !v_scale || !table || !lens) return W8A8_ERR_NULL_POINTER;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(k_scale) || !aligned16(v_codes) ||
      !aligned16(v_scale) || !aligned16(table) || !aligned16(lens))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  const w8a8::KvCache c{const_cast<int8_t*>(k_codes), const_cast<int8_t*>(v_codes), const_cast<float*>(k_scale),
                        const_cast<float*>(v_scale), table, lens, pages, width, (int)heads, (int)dim, (int)page};
  return launched(w8a8::launch_kv_read(c, seqs, length, k, v, stream));
}

size_t w8a8_kv_attention_workspace_bytes(int64_t seqs, int64_t tokens, int64_t q_heads, int64_t heads, int64_t dim,
                                         int64_t page, int64_t width) {
  if (check_cache_shape(seqs, heads, dim, page, 1, width) != W8A8_OK) return 0;
  if (seqs == 0 || tokens < 1 || tokens > W8A8_KV_MAX_TOKENS || q_heads < heads || q_heads > W8A8_KV_MAX_HEADS ||
      q_heads % heads != 0)
    return 0;
  const int64_t splits = w8a8::kv_attention_splits(seqs, tokens, (int)q_heads, (int)heads, (int)dim, (int)page, width);
  return splits == 1 ? 0 : align256((size_t)(seqs * tokens * q_heads * splits) * (size_t)(dim + 2) * sizeof(float));
}

w8a8_status w8a8_kv_attention(const uint16_t* q, int64_t ldq, const int8_t* k_codes, const float* k_scale,
                              const int8_t* v_codes, const float* v_scale, int64_t pages, const int32_t* table,
                              int64_t width, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t q_heads,
                              int64_t heads, int64_t dim, int64_t page, float scale, uint16_t* y, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  w8a8_status st = check_cache_shape(seqs, heads, dim, page, pages, width);
  if (st != W8A8_OK) return st;
  if (tokens < 0 || tokens > W8A8_KV_MAX_TOKENS || q_heads < heads || q_heads > W8A8_KV_MAX_HEADS || q_heads % heads != 0)
    return W8A8_ERR_BAD_SHAPE;
  if (!ld_ok(ldq, q_heads * dim) || seqs * tokens * q_heads > 0x7fffffff) return W8A8_ERR_BAD_SHAPE;
  if (!std::isfinite(scale)) return W8A8_ERR_BAD_ARGUMENT;
  if (seqs == 0 || tokens == 0) return W8A8_OK;
  const size_t need = w8a8_kv_attention_workspace_bytes(seqs, tokens, q_heads, heads, dim, page, width);
  if (workspace_bytes < need) return W8A8_ERR_BAD_ARGUMENT;
  if (!q || !y || !k_codes || !k_scale || !v_codes || !v_scale || !table || !lens || (need && !workspace))
    return W8A8_ERR_NULL_POINTER;
  if (!aligned16(q) || !aligned16(y) || !aligned16(k_codes) || !aligned16(k_scale) || !aligned16(v_codes) ||
      !aligned16(v_scale) || !aligned16(table) || !aligned16(lens) || (need && !aligned16(workspace)))
    return W8A8_ERR_MISALIGNED;
  if ((st = check_device()) != W8A8_OK) return st;
  const w8a8::KvCache c{const_cast<int8_t*>(k_codes), const_cast<int8_t*>(v_codes), const_cast<float*>(k_scale),
                        const_cast<float*>(v_scale), table, lens, pages, width, (int)heads, (int)dim, (int)page};
  return launched(w8a8::launch_kv_attention(c, q, ldq, seqs, tokens, (int)q_heads, scale, y, workspace, stream));
}

}  // extern "C"
