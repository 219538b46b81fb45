// The operators for few tokens: host-side launch interface between their C entry points
// (decode_api.cpp) and their kernel sources.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace w8a8 {

// Workgroups of one launch: a grid has fewer than 2^32 work items along x, and a launch past that reports
// success and runs the remainder only.  What does not fit goes out in several launches.
constexpr int64_t most_blocks(int threads) { return 0xffffffffLL / threads; }

// launch(first, count) over `all` parts of `blocks` workgroups each, as many parts at a time as fit; an error if one
// alone does not.
template <typename F>
hipError_t in_launches(int64_t all, int64_t blocks, int threads, F launch) {
  const int64_t most = most_blocks(threads) / blocks;
  if (most < 1) return hipErrorInvalidValue;
  for (int64_t first = 0; first < all; first += most) {
    const hipError_t e = launch(first, all - first < most ? all - first : most);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// 4-bit weights (w4.hip).  Row-major codes [N, K / 2] and bf16 scales [N, K / group];
// packed: blocks of 16 rows x 128 columns (layout in w8a8.h), rows rounded up to 16.
hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, uint8_t* codes,
                              uint16_t* scales, hipStream_t stream);
hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, int group,
                          uint8_t* codes_packed, uint16_t* scales_packed, hipStream_t stream);
hipError_t launch_w4_linear(const uint16_t* x, const uint8_t* codes_packed, const uint16_t* scales_packed,
                            const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int group,
                            void* workspace, hipStream_t stream);
// Parts of K whose fp32 sums [splits][min(M, kSplitTokens)][N] the workspace holds (1: none): more tokens are served
// kSplitTokens at a time.
constexpr int64_t kSplitTokens = 1024;
int w4_splits(int64_t N, int64_t K);

// A paged cache of int8 codes as the kernels see it (pointers of w8a8.h's cache
// arguments): code pages [pages][heads][page][dim], scales [pages][heads].
struct KvCache {
  int8_t* k_codes;
  int8_t* v_codes;
  float* k_scale;
  float* v_scale;
  const int32_t* table;   // [seqs][width] page of each block of `page` tokens
  const int32_t* lens;    // [seqs] tokens held, the newest call's included
  int64_t pages, width;
  int heads, dim, page;
  KvCache from(int64_t seq) const {   // the sequences from `seq` on
    KvCache c = *this;
    c.table += seq * width;
    c.lens += seq;
    return c;
  }
};

// New rows k, v (kv_cache.hip): token t of sequence b at k + (b * tokens + t) * ldk.
hipError_t launch_kv_append(const KvCache& c, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                            int64_t seqs, int64_t tokens, hipStream_t stream);
hipError_t launch_kv_read(const KvCache& c, int64_t seqs, int64_t length, uint16_t* k, uint16_t* v,
                          hipStream_t stream);

// Attention over the cache (attention.hip).  kv_attention_splits: the number of
// pieces that each sequence's tokens are cut into (1: no workspace is used).
int64_t kv_attention_splits(int64_t seqs, int64_t tokens, int q_heads, int heads, int dim, int page, int64_t width);
hipError_t launch_kv_attention(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens,
                               int q_heads, float scale, uint16_t* y, void* workspace, hipStream_t stream);

}  // namespace w8a8
