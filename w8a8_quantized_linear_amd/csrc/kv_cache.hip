// A paged cache of keys and values in 8 bits: new tokens in, sequences back out.
//
// Layout.  A page holds `page` tokens of every head: int8 codes [pages][heads][page][dim] and one fp32 scale
// for each page and head, for keys and for values.  Token p of a sequence is row p % page of the page that
// the sequence's table names at p / page.
//
// What append computes, for each page and head that new tokens fall into: s = max(s_old, amax / 127), where
// amax is the largest magnitude among the new values there and s_old is the page's scale if it holds tokens
// of this sequence from before (0 if not); the codes held are moved to the new scale, c = RNE(c * (s_old / s)),
// and the new ones are RNE(x / s), the library's per-token rule with the scale of a block.  All steps are
// single fp32 operations, so the codes are the same on every run and machine.
//
// Bound: memory traffic (append 2 bytes read and 1 written per value, read 1 and 2) and, for single tokens,
// latency.  8 sequences of 1,502 tokens (8 heads of 128): append 17.8 us (4.1 TB/s), read 16.2 us (4.6 TB/s; a copy of
// 2 GiB reaches 4.9); one token for each of 61 sequences of up to 299 tokens 4.5 us, their read 8.6 us.
#include "decode.h"
#include "epilogue_math.h"
#include "quant_math.h"

namespace w8a8 {
namespace {

using namespace qm;
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

// The page of a sequence's block, or -1 where the table names none that exists.
__device__ __forceinline__ int64_t page_of(const KvCache& c, int64_t seq, int64_t block) {
  if (block >= c.width) return -1;
  const int32_t id = c.table[seq * c.width + block];
  return id >= 0 && id < c.pages ? id : -1;
}

// A sequence's length, and what of it its table row can address.
__device__ __forceinline__ int64_t len_of(const KvCache& c, int64_t seq) { return max(c.lens[seq], 0); }
__device__ __forceinline__ int64_t held_of(const KvCache& c, int64_t seq) { return min(len_of(c, seq), c.width * c.page); }

// One workgroup per (sequence, touched block, head, keys or values): it alone reads and writes that block's
// codes and scale.  A thread holds up to 8 pieces of 8 values.
template <int DIM>
__global__ void __launch_bounds__(256)
kv_append_kernel(KvCache c, const uint16_t* __restrict__ k, int64_t ldk, const uint16_t* __restrict__ v, int64_t ldv,
                 int64_t tokens, unsigned touched) {
  constexpr int kPieces = 128 * DIM / 8 / 256;   // of the largest page
  __shared__ float wave_max[4];
  const int page_log = __builtin_ctz(c.page);
  unsigned at = blockIdx.x;
  const bool values = at & 1;
  at >>= 1;
  const int head = at % c.heads;
  at /= c.heads;
  const int64_t seq = at / touched, held = held_of(c, seq), first = len_of(c, seq) - tokens;
  const int64_t block = (max(first, (int64_t)0) >> page_log) + at % touched, start = block << page_log;
  if (start >= held) return;
  const int64_t id = page_of(c, seq, block);
  if (id < 0) return;
  const uint16_t* src = (values ? v + seq * tokens * ldv : k + seq * tokens * ldk) + head * DIM;
  const int64_t ld = values ? ldv : ldk;
  const int64_t base = id * c.heads + head;
  int8_t* dst = (values ? c.v_codes : c.k_codes) + base * c.page * DIM;
  float* scale = (values ? c.v_scale : c.k_scale) + base;
  const int rows = (int)min((int64_t)c.page, held - start);         // rows of the block in use
  const int old_rows = (int)min(max(first - start, (int64_t)0), (int64_t)rows);   // from before

  u32x4 raw[kPieces];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int piece = i * 256 + threadIdx.x, row = piece / (DIM / 8);
    raw[i] = u32x4{0, 0, 0, 0};
    if (row >= old_rows && row < rows) {
      raw[i] = *reinterpret_cast<const u32x4*>(src + (start + row - first) * ld + piece % (DIM / 8) * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(raw[i][j])), fabsf(bf16hi(raw[i][j]))));
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
  if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = amax;
  const float s_old = old_rows ? *scale : 0.0f;
  __syncthreads();
  amax = fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3]));
  const float s = fmaxf(s_old, amax / 127.0f);      // IEEE division
  const QuotientScale qs = quotient_scale(s);
  const bool grew = s > s_old && old_rows;
  const float ratio = grew ? s_old / s : 1.0f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int piece = i * 256 + threadIdx.x, row = piece / (DIM / 8);
    if (row >= rows) continue;
    u32x2_t* out = reinterpret_cast<u32x2_t*>(dst + piece * 8);
    if (row >= old_rows) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16lo(raw[i][j]) * qs.pre;
        x[2 * j + 1] = bf16hi(raw[i][j]) * qs.pre;
      }
      *out = u32x2_t{int8_codes4(x[0], x[1], x[2], x[3], qs.s, qs.r), int8_codes4(x[4], x[5], x[6], x[7], qs.s, qs.r)};
    } else if (grew) {
      u32x2_t w = *out;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t word = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float code = (float)(int8_t)(w[j] >> (8 * e));
          word |= ((uint32_t)(int)rintf(code * ratio) & 0xffu) << (8 * e);
        }
        w[j] = word;
      }
      *out = w;
    }
  }
  if (threadIdx.x == 0) *scale = s;                  // every thread has read s_old (barrier above)
}

// k, v [seqs][length][heads][dim] bf16.  A workgroup takes 2048 / DIM tokens of a sequence and up to kReadHeads heads, a
// thread 8 values of each: a head's codes of those tokens are one piece of a page, and no index needs a division
// per thread (one thread per 8 values of the flat output took 9.7 us for 61 sequences of 299 tokens, 8 heads of 64).
constexpr int kReadHeads = 4;
template <int DIM>
__global__ void __launch_bounds__(256)
kv_read_kernel(KvCache c, int64_t length, int chunks, uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  constexpr int LANES = DIM / 8;
  const int d = threadIdx.x % LANES * 8, page_log = __builtin_ctz(c.page);
  const int64_t seq = blockIdx.x / chunks, pos = (int64_t)(blockIdx.x % chunks) * (256 / LANES) + threadIdx.x / LANES;
  const int head0 = blockIdx.y * kReadHeads;
  if (pos >= length) return;
  const int64_t id = pos < held_of(c, seq) ? page_of(c, seq, pos >> page_log) : -1;
  const int64_t base = max(id, (int64_t)0) * c.heads, row = (int64_t)(pos & (c.page - 1)) * DIM + d;
  u32x2_t w[kReadHeads][2];
  float s[kReadHeads][2];
#pragma unroll
  for (int i = 0; i < kReadHeads; ++i) {        // (past the last head: the last again, not stored)
    const int64_t at = base + min(head0 + i, c.heads - 1), code = at * c.page * DIM + row;
    w[i][0] = *reinterpret_cast<const u32x2_t*>(c.k_codes + code);
    w[i][1] = *reinterpret_cast<const u32x2_t*>(c.v_codes + code);
    s[i][0] = c.k_scale[at];
    s[i][1] = c.v_scale[at];
  }
#pragma unroll
  for (int i = 0; i < kReadHeads; ++i) {
    if (head0 + i >= c.heads) break;
    const int64_t to = ((seq * length + pos) * c.heads + head0 + i) * DIM + d;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      u32x4 out = {0, 0, 0, 0};
      if (id >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b = w[i][t][j / 2] >> (16 * (j % 2));
          out[j] = bf16x2_rne((float)(int8_t)b * s[i][t], (float)(int8_t)(b >> 8) * s[i][t]);
        }
      }
      *reinterpret_cast<u32x4*>((t ? v : k) + to) = out;
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const KvCache& c, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                            int64_t seqs, int64_t tokens, hipStream_t stream) {
  const int64_t touched = (tokens + c.page - 2) / c.page + 1, blocks = touched * c.heads * 2;     // of a sequence
  const auto kernel = c.dim == 64 ? kv_append_kernel<64> : kv_append_kernel<128>;
  return in_launches(seqs, blocks, 256, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(n * blocks)), dim3(256), 0, stream, c.from(b), k + b * tokens * ldk, ldk,
                       v + b * tokens * ldv, ldv, tokens, (unsigned)touched);
    return hipGetLastError();
  });
}

hipError_t launch_kv_read(const KvCache& c, int64_t seqs, int64_t length, uint16_t* k, uint16_t* v,
                          hipStream_t stream) {
  const int tokens = 2048 / c.dim;              // of a workgroup
  const int64_t chunks = (length + tokens - 1) / tokens, row = length * c.heads * c.dim;
  const unsigned head_groups = (unsigned)((c.heads + kReadHeads - 1) / kReadHeads);
  const auto kernel = c.dim == 64 ? kv_read_kernel<64> : kv_read_kernel<128>;
  return in_launches(seqs, chunks, 256, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(n * chunks), head_groups), dim3(256), 0, stream, c.from(b), length, (int)chunks,
                       k + b * row, v + b * row);
    return hipGetLastError();
  });
}

}  // namespace w8a8
