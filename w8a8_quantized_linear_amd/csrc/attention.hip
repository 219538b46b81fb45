// Attention of each sequence's newest tokens over its paged 8-bit cache.
//
// What it computes: for query i of the `tokens` new ones of a sequence of L tokens, over the keys
// j = 0 .. L - tokens + i that it sees, y = sum_j p_j v_j / sum_j p_j with p_j = exp(scale * q.k_j - max), where
// k_j and v_j are codes times the scale of their page and head; query heads q_heads / heads * h .. share
// cache head h.  A query that sees nothing gives zeros.
//
// Arithmetic.  Codes are whole numbers below 128 and exact in f16, so both products run on the f16 matrix
// cores with fp32 sums: a row of q is scaled by a power of two to below 2^8 (what falls under f16's range
// is below 2^-32 of the row's largest value); the keys' scale multiplies the fp32 score, and the values' scale rides in
// the exponent, p' = 2^(s + log2(scale) - max), so it costs nothing per element; p' is rounded to f16, 11 bits, and
// the sum of p' over a page is divided by the scale again.  The maximum is a row's own, over s + log2(scale) of what it
// sees: a key counts by what it adds to the output, however far the scales of pages lie apart, and what f16
// loses is below 2^-31 of the row's largest p * scale.  A page whose values have a scale below 2^-90 counts as one
// of that scale with codes of zero.  The running maximum moves only when it is passed by more than 2^8 (p' stays below
// 2^15), which spares most steps the rescaling of the outputs and the exchange between lanes.  Maximum, sum and
// output are fp32.
#include <algorithm>

#include "attention_math.h"

namespace w8a8 {
namespace {

using namespace kva;

constexpr int kTile = 32;                       // tokens of a wave's step: two runs of 16
static_assert(kPiece % (4 * kTile) == 0, "pieces are whole steps of four waves");

__device__ __forceinline__ float lane_value(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}

// One workgroup: 16 * NB query rows (tokens x the heads that share a cache head) against one piece of a
// sequence; its W waves take the steps of 32 tokens in turn and meet in LDS.  Bound by the cache's bytes where the
// sequences are long, by latency where they are short (length -> table -> codes -> scores -> outputs), so a wave has
// the next step's codes in flight while it computes, keeps the pages and scales of 64 blocks in a register each
// (lane i: block i) instead of LDS, and waits for no other wave before the end.  MFMA 16x16x32 f16:
//   S^T = K Q^T: a lane's 16 bytes of a key are two operands as they come from memory;
//   O^T += V^T P^T: P^T is S^T's layout as it stands; V^T takes byte b of a lane's eight values as output block b,
//   so one 8-byte piece per token serves all blocks and nothing is transposed through LDS.
// One token of 131,072 (32/8 heads of 128): 48 us and 4 for the pieces' joining (5.1 TB/s); 32 sequences of up to 2,270
// (40/8 heads) 23 us; 298 tokens (16 heads of 64) 5.7 us, the length of the chain.  Codes two or three steps ahead were 3 to 8% slower.
template <int DIM, int NB, int W>
__global__ void __launch_bounds__(64 * W)
kv_attention_kernel(KvCache c, const uint16_t* __restrict__ q, int64_t ldq, int tokens, int group, float scale,
                    int splits, int row_tiles, uint16_t* __restrict__ y, Partial part) {
  constexpr int DC = DIM / 64;                  // 16-byte pieces of a lane's key
  constexpr int DB = DIM / 16;                  // output blocks; bytes of a lane's value piece
  constexpr int OB = 4 * DB / W;                // outputs of a thread
  __shared__ float red_max[W][16], red_sum[W][16];
  __shared__ f32x4 red_out[W][DB][64];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4, r = lane & 15;
  int at = blockIdx.x;
  const int split = at % splits;
  at /= splits;
  const int tile = at % row_tiles;
  at /= row_tiles;
  const int head = at % c.heads, page_log = __builtin_ctz(c.page);
  const int64_t seq = at / c.heads;
  const int rows = tokens * group, row0 = tile * 16 * NB;
  const int len = max(c.lens[seq], 0), held = min(len, (int)c.width << page_log), piece = piece_of(held, splits);
  // a query at position p sees the keys up to p
  const int first_pos = len - tokens;
  const int last_row = min(row0 + 16 * NB, rows) - 1;
  const int begin = min(split * piece, held), end = min(min(begin + piece, held), first_pos + last_row / group + 1);
  const int all_seen = min(end, first_pos + row0 / group + 1);         // every row sees the keys before it

  // ---- queries: operand B of S^T = K Q^T, lane 16 h + r holds row r, dims 64 c + 16 h .. + 15 ----
  u32x4 qf[NB][DC][2];
  float qs[NB];                                 // scale of the scores of the lane's row, in powers of two
  int last_key[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int row = min(row0 + 16 * n + r, rows - 1);
    const uint16_t* src = q + (seq * tokens + row / group) * ldq + (head * group + row % group) * DIM + 16 * h;
    last_key[n] = first_pos + row / group;
#pragma unroll
    for (int cc = 0; cc < DC; ++cc)
#pragma unroll
      for (int u = 0; u < 2; ++u) qf[n][cc][u] = *reinterpret_cast<const u32x4*>(src + 64 * cc + 8 * u);
  }

  // ---- pages: lane i holds block base + i of the table ----
  const int32_t* table = c.table + seq * c.width;
  const int64_t page_bytes = (int64_t)c.heads * c.page * DIM;
  const int64_t head_bytes = (int64_t)head * c.page * DIM;
  const int last_block = max(end - 1, 0) >> page_log;
  // the blocks in hand: base .. base + 63, then the next 64 (of a short table all, so that loading them does not
  // wait for the length)
  int base = c.width <= 64 ? 0 : begin >> page_log;
  auto load_ids = [&](int b) { return table[min(b + lane, (int)c.width - 1)]; };
  int32_t ids = load_ids(base), next_ids = load_ids(base + 64);
  float k_scale, v_scale, v_log, v_inv;         // of the blocks in hand
  auto load_scales = [&]() {
    const bool real = ids >= 0 && ids < c.pages;
    const int64_t id = (int64_t)(real ? ids : 0) * c.heads + head;
    k_scale = c.k_scale[id];
    v_scale = c.v_scale[id];
    if (!(v_scale >= 0x1p-90f)) v_scale = 0.0f; // kLeastLog
    if (!real) v_scale = -1.0f;                 // not seen
  };
  auto take_logs = [&]() {                      // (apart from the loads, so as not to wait for them)
    v_log = v_scale > 0.0f ? __log2f(v_scale) : kLeastLog;
    v_inv = v_scale > 0.0f ? kSumBy / v_scale : kSumBy * 0x1p90f;
  };

  struct Codes {
    u32x4 k[2][DC];
    uint32_t v[8][DB / 4];
  };
  auto load_codes = [&](Codes& to, int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // (a run past the end reads the last block again, at rows that exist)
      const int t = t0 + 16 * u, block = max(min(t >> page_log, last_block) - base, 0);
      const int id = block < 64 ? __builtin_amdgcn_readlane(ids, block) : __builtin_amdgcn_readlane(next_ids, block - 64);
      const int64_t at = (int64_t)(id >= 0 && id < c.pages ? id : 0) * page_bytes + head_bytes + (int64_t)(t & (c.page - 1)) * DIM;
      const int8_t* kp = c.k_codes + at;
      const int8_t* vp = c.v_codes + at;
#pragma unroll
      for (int cc = 0; cc < DC; ++cc) to.k[u][cc] = *reinterpret_cast<const u32x4*>(kp + (r * DIM + 16 * h) + 64 * cc);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(vp + (4 * h * DIM + DB * r) + i * DIM);
        if constexpr (DB == 8) {
          const u32x2 two = *reinterpret_cast<const u32x2*>(p);
          to.v[4 * u + i][0] = two[0];
          to.v[4 * u + i][DB / 4 - 1] = two[1];
        } else {
          to.v[4 * u + i][0] = *p;
        }
      }
    }
  };

  f32x4 out[NB][DB];                            // O^T: lane 16 h + r, block b: row r, dims DB (4 h + i) + b
  float top[NB], sum[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    top[n] = -INFINITY;
    sum[n] = 0.0f;
#pragma unroll
    for (int b = 0; b < DB; ++b) out[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  auto step = [&](const Codes& x, int t0) __attribute__((always_inline)) {
    // ---- scores S^T: lane 16 h + r, run u: row r, tokens 4 h + i ----
    f32x4 s[NB][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int n = 0; n < NB; ++n) s[n][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int cc = 0; cc < DC; ++cc)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          u32x4 a;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t two[2];
            f16_word(x.k[u][cc][2 * half + j], two);
            a[2 * j] = two[0], a[2 * j + 1] = two[1];
          }
#pragma unroll
          for (int n = 0; n < NB; ++n)
            s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                            __builtin_bit_cast(f16x8, qf[n][cc][half]), s[n][u], 0, 0, 0);
        }
    }
    float rk[2], rv[2], rlog[2], rinv[2];       // the runs' scales, the same for the whole wave
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int block = min((t0 + 16 * u) >> page_log, last_block) - base;
      rk[u] = lane_value(k_scale, block);
      rv[u] = t0 + 16 * u < end ? lane_value(v_scale, block) : -1.0f;
      rlog[u] = lane_value(v_log, block);
      rinv[u] = lane_value(v_inv, block);
    }
    const bool whole = t0 + kTile <= all_seen && rv[0] >= 0.0f && rv[1] >= 0.0f;
    // ---- running softmax; P^T as the second product's operand: lane 16 h + r: row r, tokens 4 h + i of both runs ----
    u32x4 p[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      float factor[2], vlog[2], m = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        factor[u] = rk[u] * qs[n];
        vlog[u] = rlog[u];
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = t0 + 16 * u + 4 * h + i;
            const bool seen = key < end && key <= last_key[n] && rv[u] >= 0.0f;
            s[n][u][i] = seen ? s[n][u][i] * factor[u] : -INFINITY;
          }
          factor[u] = 1.0f;
          // (a row that sees none of the run: its values' scale, which may be infinite, must not count)
          if (t0 + 16 * u > last_key[n]) vlog[u] = kLeastLog;
        }
        m = fmaxf(m, __builtin_fmaf(fmaxf(fmaxf(s[n][u][0], s[n][u][1]), fmaxf(s[n][u][2], s[n][u][3])), factor[u], vlog[u]));
      }
      if (__any(m > top[n] + kLazy)) {
        const float next = fmaxf(max_quarters(m), top[n]), ref = next == -INFINITY ? 0.0f : next;
        const float scaled = __builtin_amdgcn_exp2f(top[n] - ref);
        sum[n] *= scaled;
#pragma unroll
        for (int b = 0; b < DB; ++b) out[n][b] *= scaled;
        top[n] = next;
      }
      const float ref = top[n] == -INFINITY ? 0.0f : top[n];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool some = rv[u] > 0.0f;         // (zeros: codes of zero, whatever they are)
        const float off = vlog[u] + (kProbExp - ref);
        float add = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][u][i], factor[u], off));
          const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[n][u][i + 1], factor[u], off));
          add += a + b;
          p[n][2 * u + i / 2] = some ? f16_pair(a, b) : 0u;
        }
        sum[n] = __builtin_fmaf(add, rinv[u], sum[n]);
      }
    }
    // ---- O^T += V^T P^T: block b's operand is byte b of the lane's eight values ----
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      u32x4 a;
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = f16_bytes(x.v[2 * j + 1][b / 4], x.v[2 * j][b / 4], b % 4);
#pragma unroll
      for (int n = 0; n < NB; ++n)
        out[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, p[n]),
                                                          out[n][b], 0, 0, 0);
    }
  };

  // (the wave's first step may lie past the end: its codes are loaded all the same, from the last block)
  Codes codes[2];
  int t0 = begin + wave * kTile;
  load_codes(codes[0], t0);
  load_scales();
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    uint32_t most = 0;
#pragma unroll
    for (int cc = 0; cc < DC; ++cc)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max(most, max((qf[n][cc][u][j] << 16) & 0x7fffffffu, qf[n][cc][u][j] & 0x7fff0000u));
    const int up = query_exp(__float_as_uint(max_quarters(__uint_as_float(most))));
    const float by = ldexpf(scale < 0.0f ? -1.0f : 1.0f, up);      // scores are scaled by what is not negative
    qs[n] = ldexpf(fabsf(scale) * 1.44269504088896341f, -up);
#pragma unroll
    for (int cc = 0; cc < DC; ++cc)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[n][cc][u][j] = f16_pair(__uint_as_float(qf[n][cc][u][j] << 16) * by, __uint_as_float(qf[n][cc][u][j] & 0xffff0000u) * by);
  }
  take_logs();
  while (t0 < end) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      load_codes(codes[d ^ 1], t0 + W * kTile);
      step(codes[d], t0);
      t0 += W * kTile;
      if (t0 >= end) break;
      if ((t0 >> page_log) - base >= 64) {      // the next 64 blocks
        base += 64;
        ids = next_ids;
        next_ids = load_ids(base + 64);
        load_scales();
        take_logs();
      }
    }
  }

  // ---- the waves' parts meet ----
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const float total = sum_quarters(sum[n]);
    if (n) __syncthreads();
    if (h == 0) {
      red_max[wave][r] = top[n];
      red_sum[wave][r] = total;
    }
    __syncthreads();
    float m = red_max[0][r];
#pragma unroll
    for (int w = 1; w < W; ++w) m = fmaxf(m, red_max[w][r]);
    const float ref = m == -INFINITY ? 0.0f : m;
    const float by = __builtin_amdgcn_exp2f(top[n] - ref);
#pragma unroll
    for (int b = 0; b < DB; ++b) red_out[wave][b][lane] = out[n][b] * by;
    __syncthreads();
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) l += red_sum[w][r] * __builtin_amdgcn_exp2f(red_max[w][r] - ref);
    // thread: lane's row r; wave w finishes i = w % 4: OB of the dims DB (4 h + i) + 0 .. DB - 1
    const int ob = OB * (wave / 4);
    float o[OB];
#pragma unroll
    for (int b = 0; b < OB; ++b) {
      o[b] = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) o[b] += red_out[w][ob + b][lane][wave % 4];
    }
    const int row = row0 + 16 * n + r;
    if (row >= rows) continue;
    const int d0 = DB * (4 * h + wave % 4) + ob;
    if (splits == 1) {
      const float inv = l > 0.0f ? kSumBy / l : 0.0f;
      uint16_t* dst = y + ((seq * tokens + row / group) * c.heads * group + head * group + row % group) * DIM + d0;
#pragma unroll
      for (int b = 0; b < OB; b += 2) *reinterpret_cast<uint32_t*>(dst + b) = bf16x2_rne(o[b] * inv, o[b + 1] * inv);
    } else {
      const int64_t index = ((seq * c.heads + head) * rows + row) * splits + split;
#pragma unroll
      for (int b = 0; b < OB; b += 2) *reinterpret_cast<float2*>(part.out + index * DIM + d0 + b) = float2{o[b], o[b + 1]};
      if (h == 0 && wave == 0) {
        part.stat[2 * index] = m;
        part.stat[2 * index + 1] = l;
      }
    }
  }
}

// The pieces of a row meet, four dims a thread.  Many pieces of few rows: a workgroup a row (WIDE), the pieces dealt to
// its threads and summed in LDS; latency bound, two dependent loads and the sum.  Few pieces of many rows: a thread
// adds all pieces of its dims, 256 / (DIM / 4) rows a workgroup; bound by the partial results' bytes.
template <int DIM, bool WIDE>
__global__ void __launch_bounds__(256)
kv_combine_kernel(int64_t all, int rows, int heads, int group, int splits, uint16_t* __restrict__ y, Partial part) {
  constexpr int COLS = DIM / 4, PARTS = 256 / COLS;
  __shared__ f32x4 red_out[PARTS][COLS];
  __shared__ float red_sum[PARTS];
  const int col = threadIdx.x % COLS, mine = threadIdx.x / COLS;
  const int64_t index = WIDE ? blockIdx.x : (int64_t)blockIdx.x * PARTS + mine;
  if (index >= all) return;
  const float* stat = part.stat + 2 * index * splits;
  const float* out = part.out + index * splits * DIM + 4 * col;
  float m = -INFINITY;
  if constexpr (WIDE) {
    for (int s = threadIdx.x & 63; s < splits; s += 64) m = fmaxf(m, stat[2 * s]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  } else {
    for (int s = 0; s < splits; ++s) m = fmaxf(m, stat[2 * s]);
  }
  const float ref = m == -INFINITY ? 0.0f : m;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.0f;
#pragma unroll 4
  for (int s = WIDE ? mine : 0; s < splits; s += WIDE ? PARTS : 1) {    // (a piece without a key: outputs and sum of zero)
    const float by = __builtin_amdgcn_exp2f(stat[2 * s] - ref);
    l = __builtin_fmaf(by, stat[2 * s + 1], l);
    o += *reinterpret_cast<const f32x4*>(out + (int64_t)s * DIM) * by;
  }
  if constexpr (WIDE) {
    red_out[mine][col] = o;
    if (col == 0) red_sum[mine] = l;
    __syncthreads();
    if (mine) return;
#pragma unroll
    for (int g = 1; g < PARTS; ++g) {
      o += red_out[g][col];
      l += red_sum[g];
    }
  }
  const float inv = l > 0.0f ? kSumBy / l : 0.0f;
  const int64_t row = index % rows, seq = index / rows / heads, head = index / rows % heads;
  uint16_t* dst = y + ((seq * (rows / group) + row / group) * heads * group + head * group + row % group) * DIM + 4 * col;
  *reinterpret_cast<u32x2*>(dst) = u32x2{bf16x2_rne(o[0] * inv, o[1] * inv), bf16x2_rne(o[2] * inv, o[3] * inv)};
}

// Blocks of 16 rows of a workgroup: two read the codes once for both, one leaves more workgroups and shorter steps.
// Two where a CU has more than 256 tokens of a cache head to read (64 rows: 8 x 8,000 tokens of 8 heads 32 against 40 us,
// 30,000 of 4 heads 22.7 and 24.7 us; but 500 of 8 heads 12.7 and 9.2 us, 8 x 1,500 of 4 heads 14.8 and 12.4 us; four blocks
// were never faster than two).
int blocks_of(int64_t rows, int64_t head_tokens) { return rows > 16 && head_tokens > 256 * 256 ? 2 : 1; }
// Eight waves on one piece where its workgroups are at most half the CUs: up to 1,536 tokens (1,024 for 128 dims) they are
// done before four waves on several pieces and the pieces' joining (64 dims: 16 sequences of 1,000, 32/8 heads, 11.4 and 8.8
// us, 7 x 4 tokens of 1,502 12.0 and 10.9; 128 dims: 1,000 tokens of 32/8 heads 11.7 and 11.5, 1,502 11.8 and 14.4); with more
// workgroups four waves are better (500 tokens of 500, 8/8 heads: 9.5 against 10.2 us).
bool eight_waves(int64_t rows, int64_t seq_heads, int64_t length, int dim) {
  return length > 128 && length <= (dim == 64 ? 1536 : 1024) && blocks_of(rows, seq_heads * length) == 1 &&
         seq_heads * ((rows + 15) / 16) <= 128;
}
// The prompt form, from 65 rows on and where every CU has more than 16 rows against 1,536 tokens that they see (at 128
// dims): below, its few long workgroups take longer (500 tokens of 8/8 heads 17.7 against 9.4 us here, 40 of 500 of 32/8
// 14.0 and 9.3, 64 of 2,000 22.3 and 18.4, 1,502 of 2/2 22.4 and 19.4, 636 of 16/2 of 64 18.7 and 10.5; but 20 tokens of
// 4 x 4,000 26.6 against 35 us, 400 of 633 of 40/8 25.6 and 26.1).
bool prompt_form(int64_t rows, int64_t tokens, int64_t head_tokens, int64_t length, int dim) {
  return rows > 64 && (double)rows * (double)head_tokens * seen_of(tokens, length) * dim > 256.0 * 16 * 1536 * 128;
}

template <int DIM, int NB, int W>
hipError_t launch(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group, float scale,
                  int64_t splits, uint16_t* y, Partial part, hipStream_t stream) {
  const int64_t rows = tokens * group, tiles = (rows + 16 * NB - 1) / (16 * NB);
  const int64_t blocks = c.heads * tiles * splits;              // of a sequence
  return in_launches(seqs, blocks, 64 * W, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL((kv_attention_kernel<DIM, NB, W>), dim3((unsigned)(n * blocks)), dim3(64 * W), 0, stream, c.from(b),
                       q + b * tokens * ldq, ldq, (int)tokens, group, scale, (int)splits, (int)tiles, y + b * c.heads * rows * DIM,
                       part.from(b * c.heads * rows * splits, DIM));
    return hipGetLastError();
  });
}

template <int DIM>
hipError_t launch_all(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group, float scale,
                      int64_t splits, uint16_t* y, Partial part, hipStream_t stream) {
  const int64_t rows = tokens * group, all = seqs * c.heads * rows, head_tokens = seqs * c.heads * c.width * c.page;
  hipError_t e;
  if (prompt_form(rows, tokens, head_tokens, c.width * c.page, DIM)) e = launch_prompt<DIM>(c, q, ldq, seqs, tokens, group, scale, prompt_cut(seqs, rows, tokens, c.heads, DIM, c.width * c.page), y, part, stream);
  else if (eight_waves(rows, seqs * c.heads, c.width * c.page, DIM)) e = launch<DIM, 1, 8>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  else if (blocks_of(rows, head_tokens) == 1) e = launch<DIM, 1, 4>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  else e = launch<DIM, 2, 4>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  if (e != hipSuccess || splits == 1) return e;
  // a workgroup a row while those fit the GPU's 256 CUs a few times over
  const bool wide = all <= 2048;
  const int64_t blocks = wide ? all : (all + 1024 / DIM - 1) / (1024 / DIM);
  const auto kernel = wide ? kv_combine_kernel<DIM, true> : kv_combine_kernel<DIM, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, stream, all, (int)rows, c.heads, group, (int)splits, y, part);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_splits(int64_t seqs, int64_t tokens, int q_heads, int heads, int dim, int page, int64_t width) {
  const int64_t rows = tokens * (q_heads / heads), most_tokens = width * page, head_tokens = seqs * heads * most_tokens;
  if (prompt_form(rows, tokens, head_tokens, most_tokens, dim)) return prompt_cut(seqs, rows, tokens, heads, dim, most_tokens).splits;
  // as many workgroups as make one round of the 256 CUs (32 sequences up to 2,270 tokens: 25.3 us, with twice as many
  // 27.2 us; one of 131,072: 52.9 and 55.5 us; 5 of 4,043, 24/8 heads: 15.0 us in 6 pieces, 17.4 in 7, which are 280), two
  // of them a CU for 64 dims, whose steps have half the bytes in flight (12 of 8,000, 32/4 heads: 16.9 and 14.3 us); but
  // one piece alone up to 512 tokens of a full table (a step of 128 takes less than the combination's 3 us) and no piece
  // below 256
  const int64_t tile = 16 * blocks_of(rows, head_tokens), one = seqs * heads * ((rows + tile - 1) / tile);
  if (most_tokens <= 512 || eight_waves(rows, seqs * heads, most_tokens, dim)) return 1;
  return std::max<int64_t>(1, std::min<int64_t>((dim == 64 ? 512 : 256) / one, most_tokens / 256));
}

hipError_t launch_kv_attention(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens,
                               int q_heads, float scale, uint16_t* y, void* workspace, hipStream_t stream) {
  const int64_t splits = kv_attention_splits(seqs, tokens, q_heads, c.heads, c.dim, c.page, c.width);
  Partial part{nullptr, nullptr};
  if (splits > 1) {
    part.out = static_cast<float*>(workspace);
    part.stat = part.out + seqs * tokens * q_heads * splits * c.dim;
  }
  const int group = q_heads / c.heads;
  return c.dim == 64 ? launch_all<64>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream)
                     : launch_all<128>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
}

}  // namespace w8a8
