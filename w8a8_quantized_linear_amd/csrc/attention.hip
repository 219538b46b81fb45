// Attention of each sequence's newest tokens over its paged 8-bit cache.
//
// What it computes: for query i of the `tokens` new ones of a sequence of L tokens, over the keys
// j = 0 .. L - tokens + i that it sees, y = sum_j p_j v_j / sum_j p_j with p_j = exp(scale * q.k_j - max), where
// k_j and v_j are codes times the scale of their page and head; query heads q_heads / heads * h .. share
// cache head h.  A query that sees nothing gives zeros.
//
// Arithmetic.  Codes are whole numbers below 128 and exact in f16, so both products run on the f16 matrix
// cores with fp32 sums: a row of q is scaled by a power of two to below 2^8 (what falls under f16's range
// is below 2^-32 of the row's largest value), the keys' scale multiplies the fp32 score, and the probabilities
// (below 1, times the values' scale relative to a power of two, times 2^14) are rounded to f16, 11 bits.
// Maximum, sum and output are fp32.
#include <algorithm>

#include "attention_math.h"

namespace w8a8 {
namespace {

using namespace kva;

constexpr int kWaves = 4;
constexpr int kTile = 32;                       // tokens of a wave's step: two MFMA tiles of 16
constexpr int kSegment = 2048;                  // tokens whose page entries are in LDS at once
constexpr int kEntries = kSegment / 16;         // pages of a segment at the smallest page
constexpr int kStep = kWaves * kTile;           // pieces of a sequence are whole steps of a workgroup
static_assert(kPiece % kStep == 0, "pieces are whole steps");
constexpr int kProbExp = 14;                    // probabilities are rounded below 2^14 (f16 ends at 2^16)

// The largest of the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float max_quarters(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum_quarters(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

struct Entry {
  int32_t id;        // page, -1: none
  float k, v;        // its scales
};

// One workgroup: 16 * NB query rows (tokens x the heads that share a cache head) against one piece of a
// sequence; its waves take every fourth step of 32 tokens and meet in LDS.
template <int DIM, int NB>
__global__ void __launch_bounds__(256)
kv_attention_kernel(KvCache c, const uint16_t* __restrict__ q, int64_t ldq, int tokens, int group, float scale,
                    int splits, int row_tiles, uint16_t* __restrict__ y, Partial part) {
  constexpr int DC = DIM / 64;                  // 16-byte pieces of a lane's key
  constexpr int DB = DIM / 16;                  // output blocks; bytes of a lane's value piece
  __shared__ Entry entries[kEntries];
  __shared__ float red_max[kWaves][16], red_sum[kWaves][16];
  __shared__ f32x4 red_out[kWaves][DB][64];

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

  // ---- queries: operand B of S^T = K Q^T, lane 16 h + r holds row r, dims 64 c + 16 h .. + 15 ----
  u32x4 qf[NB][DC][2];
  float qs[NB];                                 // scale of the scores of the lane's row, in powers of two
  int last_key[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const int row = min(row0 + 16 * n + r, rows - 1);
    const uint16_t* src = q + (seq * tokens + row / group) * ldq + (head * group + row % group) * DIM + 16 * h;
    last_key[n] = first_pos + row / group;
    u32x4 raw[DC][2];
    uint32_t top = 0;
#pragma unroll
    for (int cc = 0; cc < DC; ++cc)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        raw[cc][u] = *reinterpret_cast<const u32x4*>(src + 64 * cc + 8 * u);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max((raw[cc][u][j] << 16) & 0x7fffffffu, raw[cc][u][j] & 0x7fff0000u));
      }
    top = __float_as_uint(max_quarters(__uint_as_float(top)));
    const int up = query_exp(top);
    const float by = ldexpf(1.0f, up);
    qs[n] = ldexpf(scale * 1.44269504088896341f, -up);
#pragma unroll
    for (int cc = 0; cc < DC; ++cc)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[n][cc][u][j] = f16_pair(__uint_as_float(raw[cc][u][j] << 16) * by, __uint_as_float(raw[cc][u][j] & 0xffff0000u) * by);
  }

  f32x4 out[NB][DB];                            // O^T: lane 16 h + r, block b: row r, dims DB (4 h + i) + b
  float top[NB], sum[NB];
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    top[n] = -INFINITY;
    sum[n] = 0.0f;
#pragma unroll
    for (int b = 0; b < DB; ++b) out[n][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int v_exp = -1000;                            // the values' scales are taken relative to 2^v_exp

  const int64_t page_bytes = (int64_t)c.heads * c.page * DIM;
  for (int seg = begin; seg < end; seg += kSegment) {
    // ---- the segment's pages and scales ----
    const int seg_end = min(seg + kSegment, end);
    const int count = ((seg_end - 1) >> page_log) - (seg >> page_log) + 1;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += 256) {
      const int32_t id = c.table[seq * c.width + (seg >> page_log) + i];
      const bool real = id >= 0 && id < c.pages;
      const int64_t base = (int64_t)(real ? id : 0) * c.heads + head;
      entries[i] = Entry{real ? id : -1, real ? c.k_scale[base] : 0.0f, real ? c.v_scale[base] : 0.0f};
    }
    __syncthreads();
    float v_top = 0.0f;
    for (int i = lane; i < count; i += 64) v_top = fmaxf(v_top, entries[i].v);
    v_top = fmaxf(v_top, __shfl_xor(v_top, 1));
    v_top = fmaxf(v_top, __shfl_xor(v_top, 2));
    v_top = fmaxf(v_top, __shfl_xor(v_top, 4));
    v_top = fmaxf(v_top, __shfl_xor(v_top, 8));
    v_top = max_quarters(v_top);
    const int seg_exp = scale_exp(v_top);
    if (seg_exp > v_exp) {
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int b = 0; b < DB; ++b) out[n][b] *= ldexpf(1.0f, max(v_exp - seg_exp, -200));
      v_exp = seg_exp;
    }
    const float v_by = ldexpf(1.0f, kProbExp - v_exp);

    for (int t0 = seg + wave * kTile; t0 < seg_end; t0 += kStep) {
      Entry e[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) e[u] = entries[min(((t0 + 16 * u) >> page_log) - (seg >> page_log), count - 1)];
      u32x4 kraw[2][DC];
      uint32_t vraw[8][DB / 4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int64_t base = max(e[u].id, 0) * page_bytes + ((int64_t)head * c.page + ((t0 + 16 * u) & (c.page - 1))) * DIM;
#pragma unroll
        for (int cc = 0; cc < DC; ++cc)
          kraw[u][cc] = *reinterpret_cast<const u32x4*>(c.k_codes + base + r * DIM + 64 * cc + 16 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < DB / 4; ++w)
            vraw[4 * u + i][w] = reinterpret_cast<const uint32_t*>(c.v_codes + base + (4 * h + i) * DIM + DB * r)[w] ^ 0x80808080u;
      }
      // ---- scores S^T: lane 16 h + r, tile u: row r, tokens 4 h + i ----
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
              f16_word(kraw[u][cc][2 * half + j], two);
              a[2 * j] = two[0], a[2 * j + 1] = two[1];
            }
#pragma unroll
            for (int n = 0; n < NB; ++n)
              s[n][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                              __builtin_bit_cast(f16x8, qf[n][cc][half]), s[n][u], 0, 0, 0);
          }
      }
      // ---- running softmax; P^T as the second product's operand: lane 16 h + r: row r, tokens 4 h + i of both tiles ----
      u32x4 p[NB];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = t0 + 16 * u + 4 * h + i;
            const bool seen = key < end && key <= last_key[n] && e[u].id >= 0;
            s[n][u][i] = seen ? s[n][u][i] * (e[u].k * qs[n]) : -INFINITY;
            m = fmaxf(m, s[n][u][i]);
          }
        m = fmaxf(max_quarters(m), top[n]);
        const float ref = m == -INFINITY ? 0.0f : m;
        const float shrink = __builtin_amdgcn_exp2f(top[n] - ref);
        top[n] = m;
        float add = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float by = e[u].v * v_by;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float a = __builtin_amdgcn_exp2f(s[n][u][i] - ref), b = __builtin_amdgcn_exp2f(s[n][u][i + 1] - ref);
            add += a + b;
            p[n][2 * u + i / 2] = f16_pair(a * by, b * by);
          }
        }
        sum[n] = __builtin_fmaf(sum[n], shrink, add);
#pragma unroll
        for (int b = 0; b < DB; ++b) out[n][b] *= shrink;
      }
      // ---- O^T += V^T P^T: block b's operand is byte b of the lane's eight values ----
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        u32x4 a;
        const uint32_t pick = 0x0c000c00u | (4 + b % 4) << 16 | (b % 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = f16_codes(__builtin_amdgcn_perm(vraw[2 * j + 1][b / 4], vraw[2 * j][b / 4], pick));
#pragma unroll
        for (int n = 0; n < NB; ++n)
          out[n][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, p[n]),
                                                            out[n][b], 0, 0, 0);
      }
    }
  }

  // ---- the waves' parts meet ----
  const float back = v_exp < -500 ? 0.0f : ldexpf(1.0f, v_exp - kProbExp);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    const float total = sum_quarters(sum[n]);
    __syncthreads();
    if (h == 0) {
      red_max[wave][r] = top[n];
      red_sum[wave][r] = total;
    }
    __syncthreads();
    float m = red_max[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, red_max[w][r]);
    const float ref = m == -INFINITY ? 0.0f : m;
    const float by = __builtin_amdgcn_exp2f(top[n] - ref) * back;
#pragma unroll
    for (int b = 0; b < DB; ++b) red_out[wave][b][lane] = out[n][b] * by;
    __syncthreads();
    float l = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) l += red_sum[w][r] * __builtin_amdgcn_exp2f(red_max[w][r] - ref);
    // thread: lane's row r; wave w finishes i = w: dims DB (4 h + w) + 0 .. DB - 1
    float o[DB];
#pragma unroll
    for (int b = 0; b < DB; ++b) {
      o[b] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) o[b] += red_out[w][b][lane][wave];
    }
    const int row = row0 + 16 * n + r;
    if (row >= rows) continue;
    const int d0 = DB * (4 * h + wave);
    if (splits == 1) {
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      uint16_t* dst = y + ((seq * tokens + row / group) * c.heads * group + head * group + row % group) * DIM + d0;
#pragma unroll
      for (int b = 0; b < DB; b += 4)
        *reinterpret_cast<u32x2*>(dst + b) = u32x2{bf16x2_rne(o[b] * inv, o[b + 1] * inv), bf16x2_rne(o[b + 2] * inv, o[b + 3] * inv)};
    } else {
      const int64_t index = ((seq * c.heads + head) * rows + row) * splits + split;
      if (m != -INFINITY) {
#pragma unroll
        for (int b = 0; b < DB; b += 4) *reinterpret_cast<f32x4*>(part.out + index * DIM + d0 + b) = f32x4{o[b], o[b + 1], o[b + 2], o[b + 3]};
      }
      if (h == 0 && wave == 0) {
        part.stat[2 * index] = m;
        part.stat[2 * index + 1] = l;
      }
    }
  }
}

// The pieces of a row meet: one workgroup per row, four dims a thread, the pieces dealt to the DIM / 4 lanes'
// groups.  Latency bound (two dependent loads and a sum in LDS): for 128 pieces of 32 rows 3 us, where one wave
// per row that walked the pieces took 70 us.
template <int DIM>
__global__ void __launch_bounds__(256)
kv_combine_kernel(int rows, int heads, int group, int splits, uint16_t* __restrict__ y, Partial part) {
  constexpr int COLS = DIM / 4, PARTS = 256 / COLS;
  __shared__ f32x4 red_out[PARTS][COLS];
  __shared__ float red_sum[PARTS];
  const int64_t index = blockIdx.x;
  const int col = threadIdx.x % COLS, mine = threadIdx.x / COLS;
  const float* stat = part.stat + 2 * index * splits;
  float m = -INFINITY;
  for (int s = threadIdx.x & 63; s < splits; s += 64) m = fmaxf(m, stat[2 * s]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float ref = m == -INFINITY ? 0.0f : m;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  float l = 0.0f;
  for (int s = mine; s < splits; s += PARTS) {
    const float ms = stat[2 * s];
    if (ms == -INFINITY) continue;             // a piece without a key has written no outputs
    const float by = __builtin_amdgcn_exp2f(ms - ref);
    l = __builtin_fmaf(by, stat[2 * s + 1], l);
    o += *reinterpret_cast<const f32x4*>(part.out + (index * splits + s) * DIM + 4 * col) * by;
  }
  red_out[mine][col] = o;
  if (col == 0) red_sum[mine] = l;
  __syncthreads();
  if (mine) return;
#pragma unroll
  for (int g = 1; g < PARTS; ++g) {
    o += red_out[g][col];
    l += red_sum[g];
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const int64_t row = index % rows, seq = index / rows / heads, head = index / rows % heads;
  uint16_t* dst = y + ((seq * (rows / group) + row / group) * heads * group + head * group + row % group) * DIM + 4 * col;
  *reinterpret_cast<u32x2*>(dst) = u32x2{bf16x2_rne(o[0] * inv, o[1] * inv), bf16x2_rne(o[2] * inv, o[3] * inv)};
}

// Blocks of 16 rows of a workgroup; rows past 64 take the prompt form.
int blocks_of(int64_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }
bool prompt_rows(int64_t rows) { return rows > 64; }

template <int DIM, int NB>
hipError_t launch(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group, float scale,
                  int64_t splits, uint16_t* y, Partial part, hipStream_t stream) {
  const int64_t rows = tokens * group, tiles = (rows + 16 * NB - 1) / (16 * NB);
  const int64_t blocks = seqs * c.heads * tiles * splits;
  if (blocks > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((kv_attention_kernel<DIM, NB>), dim3((unsigned)blocks), dim3(256), 0, stream, c, q, ldq, (int)tokens, group,
                     scale, (int)splits, (int)tiles, y, part);
  return hipGetLastError();
}

template <int DIM>
hipError_t launch_all(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group, float scale,
                      int64_t splits, uint16_t* y, Partial part, hipStream_t stream) {
  const int64_t rows = tokens * group, all = seqs * c.heads * rows;
  hipError_t e;
  if (prompt_rows(rows)) e = launch_prompt<DIM>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  else if (blocks_of(rows) == 1) e = launch<DIM, 1>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  else if (blocks_of(rows) == 2) e = launch<DIM, 2>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  else e = launch<DIM, 4>(c, q, ldq, seqs, tokens, group, scale, splits, y, part, stream);
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL((kv_combine_kernel<DIM>), dim3((unsigned)all), dim3(256), 0, stream, (int)rows, c.heads, group, (int)splits,
                     y, part);
  return hipGetLastError();
}

}  // namespace

int64_t kv_attention_splits(int64_t seqs, int64_t tokens, int q_heads, int heads, int page, int64_t width) {
  const int64_t rows = tokens * (q_heads / heads);
  const int64_t most = (width * page + kPiece - 1) / kPiece;
  if (prompt_rows(rows)) {
    // one workgroup fits a CU: the cut that leaves the fewest rounds of 256, a piece more costing a twentieth
    // (its partial results pass through memory)
    const int64_t one = seqs * heads * ((rows + kPromptRows - 1) / kPromptRows);
    int64_t best = 1;
    double least = 0.0;
    for (int64_t s = 1; s <= std::min<int64_t>(8, most); ++s) {
      const double cost = (double)((one * s + 255) / 256) / (double)s * (1.0 + 0.05 * (double)(s - 1));
      if (s == 1 || cost < least) best = s, least = cost;
    }
    return best;
  }
  // workgroups enough for four on each of the 256 CUs, but no piece of a full table below one step
  const int64_t tile = 16 * blocks_of(rows), one = seqs * heads * ((rows + tile - 1) / tile);
  return std::max<int64_t>(1, std::min<int64_t>((1024 + one - 1) / one, most));
}

hipError_t launch_kv_attention(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens,
                               int q_heads, float scale, uint16_t* y, void* workspace, hipStream_t stream) {
  const int64_t splits = kv_attention_splits(seqs, tokens, q_heads, c.heads, c.page, c.width);
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
