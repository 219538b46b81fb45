// Attention over the paged 8-bit cache for prompts and long pieces of prompts: many query rows, much work.
//
// The mathematics is that of attention.hip.  Here the arithmetic bounds the time, not the cache's bytes, so a
// workgroup turns each tile of 64 tokens of codes into f16 once, in LDS, for all its query rows (32 a wave): keys
// [token][dim], values transposed [dim][token].  MFMA 32x32x16 f16:
//   S^T = K Q^T: lane 32 h + r holds row r, tokens 8 (i / 4) + 4 h + i % 4 of a 32-token block in register i, which is the
//   second operand of O^T += V^T P^T as it stands, if the tokens of a 16-token step are taken in the order
//   4 h + j, 8 + 4 h + j (j < 4) for each half h: the order in which the values are written to LDS.
// Per wave and tile (dim 128) the matrix core needs 1,024 cycles, the vector unit about 900 and the exponentials 530.
// The units overlap only in part (two waves of a SIMD, one with products and one with multiply-adds, together take
// 0.71 of the sum of their times; products and exponentials overlap fully, measured), so ~1,500 is what a tile
// could take; it takes about 2,600: two waves a SIMD leave waits for LDS, for the products and at the barrier.  Four
// prompts of 1,502 tokens (40/8 heads of 128) take 140 us (660 TFLOP/s), 500 tokens behind 12,016 (32/8) 120 us (800);
// at 64 dims, with half the products for the same softmax, 98 us (471) and 90 us (535).
#include <algorithm>

#include "attention_math.h"

namespace w8a8 {
namespace kva {
namespace {

constexpr int kTile = 64;                       // tokens
constexpr int kSubs = kTile / 16;               // 16-token runs: no page boundary falls inside one

struct Run {
  float k;           // the keys' scale
  float v_log;       // log2 of the values' scale (zeros: kLeastLog)
  float v_inv;       // kSumBy / the scale
  int real;          // 0: the table names no page
};

// WAVES = 8: 256 rows, waves 0 .. 3 bring the values of a run of 16 tokens each and waves 4 .. 7 the keys.  WAVES = 4: 128
// rows, two workgroups a CU, each wave brings the keys and values of a run: twice the conversions for every row,
// but less to wait for where there are few tiles.
template <int DIM, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 2)
kv_prompt_kernel(KvCache c, const uint16_t* __restrict__ q, int64_t ldq, int tokens, int group, float scale, int splits,
                 int row_tiles, int total, uint16_t* __restrict__ y, Partial part) {
  constexpr int KS = DIM / 16;                  // MFMA steps of a key
  constexpr int DB = DIM / 32;                  // output blocks
  constexpr int KCH = DIM / 8;                  // 16-byte chunks of an f16 key row
  constexpr int KP = kTile * DIM / 16 / 256;    // 16-byte pieces of codes per lane that brings keys
  constexpr int ROWS = 32 * WAVES;
  __shared__ __attribute__((aligned(16))) u32x4 k_lds[2][kTile * KCH];
  __shared__ __attribute__((aligned(16))) u32x4 v_lds[2][DIM * (kTile / 8)];
  __shared__ Run runs[2][kSubs];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, r = lane & 31;
  // consecutive items to one XCD (workgroups go round the 8 XCDs), so that those of one sequence and head share an L2
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8;
  int at = xcd * (total / 8) + min(xcd, total % 8) + slot;
  const int split = at % splits;
  at /= splits;
  const int tile = row_tiles - 1 - at % row_tiles;          // the longest first
  at /= row_tiles;
  const int head = at % c.heads, page_log = __builtin_ctz(c.page);
  const int64_t seq = at / c.heads;
  const int rows = tokens * group, row0 = tile * ROWS + 32 * wave;
  const int len = max(c.lens[seq], 0), held = min(len, (int)c.width << page_log), piece = piece_of(held, splits);
  const int first_pos = len - tokens;
  const int tile_last = min((tile + 1) * ROWS, rows) - 1;
  const int begin = min(split * piece, held), end = min(min(begin + piece, held), first_pos + tile_last / group + 1);
  const int row = min(row0 + r, rows - 1), last_key = first_pos + row / group;
  // this wave's keys: none if it has no rows; every row sees those before `all_seen`
  const int wave_end = row0 < rows ? min(end, first_pos + min(row0 + 31, rows - 1) / group + 1) : 0;
  const int all_seen = min(end, first_pos + row0 / group + 1);

  // ---- queries ----
  u32x4 qf[KS];
  float qs;
  {
    const uint16_t* src = q + (seq * tokens + row / group) * ldq + (head * group + row % group) * DIM + 8 * h;
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      qf[s] = *reinterpret_cast<const u32x4*>(src + 16 * s);
#pragma unroll
      for (int j = 0; j < 4; ++j) top = max(top, max((qf[s][j] << 16) & 0x7fffffffu, qf[s][j] & 0x7fff0000u));
    }
    top = __float_as_uint(max_halves(__uint_as_float(top)));
    const int up = query_exp(top);
    const float by = ldexpf(scale < 0.0f ? -1.0f : 1.0f, up);      // scores are scaled by what is not negative
    qs = ldexpf(fabsf(scale) * 1.44269504088896341f, -up);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        qf[s][j] = f16_pair(__uint_as_float(qf[s][j] << 16) * by, __uint_as_float(qf[s][j] & 0xffff0000u) * by);
  }

  // ---- staging ----
  const bool keys = WAVES == 4 || wave >= 4, values = wave < 4;         // what this wave brings
  const int stage = wave & 3;
  const int v_quad = lane % (DIM / 4), v_half = lane / (DIM / 4);       // (dim 64: lanes 32 .. 63 have no values)
  const int64_t head_base = (int64_t)head * c.page * DIM;
  const int64_t page_bytes = (int64_t)c.heads * c.page * DIM;
  const int32_t* table = c.table + seq * c.width;
  // An instruction brings 64 / KL keys, KL lanes of 16 codes each.  The run and the first token in it of piece i:
  // a wave's own run where it brings values too or a piece is a run, else (8 waves, dim 128: 8 keys) waves 4, 5 share
  // runs 0 and 2, waves 6, 7 runs 1 and 3.
  constexpr int KL = DIM / 16;
  constexpr bool SHARED = WAVES == 8 && DIM == 128;
  const int k_row = lane / KL, k_piece = lane % KL;
  auto run_of = [&](int i) { return SHARED && keys ? stage / 2 + 2 * i : stage; };
  auto token_of = [&](int i) { return (SHARED ? 8 * (stage & 1) : (64 / KL) * i) + k_row; };
  const int v_lane = (4 * v_half) * DIM + 4 * v_quad;
  int ids[KP];                                  // pages of the runs of the tile to be loaded next
  u32x4 raw_k[2][KP], raw_v[2][2];              // codes of the next two tiles
  float run_k[2][KP], run_v[2];
  auto load_ids = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < KP; ++i) ids[i] = table[min((t0 + 16 * run_of(i)) >> page_log, (int)c.width - 1)];
  };
  auto load_codes = [&](int d, int t0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < KP; ++i) {
      const int t = t0 + 16 * run_of(i), named = __builtin_amdgcn_readfirstlane(ids[i]);
      const bool real = named >= 0 && named < c.pages && t < end;
      const int64_t id = real ? named : 0;
      const int64_t base = id * page_bytes + head_base + (int64_t)(t & (c.page - 1)) * DIM;
      if (keys) {
        raw_k[d][i] = *reinterpret_cast<const u32x4*>(c.k_codes + base + token_of(i) * DIM + 16 * k_piece);
        run_k[d][i] = real ? c.k_scale[id * c.heads + head] : 0.0f;
      }
      if (values && i == 0) {
        if (v_half < 2) {
          const int8_t* from = c.v_codes + base + v_lane;
#pragma unroll
          for (int j = 0; j < 8; ++j) raw_v[d][j / 4][j % 4] = *reinterpret_cast<const uint32_t*>(from + (j % 4 + 8 * (j / 4)) * DIM);
        }
        run_v[d] = real ? c.v_scale[id * c.heads + head] : -1.0f;
      }
    }
  };
  auto store = [&](int n) __attribute__((always_inline)) {
    if (keys) {
#pragma unroll
      for (int i = 0; i < KP; ++i) {
        const int t = 16 * run_of(i) + token_of(i), ch = 2 * k_piece;
        u32x4 lo, hi;
        uint32_t two[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f16_word(raw_k[n][i][j], two);
          if (j < 2) lo[2 * j] = two[0], lo[2 * j + 1] = two[1];
          else hi[2 * j - 4] = two[0], hi[2 * j - 3] = two[1];
        }
        k_lds[n][t * KCH + (ch ^ (t & (KCH - 1)))] = lo;
        k_lds[n][t * KCH + ((ch + 1) ^ (t & (KCH - 1)))] = hi;
        if (t % 16 == 0 && k_piece == 0) runs[n][t / 16].k = run_k[n][i];
      }
    }
    if (values) {
      const int ch = 2 * stage + v_half;
      const bool zeros = !(run_v[n] >= 0x1p-90f);  // kLeastLog
      if (v_half < 2) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          u32x4 a;
#pragma unroll
          for (int j = 0; j < 4; ++j) a[j] = f16_bytes(raw_v[n][j / 2][2 * (j % 2) + 1], raw_v[n][j / 2][2 * (j % 2)], b);
          const int d = 4 * v_quad + b;
          v_lds[n][d * (kTile / 8) + (ch ^ ((d ^ (d >> 2)) & 7))] = zeros ? u32x4{0, 0, 0, 0} : a;
        }
      }
      if (lane == 0) {
        runs[n][stage].v_log = zeros ? kLeastLog : __log2f(run_v[n]);
        runs[n][stage].v_inv = zeros ? kSumBy * 0x1p90f : kSumBy / run_v[n];
        runs[n][stage].real = run_v[n] != -1.0f;
      }
    }
  };

  f32x16 out[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) out[b][i] = 0.0f;
  float top = -INFINITY, sum = 0.0f;

  // Codes are loaded two tiles ahead (one ahead: 3% more for four prompts of 1,502 tokens, 5% for 400 tokens of 633).  Of 8
  // waves the keys' convert the next tile before they multiply, the values' after it, so that the two waves of a SIMD are
  // out of step: one's products run under the other's softmax and conversions (149 us, in step 160 us).
  const bool ahead = WAVES == 8 && keys;
  if (begin < end) {
    load_ids(begin);
    load_codes(0, begin);
    load_ids(begin + kTile);
    load_codes(1, begin + kTile);               // (past the end: rows of a page that exists, not seen)
    load_ids(begin + 2 * kTile);
    store(0);
    __syncthreads();
  }
  for (int t0 = begin; t0 < end;) {
#pragma unroll
    for (int buf = 0; buf < 2; ++buf) {
      if (buf && t0 >= end) break;
      const bool more = t0 + kTile < end;
      if (more) {
        if (ahead) store(buf ^ 1);
        load_codes(buf, t0 + 2 * kTile);
        load_ids(t0 + 3 * kTile);
      }
      if (t0 < wave_end) {
        f32x16 s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int t = 32 * b + r;
            const u32x4 a = k_lds[buf][t * KCH + ((2 * k + h) ^ (t & (KCH - 1)))];
            s[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, qf[k]), s[b], 0, 0, 0);
          }
        }
        Run run[kSubs];
        float factor[kSubs];
        int real = 1;
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          run[u] = runs[buf][u];
          factor[u] = run[u].k * qs;
          real &= __builtin_amdgcn_readfirstlane(run[u].real);
        }
        if (t0 + kTile > all_seen || !real) {             // some row does not see some token
#pragma unroll
          for (int u = 0; u < kSubs; ++u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int key = t0 + 16 * u + 8 * (i / 4) + 4 * h + i % 4;
              const bool seen = key < end && key <= last_key && run[u].real;
              s[u / 2][8 * (u % 2) + i] = seen ? s[u / 2][8 * (u % 2) + i] * factor[u] : -INFINITY;
            }
            factor[u] = 1.0f;
            // (a row that sees none of the run: its values' scale, which may be infinite, must not count)
            if (t0 + 16 * u > last_key) run[u].v_log = kLeastLog;
          }
        }
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          float mu = s[u / 2][8 * (u % 2)];
#pragma unroll
          for (int i = 1; i < 8; ++i) mu = fmaxf(mu, s[u / 2][8 * (u % 2) + i]);
          m = fmaxf(m, __builtin_fmaf(mu, factor[u], run[u].v_log));
        }
        if (__any(m > top + kLazy)) {
          const float next = fmaxf(max_halves(m), top), ref = next == -INFINITY ? 0.0f : next;
          const float scaled = __builtin_amdgcn_exp2f(top - ref);
          sum *= scaled;
#pragma unroll
          for (int b = 0; b < DB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) out[b][i] *= scaled;
          top = next;
        }
        const float ref = top == -INFINITY ? 0.0f : top, rest = kProbExp - ref;
        u32x4 p[kSubs];
#pragma unroll
        for (int u = 0; u < kSubs; ++u) {
          const float off = run[u].v_log + rest;
          float add = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u / 2][8 * (u % 2) + i], factor[u], off));
            const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u / 2][8 * (u % 2) + i + 1], factor[u], off));
            add += a + b;
            p[u][i / 2] = f16_pair(a, b);
          }
          sum = __builtin_fmaf(add, run[u].v_inv, sum);
        }
#pragma unroll
        for (int u = 0; u < kSubs; ++u)
#pragma unroll
          for (int b = 0; b < DB; ++b) {
            const int d = 32 * b + r;
            const u32x4 a = v_lds[buf][d * (kTile / 8) + ((2 * u + h) ^ ((d ^ (d >> 2)) & 7))];
            out[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, p[u]), out[b], 0, 0, 0);
          }
      }
      if (more && !ahead) store(buf ^ 1);
      __syncthreads();
      t0 += kTile;
    }
  }

  // ---- outputs: register i of block b is dim 32 b + 8 (i / 4) + 4 h + i % 4 ----
  sum = sum_halves(sum);
  if (row0 + r >= rows) return;
  const float by = splits == 1 ? (sum > 0.0f ? kSumBy / sum : 0.0f) : 1.0f;
  const int64_t index = ((seq * c.heads + head) * rows + row) * splits + split;
  uint16_t* dst = y + ((seq * tokens + row / group) * c.heads * group + head * group + row % group) * DIM;
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int d = 32 * b + 2 * i + 4 * h;
      const f32x4 o = {out[b][i] * by, out[b][i + 1] * by, out[b][i + 2] * by, out[b][i + 3] * by};
      if (splits == 1)
        *reinterpret_cast<u32x2*>(dst + d) = u32x2{bf16x2_rne(o[0], o[1]), bf16x2_rne(o[2], o[3])};
      else
        *reinterpret_cast<f32x4*>(part.out + index * DIM + d) = o;
    }
  if (splits > 1 && h == 0) {
    part.stat[2 * index] = top;
    part.stat[2 * index + 1] = sum;
  }
}

}  // namespace

// What a cut takes, in microseconds as measured (dim 128; 64 in proportion): a workgroup takes 4 and, for a tile
// of 64 tokens, 1.8 with 128 rows alone on its CU, 3.1 with two of them there, 2.5 with 256 rows; the pieces'
// results take 5 and their bytes twice at 4 TB/s.  The longest a table can hold stands for every sequence, and
// a row of a prompt sees half of the prompt.  (400 tokens of 633, 40/8 heads: one piece 25 us, two 31; 64 of 2,000, 32/8: 63
// us in one, 22 in eight pieces of 128 rows, 26 of 256; 500 of 12,016, 32/8: 135 us in four of 128, 121 of 256; 100 of
// 20,000, 16/4: 84 us in eight, 52 in sixteen.)
PromptCut prompt_cut(int64_t seqs, int64_t rows, int64_t tokens, int heads, int dim, int64_t length) {
  const double by_dim = dim / 128.0;
  const double seen = seen_of(tokens, length);
  PromptCut best{0, 0};
  double least = 0.0;
  for (int tile = 128; tile <= 256; tile *= 2) {
    const int64_t one = seqs * heads * ((rows + tile - 1) / tile);
    for (int64_t s = 1; s <= 32; ++s) {
      const int64_t piece = piece_of((int)length, (int)s);
      if (s > 1 && (s - 1) * piece >= length) continue;       // no more pieces than with fewer
      const int64_t n = one * s;
      const double tiles = (double)((piece + kTile - 1) / kTile);
      // (two on a CU, until the one of fewer tiles ends)
      const double per = tile == 256 ? 0.8 + 1.7 * by_dim : 0.9 + 0.9 * by_dim + (n > 256 ? seen * (0.1 + 1.2 * by_dim) : 0.0);
      const double slots = tile == 256 ? 256.0 : 512.0;
      const double whole = 4.0 + tiles * per, all = (double)n * (4.0 + tiles * seen * per) / slots;
      const double join = s > 1 ? 5.0 + 2.0 * (double)(seqs * heads * rows * s) * dim * 4.0 / 4e6 : 0.0;
      const double cost = std::max(whole, all) + join;
      if (!best.rows || cost < least) best = {tile, s}, least = cost;
    }
  }
  return best;
}

template <int DIM>
hipError_t launch_prompt(const KvCache& c, const uint16_t* q, int64_t ldq, int64_t seqs, int64_t tokens, int group,
                         float scale, PromptCut cut, uint16_t* y, Partial part, hipStream_t stream) {
  const int rows = cut.rows;
  const int64_t tiles = (tokens * group + rows - 1) / rows, blocks = c.heads * tiles * cut.splits;      // of a sequence
  const int64_t row = (int64_t)c.heads * tokens * group;                                                // rows of y
  const auto kernel = rows == 256 ? kv_prompt_kernel<DIM, 8> : kv_prompt_kernel<DIM, 4>;
  return in_launches(seqs, blocks, 2 * rows, [&](int64_t b, int64_t n) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(n * blocks)), dim3(2 * rows), 0, stream, c.from(b), q + b * tokens * ldq, ldq, (int)tokens,
                       group, scale, (int)cut.splits, (int)tiles, (int)(n * blocks), y + b * row * DIM,
                       part.from(b * row * cut.splits, DIM));
    return hipGetLastError();
  });
}

template hipError_t launch_prompt<64>(const KvCache&, const uint16_t*, int64_t, int64_t, int64_t, int, float, PromptCut,
                                      uint16_t*, Partial, hipStream_t);
template hipError_t launch_prompt<128>(const KvCache&, const uint16_t*, int64_t, int64_t, int64_t, int, float, PromptCut,
                                       uint16_t*, Partial, hipStream_t);

}  // namespace kva
}  // namespace w8a8
