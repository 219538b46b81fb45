// Projections of a few tokens with 4-bit weights.
//
// What it computes: y[m][n] = bf16( sum_g s[n][g] * sum_{k in g} x[m][k] * c[n][k] + bias[n] ) with codes
// c in [-8, 7], one bf16 scale for each row and group of 32, 64 or 128 columns, bf16 activations and
// fp32 sums.  For a few tokens the weight codes are the traffic (half a byte for every 2M operations),
// so the kernel is built around one pass over them.
#include "decode.h"
#include "epilogue_math.h"

namespace w8a8 {
namespace {

typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 16;          // rows of a packed block (an MFMA operand's rows)
constexpr int kCols = 128;         // columns of a packed block
constexpr int kBlockBytes = kRows * kCols / 2;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) { return (uint16_t)bf16x2_rne(f, 0.0f); }

// ---- quantizer: rows of w -> row-major codes and scales ------------------------
// One thread per 8 columns, group / 8 neighbouring lanes per group: s = bf16(amax / 7), codes
// RNE(w / s) clamped to +-7 (the rounded scale may be below amax / 7, by up to 2^-9 of it).
// 17,408 x 5,120 take 65 us (3.5 TB/s), packing them 33 us: both run once, when a weight is loaded.
__global__ void __launch_bounds__(256)
w4_quantize_kernel(const uint16_t* __restrict__ w, int64_t chunks, int lanes, uint32_t* __restrict__ codes,
                   uint16_t* __restrict__ scales) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool live = j < chunks;
  const u32x4 raw = *reinterpret_cast<const u32x4*>(w + 8 * (live ? j : chunks - 1));
  float v[8], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(raw[i] << 16);
    v[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
  for (int d = 1; d < lanes; d <<= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
  const uint16_t sb = f32_to_bf16(amax / 7.0f);
  const float s = bf16_to_f32(sb);
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = s > 0.0f ? fminf(fmaxf(rintf(v[i] / s), -7.0f), 7.0f) : 0.0f;
    word |= (uint32_t)((int)c + 8) << (4 * i);
  }
  if (!live) return;
  codes[j] = word;
  if (j % lanes == 0) scales[j / lanes] = sb;
}

// ---- row-major codes and scales -> the packed layout ------------------------------
// One thread per word of 8 codes: element i of the row-major word is nibble i; in the packed word the even
// elements 2p sit at bits 4p and the odd ones at 16 + 4p, so that one shift and mask give an aligned pair.
__global__ void __launch_bounds__(256)
w4_pack_codes_kernel(const uint32_t* __restrict__ codes, int64_t N, int64_t K, int64_t words, uint32_t* __restrict__ out) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= words) return;
  const int st = j % 4, r = j / 4 % 16, h = j / 64 % 4;
  const int64_t block = j / 256, kb = block % (K / kCols), n = block / (K / kCols) * kRows + r;
  uint32_t word = 0x88888888u;                 // padding rows: code 0
  if (n < N) {
    const uint32_t c = codes[(n * K + kb * kCols + st * 32 + h * 8) / 8];
    word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= ((c >> (4 * i)) & 15u) << (4 * (i / 2) + 16 * (i % 2));
  }
  out[j] = word;
}

__global__ void __launch_bounds__(256)
w4_pack_scales_kernel(const uint16_t* __restrict__ scales, int64_t N, int64_t groups, int64_t total,
                      uint16_t* __restrict__ out) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= total) return;
  const int64_t r = j % kRows, g = j / kRows % groups, n = j / kRows / groups * kRows + r;
  out[j] = n < N ? scales[n * groups + g] : 0;
}

// ---- the projection --------------------------------------------------------------
// K is cut into kSegs * splits runs of 128-column blocks, run j from blocks * j / runs on; `splits` follows from N
// and K alone.  Every form below sums a run block by block and group by group and then adds the runs in order
// (those of a split first, then the splits), so an output does not depend on which form computed it.
constexpr int kSegs = 8;
__device__ __forceinline__ int run_begin(int blocks, int run, int runs) {
  return (int)((unsigned)(blocks * run) / (unsigned)runs);
}

// Eight nibbles of a packed word -> eight bf16 values 128 + (code + 8): a bf16 between 128 and 256 has
// steps of one, so the nibble is its low mantissa bits and one and-or makes two values (with the mask in a vector
// register: the instruction takes one scalar).
__device__ __forceinline__ bf16x8 widen(uint32_t w, uint32_t mask) {
  u32x4 v;
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = ((w >> (4 * p)) & mask) | 0x43004300u;
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ uint32_t nibble_mask() {
  uint32_t m = 0x000f000fu;
  asm volatile("" : "+v"(m));
  return m;
}
// Eight times -136: the widened codes' offset goes out through the accumulator, which starts a group at
// -136 * sum(x), itself an MFMA.
__device__ __forceinline__ bf16x8 minus_offset() {
  const u32x4 v = {0xc308c308u, 0xc308c308u, 0xc308c308u, 0xc308c308u};
  return __builtin_bit_cast(bf16x8, v);
}

// v + bias[n .. n + 3], rounded to y[m][n .. n + 3]; or a split's part of it.
__device__ __forceinline__ void store_outputs(f32x4 v, int64_t m, int64_t n, int64_t M, int64_t N, const uint16_t* bias,
                                              uint16_t* y, float* part, int split, int splits) {
  if (splits > 1) {
    *reinterpret_cast<f32x4*>(part + (split * M + m) * N + n) = v;
    return;
  }
  if (bias) {
    float b[4];
    bf16x4(*reinterpret_cast<const uint2*>(bias + n), b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b[i];
  }
  *reinterpret_cast<u32x2*>(y + m * N + n) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
}

// Up to 16 tokens.  A workgroup computes RB blocks of 16 rows; each of its kSegs waves takes one run of columns,
// and the runs meet in LDS.  MFMA 16x16x32: A = weights (lane 16 h + r: row r, columns 8 h .. 8 h + 7 of a
// 32-column step), B = tokens, D: lane 16 h + t holds rows 4 h .. 4 h + 3 of token t.  Bound by the weights' bytes:
// a wave has the next block's loads in flight while it multiplies.  x and the scales pass through an LDS area
// of the wave's own: loaded straight into operands, a block of x takes 4 instructions that touch 16 rows
// each (and with groups of 32 the scales 4 more per row block), which held 5 tokens of 17,408 x 5,120 to 27 us; as
// XI instructions of 4 whole row pieces and one for the scales they take 14.8 us.  1 token of
// 5,120 x 34,816 takes 18.6 us (4.9 TB/s), 16 take 22.0 us.
template <int XI, int RB, int GPB>
__global__ void __launch_bounds__(64 * kSegs)
w4_few_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint16_t* __restrict__ s,
              const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, float* __restrict__ part, int64_t M, int64_t N,
              int64_t K) {
  constexpr int XROWS = 4 * XI;                // token rows kept (M <= XROWS; the operand's other lanes repeat them)
  constexpr int SL = 2 * GPB;                  // 16-byte pieces of a row block's scales
  static_assert(RB * SL <= 64, "one instruction brings the scales");
  constexpr int AREA = XROWS * 16 + 64;        // 16-byte units of a wave's area
  constexpr int UNITS = kSegs * (AREA > RB * 64 ? AREA : RB * 64);
  __shared__ __attribute__((aligned(16))) u32x4 lds[UNITS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4, t = lane & 15;
  const int split = blockIdx.z, splits = gridDim.z;
  const int64_t blocks = (N + kRows - 1) / kRows, b0 = (int64_t)blockIdx.x * RB;
  const int kb_all = (int)(K / kCols);
  const int first = run_begin(kb_all, split * kSegs + wave, kSegs * splits);
  const int n = run_begin(kb_all, split * kSegs + wave + 1, kSegs * splits) - first;
  u32x4* xl = lds + wave * AREA;
  u32x4* sl = xl + XROWS * 16;

  const uint16_t* xp[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) xp[i] = x + min((int64_t)(4 * i + h), M - 1) * K + 8 * t;     // past M: row M - 1, not stored
  const uint8_t* wp[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) wp[rb] = w + min(b0 + rb, blocks - 1) * kb_all * kBlockBytes + 16 * lane;
  const int sc_piece = min(lane, RB * SL - 1);
  const uint16_t* sp = s + min(b0 + sc_piece / SL, blocks - 1) * kb_all * (GPB * kRows) + sc_piece % SL * 8;
  const bf16x8 offset = minus_offset();
  const uint32_t mask = nibble_mask();

  f32x4 tot[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) tot[rb] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 wv[2][RB], xv[XI], sv;
  auto load_w = [&](int d, int i) __attribute__((always_inline)) {
    const int64_t kb = first + min(i, n - 1);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) wv[d][rb] = *reinterpret_cast<const u32x4*>(wp[rb] + kb * kBlockBytes);
  };
  auto load_x = [&](int i) __attribute__((always_inline)) {
    const int kb = first + min(i, n - 1);
#pragma unroll
    for (int j = 0; j < XI; ++j) xv[j] = *reinterpret_cast<const u32x4*>(xp[j] + kb * kCols);
    sv = *reinterpret_cast<const u32x4*>(sp + kb * (GPB * kRows));
  };
  // a wave's LDS operations are done in their order, so its area needs no barrier
  auto put_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < XI; ++j) xl[(4 * j + h) * 16 + (t ^ (4 * j + h))] = xv[j];
    sl[lane] = sv;
  };
  auto multiply = [&](int d) __attribute__((always_inline)) {
    constexpr int SPG = 4 / GPB;               // MFMA steps per group
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      bf16x8 xf[SPG];
      f32x4 base = {0.f, 0.f, 0.f, 0.f};
      uint2 sw[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) sw[rb] = reinterpret_cast<const uint2*>(sl)[(rb * GPB + g) * 4 + h];
#pragma unroll
      for (int st = 0; st < SPG; ++st) {
        const int row = t % XROWS;
        xf[st] = __builtin_bit_cast(bf16x8, xl[row * 16 + ((4 * (g * SPG + st) + h) ^ row)]);
        base = __builtin_amdgcn_mfma_f32_16x16x32_bf16(offset, xf[st], base, 0, 0, 0);
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        f32x4 acc = base;
#pragma unroll
        for (int st = 0; st < SPG; ++st)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(wv[d][rb][g * SPG + st], mask), xf[st], acc, 0, 0, 0);
        float sc[4];
        bf16x4(sw[rb], sc);
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[rb][i] = __builtin_fmaf(sc[i], acc[i], tot[rb][i]);
      }
    }
  };
  if (n > 0) {
    load_x(0);
    load_w(0, 0);
    for (int i = 0; i < n; i += 2) {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        if (d && i + d >= n) break;
        __builtin_amdgcn_sched_barrier(0);
        load_w(d ^ 1, i + d + 1);
        __builtin_amdgcn_sched_barrier(0);
        put_x();
        load_x(i + d + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(d);
      }
    }
  }

  f32x4* red = reinterpret_cast<f32x4*>(lds);
  __syncthreads();                             // every wave is done with its area
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) red[(wave * RB + rb) * 64 + lane] = tot[rb];
  __syncthreads();
  for (int j = threadIdx.x; j < RB * 64; j += 64 * kSegs) {
    const int64_t m = j % 16, row = (b0 + j / 64) * kRows + 4 * (j % 64 / 16);
    if (m >= M || row >= N) continue;          // N % 8 == 0: the four rows are whole or absent
    f32x4 v = red[j];
#pragma unroll
    for (int wv = 1; wv < kSegs; ++wv) v += red[wv * RB * 64 + j];
    store_outputs(v, m, row, M, N, bias, y, part, split, splits);
  }
}

__device__ __forceinline__ void lds_barrier() {       // __syncthreads would wait for the loads in flight, too
  asm volatile("" ::: "memory");                      // (no store moves below the wait, no load above the barrier)
  __builtin_amdgcn_s_waitcnt(0xc07f);                 // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// From 17 tokens on, 32 at a time, while the workgroups go a few times round the 256 CUs.  As above, a wave takes a
// run of columns through an LDS area of its own; a widened weight serves two blocks of tokens, and the
// offset's MFMA RB blocks of rows.  A workgroup walks over items (RB blocks of rows, 32 tokens, a split) and
// loads the next item's first step while it still multiplies and adds up the present one.  What bounds it is the
// issue of a step's MFMAs (40 for RB = 4, 640 cycles) and vector instructions (210, 840 cycles) by two waves a SIMD,
// which overlap little: 4,400 cycles a step, and 4,000 with every load a cache hit.  64 tokens of 5,120 x 5,120 take
// 11.4 us and 64 of 4,096 x 4,096 8.8 us, where a tile of x shared by waves of different rows (the form below) takes
// 27.3 and 22.2 us with its few waves.  The scales are read with the operands: read where they are used they
// cost 34.9 us instead of 31.0 (64 tokens of 17,408 x 5,120, groups of 32).  x and scales two steps ahead, four blocks
// of tokens a wave, or workgroups that end with their item were no faster.
template <int RB, int GPB>
__global__ void __launch_bounds__(64 * kSegs)
w4_mid_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint16_t* __restrict__ s,
               const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, float* __restrict__ part, int64_t M, int64_t N,
               int64_t K, unsigned m_blocks, unsigned row_items, int splits) {
  constexpr int MB = 2, TOKENS = 16 * MB, XI = 4 * MB, SPG = 4 / GPB;
  constexpr int SL = 2 * GPB;                  // 16-byte pieces of a row block's scales
  static_assert(RB * SL <= 64, "one instruction brings the scales");
  constexpr int AREA = TOKENS * 16 + 64;       // 16-byte units of a wave's area
  __shared__ __attribute__((aligned(16))) u32x4 lds[kSegs * (AREA + RB * MB * 64)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4, t = lane & 15;
  const int64_t blocks = (N + kRows - 1) / kRows;
  const int kb_all = (int)(K / kCols);
  u32x4* xl = lds + wave * AREA;
  u32x4* sl = xl + TOKENS * 16;
  f32x4* red = reinterpret_cast<f32x4*>(lds + kSegs * AREA);
  const unsigned xcd = blockIdx.x % 8;

  // the XCD's item j: an XCD's workgroups take all tokens of a split of RB row blocks together, so its L2 brings
  // the weights once
  struct Item {
    int64_t m0, b0;
    int split, first, n;
  };
  auto item_at = [&](unsigned j) __attribute__((always_inline)) {
    Item a;
    const unsigned r = j / m_blocks, c = r / splits;
    a.m0 = (int64_t)(j - r * m_blocks) * TOKENS;
    a.split = r - c * splits;
    a.b0 = (int64_t)(c * 8 + xcd) * RB;
    a.first = run_begin(kb_all, a.split * kSegs + wave, kSegs * splits);
    a.n = run_begin(kb_all, a.split * kSegs + wave + 1, kSegs * splits) - a.first;
    return a;
  };
  const unsigned rows_here = (row_items + 7 - xcd) / 8, mine = rows_here * splits * m_blocks, step = gridDim.x / 8;
  unsigned j = blockIdx.x / 8;
  if (j >= mine) return;
  Item cur = item_at(j), nxt = cur;            // the one that is multiplied, and the one that is loaded: its
  unsigned jn = j;                             // number and its step
  int ln = 0;
  uint32_t xo[XI], so;                         // bytes; past M and past N: the last row again, not stored
  auto lanes = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XI; ++i) xo[i] = 2 * ((uint32_t)min((int64_t)(4 * i + h), M - 1 - nxt.m0) * (uint32_t)K + 8 * t);
    const int piece = min(lane, RB * SL - 1);
    so = 2 * ((uint32_t)min((int64_t)(piece / SL), blocks - 1 - nxt.b0) * (uint32_t)(kb_all * GPB * kRows) + piece % SL * 8);
  };
  lanes();
  const bf16x8 offset = minus_offset();
  const uint32_t mask = nibble_mask();
  f32x4 tot[RB][MB];
  u32x4 wv[2][RB], xv[XI], sv;
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) tot[rb][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  auto load_w = [&](int d) __attribute__((always_inline)) {
    const int64_t kb = min(nxt.first + ln, kb_all - 1);
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      wv[d][rb] = *reinterpret_cast<const u32x4*>(w + (min(nxt.b0 + rb, blocks - 1) * kb_all + kb) * kBlockBytes + 16 * lane);
  };
  auto load_x = [&]() __attribute__((always_inline)) {
    const int64_t kb = min(nxt.first + ln, kb_all - 1);
    const char* xb = reinterpret_cast<const char*>(x + nxt.m0 * K + kb * kCols);
#pragma unroll
    for (int i = 0; i < XI; ++i) xv[i] = *reinterpret_cast<const u32x4*>(xb + xo[i]);
    sv = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(s + (nxt.b0 * kb_all + kb) * (GPB * kRows)) + so);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    if (++ln < nxt.n) return;
    ln = 0;
    jn += step;
    if (jn < mine) nxt = item_at(jn), lanes();
  };
  // a wave's LDS operations are done in their order, so its area needs no barrier
  auto put_x = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < XI; ++i) xl[(4 * i + h) * 16 + (t ^ ((4 * i + h) & 15))] = xv[i];
    sl[lane] = sv;
  };
  auto multiply = [&](int d) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < GPB; ++g) {
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 xf[SPG][MB];
      f32x4 base[MB];
      uint2 sw[RB];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) sw[rb] = reinterpret_cast<const uint2*>(sl)[(rb * GPB + g) * 4 + h];
#pragma unroll
      for (int st = 0; st < SPG; ++st)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          xf[st][mb] = __builtin_bit_cast(bf16x8, xl[(16 * mb + t) * 16 + ((4 * (g * SPG + st) + h) ^ t)]);
          base[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(offset, xf[st][mb], st ? base[mb] : f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        f32x4 acc[MB];
#pragma unroll
        for (int st = 0; st < SPG; ++st) {
          const bf16x8 a = widen(wv[d][rb][g * SPG + st], mask);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
            acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xf[st][mb], st ? acc[mb] : base[mb], 0, 0, 0);
        }
        float sc[4];
        bf16x4(sw[rb], sc);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) tot[rb][mb][e] = __builtin_fmaf(sc[e], acc[mb][e], tot[rb][mb][e]);
      }
    }
  };
  auto finish = [&]() __attribute__((always_inline)) {
    lds_barrier();                             // the last item's sums have been read
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
        red[((wave * RB + rb) * MB + mb) * 64 + lane] = cur.n ? tot[rb][mb] : f32x4{0.f, 0.f, 0.f, 0.f};
    clear();
    lds_barrier();
    for (int q = threadIdx.x; q < RB * MB * 64; q += 64 * kSegs) {
      const int64_t m = cur.m0 + 16 * (q / 64 % MB) + q % 16, row = (cur.b0 + q / (64 * MB)) * kRows + 4 * (q % 64 / 16);
      if (m >= M || row >= N) continue;        // N % 8 == 0: the four rows are whole or absent
      f32x4 v = red[q];
#pragma unroll
      for (int r = 1; r < kSegs; ++r) v += red[r * RB * MB * 64 + q];
      store_outputs(v, m, row, M, N, bias, y, part, cur.split, splits);
    }
  };
  load_x();
  load_w(0);
  advance();
  int i = 0;
  for (;;) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      __builtin_amdgcn_sched_barrier(0);
      load_w(d ^ 1);
      __builtin_amdgcn_sched_barrier(0);
      put_x();
      load_x();
      advance();
      __builtin_amdgcn_sched_barrier(0);
      multiply(d);
      __builtin_amdgcn_sched_barrier(0);
      if (++i >= cur.n) {
        finish();
        j += step;
        if (j >= mine) return;
        cur = item_at(j);
        i = 0;
      }
    }
  }
}

// Many tokens and rows, 64 tokens at a time.  A wave owns a block of 16 rows and walks the split's columns; the workgroup's
// waves share each 128-column tile of x in LDS (two of them, one barrier a block), so x is read once for
// all their rows.  Weights and scales go straight to registers, kAhead blocks ahead.  What bounds it is the
// step from block to block: per wave 32 MFMAs, 16 operand reads and ~120 vector instructions that the
// barrier keeps in step, about 2,600 cycles for 9 waves where each pipe alone would need 1,150: 64 tokens of
// 5,120 x 34,816 take 49 us (a wave per row block without sharing x took 197 us).
constexpr int kAhead = 4;
template <int GPB, int WMIN, int WMAX>
__global__ void __launch_bounds__(64 * WMAX)
w4_many_kernel(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, const uint16_t* __restrict__ s,
               const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, float* __restrict__ part, int64_t M, int64_t N,
               int64_t K) {
  constexpr int MB = 4, PIECES = MB * 256;     // 16-byte pieces of a tile of x
  constexpr int XP = (PIECES + 64 * WMIN - 1) / (64 * WMIN);     // of a thread, at least WMIN waves
  constexpr int SPG = 4 / GPB;
  __shared__ __attribute__((aligned(16))) u32x4 tile[2 * PIECES];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int h = lane >> 4, t = lane & 15;
  const int split = blockIdx.z, splits = gridDim.z, runs = kSegs * splits;
  const int64_t blocks = (N + kRows - 1) / kRows, mine = (int64_t)blockIdx.x * waves + wave, m0 = (int64_t)blockIdx.y * 16 * MB;
  const int kb_all = (int)(K / kCols);
  const int first = run_begin(kb_all, split * kSegs, runs), n = run_begin(kb_all, split * kSegs + kSegs, runs) - first;

  const uint16_t* xp[XP];
  int xo[XP];
#pragma unroll
  for (int i = 0; i < XP; ++i) {
    const int p = min(tid + i * 64 * waves, PIECES - 1), row = p / 16, ch = p % 16;   // (past the last: the last again)
    xp[i] = x + min(m0 + row, M - 1) * K + (int64_t)first * kCols + 8 * ch;
    xo[i] = row * 16 + (ch ^ (row & 15));
  }
  const int64_t block = min(mine, blocks - 1) * kb_all + first;
  const uint8_t* wp = w + block * kBlockBytes + 16 * lane;
  const uint16_t* sp = s + block * (GPB * kRows) + 4 * h;
  const bf16x8 offset = minus_offset();
  const uint32_t mask = nibble_mask();

  f32x4 tot[MB], sum[MB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) tot[mb] = sum[mb] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 xr[XP], wv[kAhead];
  uint2 sv[kAhead][GPB];
  auto load_x = [&](int i) __attribute__((always_inline)) {
    const int kb = min(i, n - 1);
#pragma unroll
    for (int j = 0; j < XP; ++j) xr[j] = *reinterpret_cast<const u32x4*>(xp[j] + kb * kCols);
  };
  auto put_x = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < XP; ++j) tile[b * PIECES + xo[j]] = xr[j];
  };
  auto load_w = [&](int d, int i) __attribute__((always_inline)) {
    const int64_t kb = min(i, n - 1);
    wv[d] = *reinterpret_cast<const u32x4*>(wp + kb * kBlockBytes);
#pragma unroll
    for (int g = 0; g < GPB; ++g) sv[d][g] = *reinterpret_cast<const uint2*>(sp + (kb * GPB + g) * kRows);
  };
  if (n > 0) {
    // (in the loop's order, the last weights after the second tile, so that waiting for a tile never waits for
    // weights that are not needed yet)
    load_x(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < kAhead - 1; ++d) load_w(d, d);
    __builtin_amdgcn_sched_barrier(0);
    put_x(0);
    load_x(1);
    __builtin_amdgcn_sched_barrier(0);
    load_w(kAhead - 1, kAhead - 1);
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    int run = 0, run_end = 0, b = 0;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
      for (int d = 0; d < kAhead; ++d) {
        const int i = i0 + d;
        if (d && i >= n) break;
        put_x(b ^ 1);                          // read last before the barrier just passed
        load_x(i + 2);
        __builtin_amdgcn_sched_barrier(0);
        if (i == run_end) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            sum[mb] += tot[mb];
            tot[mb] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
          do {                                 // (runs of no blocks add nothing)
            ++run;
            run_end = run < kSegs ? run_begin(kb_all, split * kSegs + run, runs) - first : n;
          } while (i == run_end);
        }
#pragma unroll
        for (int g = 0; g < GPB; ++g) {
          f32x4 acc[MB];
          bf16x8 xf[SPG][MB];
#pragma unroll
          for (int st = 0; st < SPG; ++st)
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
              xf[st][mb] = __builtin_bit_cast(bf16x8, tile[b * PIECES + (16 * mb + t) * 16 + ((4 * (g * SPG + st) + h) ^ t)]);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb) {
            acc[mb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < SPG; ++st) acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(offset, xf[st][mb], acc[mb], 0, 0, 0);
          }
#pragma unroll
          for (int st = 0; st < SPG; ++st) {
            const bf16x8 a = widen(wv[d][g * SPG + st], mask);
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) acc[mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xf[st][mb], acc[mb], 0, 0, 0);
          }
          float sc[4];
          bf16x4(sv[d][g], sc);
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int e = 0; e < 4; ++e) tot[mb][e] = __builtin_fmaf(sc[e], acc[mb][e], tot[mb][e]);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_w(d, i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
        b ^= 1;
        lds_barrier();
      }
    }
  }
  if (mine >= blocks) return;
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const int64_t m = m0 + 16 * mb + t, row = mine * kRows + 4 * h;
    if (m < M && row < N) store_outputs(sum[mb] + tot[mb], m, row, M, N, bias, y, part, split, splits);
  }
}

// The splits' parts, added in order: four outputs a thread.
__global__ void __launch_bounds__(256)
w4_combine_kernel(const float* __restrict__ part, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t M,
                  int64_t N, int splits) {
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= M * N / 4) return;
  f32x4 v = *reinterpret_cast<const f32x4*>(part + 4 * j);
  for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(part + s * M * N + 4 * j);
  store_outputs(v, 4 * j / N, 4 * j % N, M, N, bias, y, nullptr, 0, 1);
}

struct Linear {
  const uint16_t* x;
  const uint8_t* w;
  const uint16_t* s;
  const uint16_t* bias;
  uint16_t* y;
  float* part;
  int64_t M, N, K;
  int group, splits;
  hipStream_t stream;
};

template <int XI, int RB>
hipError_t launch_few(const Linear& a) {
  const int64_t blocks = (a.N + kRows - 1) / kRows, gx = (blocks + RB - 1) / RB;
  const dim3 grid((unsigned)gx, 1, (unsigned)a.splits), block(64 * kSegs);
  const auto kernel = a.group == 128 ? w4_few_kernel<XI, RB, 1> : a.group == 64 ? w4_few_kernel<XI, RB, 2> : w4_few_kernel<XI, RB, 4>;
  hipLaunchKernelGGL(kernel, grid, block, 0, a.stream, a.x, a.w, a.s, a.bias, a.y, a.part, a.M, a.N, a.K);
  return hipGetLastError();
}

template <int RB>
hipError_t launch_mid(const Linear& a) {
  const int64_t blocks = (a.N + kRows - 1) / kRows, row_items = (blocks + RB - 1) / RB, m_blocks = (a.M + 31) / 32;
  const int64_t items = (row_items + 7) / 8 * 8 * m_blocks * a.splits;           // (XCDs take the same number)
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  const auto kernel = a.group == 128 ? w4_mid_kernel<RB, 1> : a.group == 64 ? w4_mid_kernel<RB, 2> : w4_mid_kernel<RB, 4>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>(items, 256)), dim3(64 * kSegs), 0, a.stream, a.x, a.w, a.s, a.bias,
                     a.y, a.part, a.M, a.N, a.K, (unsigned)m_blocks, (unsigned)row_items, a.splits);
  return hipGetLastError();
}

template <int WMIN, int WMAX>
hipError_t launch_many(const Linear& a, int waves) {
  const int64_t blocks = (a.N + kRows - 1) / kRows;
  const dim3 grid((unsigned)((blocks + waves - 1) / waves), (unsigned)((a.M + 63) / 64), (unsigned)a.splits);
  const auto kernel = a.group == 128  ? w4_many_kernel<1, WMIN, WMAX>
                      : a.group == 64 ? w4_many_kernel<2, WMIN, WMAX>
                                      : w4_many_kernel<4, WMIN, WMAX>;
  hipLaunchKernelGGL(kernel, grid, dim3(64 * waves), 0, a.stream, a.x, a.w, a.s, a.bias, a.y, a.part, a.M, a.N, a.K);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, uint8_t* codes,
                              uint16_t* scales, hipStream_t stream) {
  constexpr int kPart = 2048;        // rows
  const int64_t parts = (N + kPart - 1) / kPart, each = kPart * (K / 8) / 256;     // (K % 128 == 0: whole workgroups)
  return in_launches(parts, each, 256, [&](int64_t p, int64_t n) {
    const int64_t row = p * kPart, chunks = std::min(n * kPart, N - row) * K / 8;
    hipLaunchKernelGGL(w4_quantize_kernel, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, stream, w + row * K, chunks, group / 8,
                       reinterpret_cast<uint32_t*>(codes + row * (K / 2)), scales + row * (K / group));
    return hipGetLastError();
  });
}

hipError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, int group,
                          uint8_t* codes_packed, uint16_t* scales_packed, hipStream_t stream) {
  constexpr int kPart = 2048;        // rows, whole packed blocks
  const int64_t rows = (N + kRows - 1) / kRows * kRows, parts = (rows + kPart - 1) / kPart, each = kPart * (K / 8) / 256;
  return in_launches(parts, each, 256, [&](int64_t p, int64_t n) {
    const int64_t row = p * kPart, count = std::min(n * kPart, rows - row), words = count * K / 8, total = count * (K / group);
    hipLaunchKernelGGL(w4_pack_codes_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, stream,
                       reinterpret_cast<const uint32_t*>(codes + row * (K / 2)), N - row, K, words,
                       reinterpret_cast<uint32_t*>(codes_packed + row * (K / 2)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(w4_pack_scales_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream, scales + row * (K / group),
                       N - row, K / group, total, scales_packed + row * (K / group));
    return hipGetLastError();
  });
}

// Splits of K: one launch is faster unless a weight is long and narrow, where too few workgroups would each walk a
// long K (5 tokens of 17,408 x 5,120: 19.3 us in one piece, 15.6 us in three with their combination; 5,120 x 5,120
// and 5,120 x 34,816 are faster in one).  It does not go by M: a token's sums are the same in every batch.
int w4_splits(int64_t N, int64_t K) {
  const int64_t blocks = (N + kRows - 1) / kRows;
  return blocks <= 512 && K / kCols >= 96 ? 3 : 1;
}

namespace {

// Up to kSplitTokens tokens, any number where K is not cut.
hipError_t launch_tokens(const Linear& a) {
  const int64_t M = a.M, N = a.N;
  const int64_t blocks = (N + kRows - 1) / kRows;
  hipError_t e;
  if (M <= 16) {
    if (M <= 4) {
      // row blocks of a workgroup share x, as long as there are workgroups for the 256 CUs
      e = blocks * a.splits >= 512 ? launch_few<1, 2>(a) : launch_few<1, 1>(a);
    } else {
      // x weighs more: a round of 256 workgroups was measured to take about 3, 4, 6 and 8 parts with 1 to 4 row blocks
      // (16 tokens of 5,120 x 34,816: 35, 26, 22 and 27 us in 9, 5, 3 and 3 rounds; of 8,192 x 8,192 11.5, 10.3, 10.8
      // and 13.4 us in 2, 1, 1 and 1)
      constexpr int kParts[5] = {0, 3, 4, 6, 8};
      int rb = 1;
      int64_t least = 0;
      for (int v = 1; v <= 4; ++v) {
        const int64_t cost = ((blocks + v - 1) / v * a.splits + 255) / 256 * kParts[v];
        if (v == 1 || cost <= least) rb = v, least = cost;
      }
      e = rb == 1 ? launch_few<4, 1>(a) : rb == 2 ? launch_few<4, 2>(a) : rb == 3 ? launch_few<4, 3>(a) : launch_few<4, 4>(a);
    }
  } else {
    // 32 tokens and RB row blocks an item, or 64 tokens and a row block for each of v waves: a round of the 256
    // CUs was measured to take about RB + 2 parts of one and 2 (v + 3) of the other (of 128 columns a run: 1.2 us
    // a part), and up to 32 tokens half of the second's work would be thrown away
    int rb = 2, waves = 0;
    int64_t least = 0;
    for (int v = 2; v <= 4; ++v) {
      const int64_t cost = (((blocks + v - 1) / v) * ((M + 31) / 32) * a.splits + 255) / 256 * (v + 2);
      if (v == 2 || cost < least) rb = v, least = cost;
    }
    for (int v = 4; v <= 12 && M > 32; ++v) {
      const int64_t cost = ((blocks + v - 1) / v * ((M + 63) / 64) * a.splits + 255) / 256 * 2 * (v + 3);
      if (cost < least) waves = v, least = cost;
    }
    if (waves) e = waves < 8 ? launch_many<4, 7>(a, waves) : launch_many<8, 12>(a, waves);
    else e = rb == 2 ? launch_mid<2>(a) : rb == 3 ? launch_mid<3>(a) : launch_mid<4>(a);
  }
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(w4_combine_kernel, dim3((unsigned)((M * N / 4 + 255) / 256)), dim3(256), 0, a.stream, a.part, a.bias, a.y, M, N,
                     a.splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_linear(const uint16_t* x, const uint8_t* codes_packed, const uint16_t* scales_packed,
                            const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int group,
                            void* workspace, hipStream_t stream) {
  const int splits = w4_splits(N, K);
  const int64_t most = splits == 1 ? M : kSplitTokens;
  for (int64_t m = 0; m < M; m += most) {
    const hipError_t e = launch_tokens({x + m * K, codes_packed, scales_packed, bias, y + m * N, static_cast<float*>(workspace),
                                        std::min(most, M - m), N, K, group, splits, stream});
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace w8a8
