// Product of E4M3 codes with block scales, y = x W^T + b, for many tokens.
//
// What it computes: y[m][n] = bf16(sum over blocks b of 128 columns of s[b][m] * sw[n / 128][b] * (sum over the block of
// q[m][k] * w[n][k]) + bias[n]): the inner sums on the E4M3 matrix instructions (block_math.h), the outer one in fp32.
//
// A workgroup of WGM x WGN waves owns BM tokens x BN weight rows; a wave accumulates 16 TM tokens x 16 TN rows.  One
// stage is one block of 128 columns of both operands, 128 bytes a row, and the scales of both, which NST LDS buffers take
// in turn by direct-to-LDS loads; each product starts from zero and is multiplied into the sums by s * sw, four
// multiply-adds a lane beside 32 cycles of the matrix unit.
//
// A stage's products run over the weight operands, each with all token operands of the wave, which stay in registers;
// weight operands are read kAhead ahead.  As many weight operands before its end the wave has read all of the stage:
// there it waits until the next stage has landed and every wave is as far (one barrier a stage), then issues the loads
// of the stage behind it into the buffer that is free now, one or two beside each product (in one go, both waves of a
// SIMD left the matrix unit idle meanwhile), and replaces each token operand by the next stage's behind its last
// product.
//
// What bounds it: a product takes the matrix unit for 32 cycles and leaves room for four vector instructions beside it;
// each further one, and with one wave a SIMD each instruction of any kind, costs four cycles.  Four are the
// multiply-adds, so the loop has little else: the scales of both operands come with the stage (a scalar load would be
// waited for together with all LDS reads), places in LDS are stepped.  512 x 17,408 x 4,096, 32 tiles of 256 x 256 with
// a CU each, takes 1.14 us a stage of 0.85 in products (1.23 with places computed anew and the weight's scales by scalar
// loads, 1.18 with the barrier a weight operand later, so that the loads come in shorter runs). With all CUs at work the
// clock is what limits: 8,192 x 8,192 x 8,192 takes 395 us (2.78 PFLOP/s), 2,270 x 5,120 x 34,816 330 (2.45), at about
// 1.9 GHz of the 2.4 that 5 PFLOP/s need.  The same products and multiply-adds on operands that stay in registers reach
// 3.45 PFLOP/s at whatever clock that leaves, products alone 4.1; without its loads from memory the kernel was 14%
// faster then, without the barrier 1%.  A matrix instruction of 32 x 32 outputs and other wave priorities were no
// faster; a wave of 128 x 128 outputs, which would read a third less from LDS, has more sums than the 256 registers that
// vector instructions reach.
//
// Smaller tiles are for what fills the CUs better with them: 1,502 x 4,096 x 4,096 26 us, one round of 256 workgroups;
// 64 x 5,120 x 34,816 38 us, the weight's bytes at 4.7 TB/s.
#include <algorithm>
#include <type_traits>

#include "block_choice.h"
#include "block_math.h"
#include "decode.h"
#include "layer.h"

namespace w8a8 {
namespace {

using namespace lm;
using block_choice::choose;
using block_choice::Choice;
using block_choice::kCus;

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// 16 (4) bytes a lane from a buffer straight into LDS, lane i's at l + 16 i (4 i); l is uniform over the wave.
__device__ __forceinline__ void lds_load16(Buffer p, uint32_t at, uint32_t from, uint8_t* l) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(p, (__attribute__((address_space(3))) void*)l, 16, (int)at, (int)from, 0, 0);
#endif
}
__device__ __forceinline__ void lds_load4(Buffer p, uint32_t at, uint32_t from, uint8_t* l) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(p, (__attribute__((address_space(3))) void*)l, 4, (int)at, (int)from, 0, 0);
#endif
}

// Until at most n of this wave's vector memory operations are in flight, and its LDS operations are done.
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "vmcnt's range");
  __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | ((n >> 4) << 14));
}

// Tiles are walked in groups of kGroupM token tiles, a contiguous range of them on each XCD, so that the workgroups that
// run at once on an XCD share panels in its L2.  (Groups of 4, 6, 8 and 16 differ by up to 5%: 12,016 x 17,408 x 5,120
// 930, 903, 935 and 947 us, 2,270 x 5,120 x 34,816 348, 350, 354 and 352.)
constexpr int kGroupM = 6;
__device__ __forceinline__ void tile_of(uint32_t t, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t per_group = kGroupM * tiles_n, group = t / per_group, first = group * kGroupM, in = t - group * per_group;
  const uint32_t size = min((uint32_t)kGroupM, tiles_m - first);
  tm = first + in % size;
  tn = in / size;
}

// Rows of 128 bytes in LDS, eight pieces of 16: piece c of row r at c ^ (r / 2 % 8).  16 lanes of a read take the same
// piece of 16 consecutive rows in one cycle; even and odd rows lie in the two halves of the 64 banks, and the key spreads
// each half's eight rows over its eight pieces.  (With r % 8 as the key, rows r and r + 8 meet and a read takes twice as
// long, which does not show where the clock is the limit: 2,270 x 5,120 x 34,816 371 us with either.)
__device__ __forceinline__ int lds_key(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int lds_piece(int r, int c) { return r * 128 + ((c ^ lds_key(r)) << 4); }

// WALK: a workgroup for each CU, which walks over tiles of its XCD's range; the stages run on from one tile into the
// next, whose first ones load while this tile's outputs leave.  Otherwise a workgroup for each tile.
template <int BM, int BN, int WGM, int WGN, int NST, bool WALK>
__global__ void __launch_bounds__(64 * WGM * WGN)
block_tile(const uint8_t* __restrict__ q, const float* __restrict__ s, const uint8_t* __restrict__ w, const float* __restrict__ sw,
           const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t M, int64_t N, int K, uint32_t tiles_m, uint32_t tiles_n, uint32_t first,
           int split_blocks, float* __restrict__ sums) {
  constexpr int NT = 64 * WGM * WGN, WTM = BM / WGM, WTN = BN / WGN, TM = WTM / 16, TN = WTN / 16;
  constexpr int A_LOADS = BM * 8 / NT, B_LOADS = BN * 8 / NT, SCALES = (BM + BN) * 128;
  constexpr int STAGE = SCALES + BM * 4 + 256, LOADS = A_LOADS + B_LOADS + 1, AREA = WALK ? 2048 : 0, BIAS = WALK ? BN * 2 : 0;
  static_assert(A_LOADS * NT == BM * 8 && B_LOADS * NT == BN * 8, "whole loads");
  static_assert(WTN <= 128 && 128 % WTN == 0, "a wave's weight rows have one scale");
  static_assert(WGM * WGN > BM / 64, "a wave for the weight's scales");
  static_assert(!WALK || NST == 2, "walking, a stage waits for every load, the bias and the last tile's stores among them");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NST * STAGE + WGM * WGN * AREA + 2 * BIAS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), c = lane & 15, h = lane >> 4;
  const int wm = wave % WGM, wn = wave / WGM;
  const int64_t s_ld = block_scale_stride(M);

  // this workgroup's tiles: `at`, at + step, ... below `end`, and its blocks of columns: `blocks` from `block0` on
  uint32_t at, end, step = 1;
  const int all_blocks = K / kScaleBlock;
  int block0 = 0, blocks = all_blocks;
  if constexpr (WALK) {
    const uint32_t tiles = tiles_m * tiles_n, q8 = tiles / 8, r8 = tiles % 8, xcd = blockIdx.x % 8, begin = xcd * q8 + min(xcd, r8);
    at = begin + blockIdx.x / 8, end = begin + q8 + (xcd < r8 ? 1 : 0), step = gridDim.x / 8;
    if (at >= end) return;
  } else {
    const uint32_t id = first + (uint32_t)xcd_order(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n, split = id / tiles;
    at = __builtin_amdgcn_readfirstlane(id - split * tiles), end = at + 1;
    block0 = __builtin_amdgcn_readfirstlane(split) * split_blocks, blocks = min(split_blocks, all_blocks - block0);
  }
  // Loads of a tile: thread t of round i fills the 16 bytes at LDS place 16 (i NT + t), piece (t % 8) ^ key of row (i NT
  // + t) / 8; rows past the last one are the last one again (their sums are not stored).  And one load of scales: the
  // first waves 64 tokens' each, the others the weight rows', one for 128 rows (all the same: every wave issues as many
  // loads).
  Buffer abuf, bbuf;
  const bool token_scales = wave < BM / 64;
  const float* load_s;                                    // the scales of the block to load (64 bits: they may lie far apart)
  const int64_t s_step = token_scales ? s_ld : 1;         // from one block to the next
  uint32_t a_at[A_LOADS], b_at[B_LOADS], s_at;
  int64_t load_m, load_n;                                 // its first token and weight row
  int aimed = 0;                                          // tiles aimed at
  const int bias_wave = wave % (BN < 128 ? 1 : BN / 128);
  auto place = [&](uint32_t r, int p) -> uint32_t { return r / 32 * 32 * (uint32_t)K + r % 32 * 64 + (p >> 2) * 2048 + (p & 3) * 16; };
  auto aim = [&](uint32_t t) __attribute__((always_inline)) {
    uint32_t tm, tn;
    tile_of(t, tiles_m, tiles_n, tm, tn);
    load_m = (int64_t)__builtin_amdgcn_readfirstlane(tm) * BM, load_n = (int64_t)__builtin_amdgcn_readfirstlane(tn) * BN;
    abuf = buffer(q + load_m * K + block0 * 4096), bbuf = buffer(w + load_n * K + block0 * 4096);
    load_s = token_scales ? s + block0 * s_ld + load_m : sw + load_n / kScaleBlock * all_blocks + block0;
    const uint32_t m_last = (uint32_t)min(M - 1 - load_m, (int64_t)BM), n_last = (uint32_t)min(N - 1 - load_n, (int64_t)BN);
    int id = tid;
    if constexpr (WALK) asm volatile("" : "+v"(id));      // (what follows from it is computed again, not kept in registers)
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i) {
      const uint32_t r = (i * NT + id) / 8;
      a_at[i] = place(min(r, m_last), (id & 7) ^ lds_key(r));
    }
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i) {
      const uint32_t r = (i * NT + id) / 8;
      b_at[i] = place(min(r, n_last), (id & 7) ^ lds_key(r));
    }
    const int lane = id & 63;
    s_at = (token_scales ? min((uint32_t)(64 * wave + lane), m_last) : min((uint32_t)lane, n_last / kScaleBlock) * all_blocks) * 4;
    // walking, the tile's bias goes to LDS too (two places in turn; pairs of columns, those past N the last pair)
    if (WALK && bias)
      lds_load4(buffer(bias + load_n), min((uint32_t)(128 * bias_wave + 2 * lane), n_last - 1) * 2, 0,
                lds + NST * STAGE + WGM * WGN * AREA + (aimed & 1) * BIAS + bias_wave * 256);
    ++aimed;
  };
  uint32_t load_at = at;
  uint32_t load_k = 0;                                    // the block to load, of tile load_at: its place, 4096 a block
  auto issue_one = [&](auto t_c, uint32_t to_stage) __attribute__((always_inline)) {   // load t of the stage at that place
    constexpr int t = decltype(t_c)::value;
    uint8_t* to = lds + to_stage;
    if constexpr (t < A_LOADS) lds_load16(abuf, a_at[t], load_k, to + wave * 1024 + t * NT * 16);
    else if constexpr (t < A_LOADS + B_LOADS) lds_load16(bbuf, b_at[t - A_LOADS], load_k, to + BM * 128 + wave * 1024 + (t - A_LOADS) * NT * 16);
    else lds_load4(buffer(load_s), s_at, 0, to + SCALES + min(wave, BM / 64) * 256);
  };

  // Places in LDS of what this lane reads, which step from stage to stage (an instruction more beside a product is one
  // too many: up to four vector instructions run in its shadow): pieces h and 4 + h, which are columns 16 h .. + 15 and
  // 64 + 16 h .. + 15, of the first row of the wave's tokens and weight rows, the first token's scale and the weight
  // rows'.
  uint32_t x_at[2], w_at[2], ts_at = SCALES + (wm * WTM + c) * 4, ws_at = SCALES + BM * 4 + wn * WTN / kScaleBlock * 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) x_at[i] = lds_piece(wm * WTM + c, h + 4 * i), w_at[i] = BM * 128 + lds_piece(wn * WTN + c, h + 4 * i);
  auto step_by = [&](uint32_t& at, int by) __attribute__((always_inline)) {
    at += by;
    asm volatile("" : "+v"(at));
  };
  auto read = [&](const uint32_t (&at)[2], int k) __attribute__((always_inline)) -> i32x8 {   // 16 rows further each
    const u32x4 u = *reinterpret_cast<const u32x4*>(lds + at[0] + 2048 * k), v = *reinterpret_cast<const u32x4*>(lds + at[1] + 2048 * k);
    return i32x8{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
  };
  // Product u of a stage (weight operand u / TM, token operand u % TM) is added to the sums behind product u + kLag: an
  // instruction that reads a product's result too early waits for it.  The last kLag of a stage are added in the next.
  // (Two weight operands ahead where few waves have few products each: 512 x 17,408 x 4,096 with 64 x 128 by four waves
  // 45.4 us, 48.7 with three; 128 x 128 by eight 55 and 51.5, 256 x 256 161 and 156.)
  constexpr int P = TM * TN, kLag = TM > 3 ? 3 : TM - 1, kParts = 4, kAhead = NT > 256 || TM > 2 ? 3 : 2, kTail = kAhead * TM;
  static_assert(TN >= 4 && TN % 4 == 0 && TM >= 2, "products in flight, weight operands ahead");
  f32x4 acc[TN][TM], part[kParts];
  i32x8 xr[TM], wr[4];
  float by[TM], raw[TM], raw_w;
  auto read_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TM; ++j) raw[j] = *reinterpret_cast<const float*>(lds + ts_at + 64 * j);
    raw_w = *reinterpret_cast<const float*>(lds + ws_at);
  };
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kParts; ++i) part[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < TM; ++j) by[j] = 0.0f;
  };
  auto add = [&](auto u_c, float f) __attribute__((always_inline)) {
    constexpr int u = decltype(u_c)::value;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[u / TM][u % TM][e] = __builtin_fmaf(part[u % kParts][e], f, acc[u / TM][u % TM][e]);
  };

  // The next stage has landed (the stages behind it may still be on their way) and this wave's LDS reads are done, and
  // so for every wave.
  auto landed = [&]() __attribute__((always_inline)) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    wait_loads<(NST - 2) * LOADS>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };

  // Outputs: a product leaves 8 bytes of each of 16 rows a store, so a wave lays rows out in LDS first, pieces of 16
  // bytes at c ^ row, and stores runs of whole row segments.  Walking, in 16 rows x 64 columns of an area of its own;
  // otherwise all at once in the stages' place.
  auto outputs = [&](int64_t mb, int64_t nb, int tile) __attribute__((always_inline)) {
    const uint32_t m_left = (uint32_t)min(M - mb, (int64_t)BM), n_left = (uint32_t)min(N - nb, (int64_t)BN);
    if (!WALK && sums) {                                  // a part of K: its sums [part][M][N], for add_splits
      const int h = lane >> 4, c = lane & 15;
      float* to = sums + (int64_t)(block0 / split_blocks) * M * N;
      static_for<0, TM>([&](auto j_c) __attribute__((always_inline)) {
        static_for<0, TN>([&](auto i_c) __attribute__((always_inline)) {
          constexpr int i = decltype(i_c)::value, j = decltype(j_c)::value;
          const uint32_t m = wm * WTM + 16 * j + c, n = wn * WTN + 16 * i + 4 * h;
          if (m < m_left && n < n_left) *reinterpret_cast<f32x4*>(to + (mb + m) * N + nb + n) = acc[i][j];
        });
      });
      return;
    }
    float bias4[WALK ? 1 : TN][4];
    if constexpr (!WALK) {
      const int h = lane >> 4;
#pragma unroll
      for (int i = 0; i < TN; ++i) {
        if (bias) bf16x4(*reinterpret_cast<const uint2*>(bias + min(nb + wn * WTN + 16 * i + 4 * h, N - 4)), bias4[i]);
        else bias4[i][0] = bias4[i][1] = bias4[i][2] = bias4[i][3] = 0.0f;
      }
    }
    int lane_ = lane;
    if constexpr (WALK) asm volatile("" : "+v"(lane_));   // (as above)
    const int lane = lane_, c = lane & 15, h = lane >> 4;
    const uint8_t* biases = lds + NST * STAGE + WGM * WGN * AREA + (tile & 1) * BIAS;
    auto lay = [&](uint8_t* to, auto i_c, auto j_c, int pieces) __attribute__((always_inline)) {   // block (i, j) at column 16 i of its row
      constexpr int i = decltype(i_c)::value, j = decltype(j_c)::value;
      float b4[4];
      if constexpr (WALK) {
        bf16x4(*reinterpret_cast<const uint2*>(biases + (wn * WTN + 16 * i + 4 * h) * 2), b4);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b4[e] = bias4[i][e];
      }
      const f32x4 v = acc[i][j];
      const uint2 o = make_uint2(bf16x2_rne(v[0] + b4[0], v[1] + b4[1]), bf16x2_rne(v[2] + b4[2], v[3] + b4[3]));
      *reinterpret_cast<uint2*>(to + c * pieces * 16 + (((2 * i + (h >> 1)) ^ c) % pieces) * 16 + (h & 1) * 8) = o;
    };
    auto laid = [&]() __attribute__((always_inline)) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
      __builtin_amdgcn_wave_barrier();
    };
    if constexpr (WALK) {
      static_assert(!WALK || WTN % 64 == 0, "64 columns at a time");
      uint8_t* area = lds + NST * STAGE + wave * AREA;
      // (an output of 256 rows lies within 2^31 bytes of its first)
      const Buffer ybuf = __builtin_amdgcn_make_buffer_rsrc(y + mb * N + nb, 0, 0x7fffffff, 0x00020000);
      static_for<0, TM>([&](auto j_c) __attribute__((always_inline)) {
        static_for<0, WTN / 64>([&](auto half) __attribute__((always_inline)) {
          static_for<0, 4>([&](auto i_c) __attribute__((always_inline)) {
            lay(area, std::integral_constant<int, 4 * decltype(half)::value + decltype(i_c)::value>{}, j_c, 8);
          });
          laid();
#pragma unroll
          for (int r = 0; r < 16; r += 8) {
            const int row = r + lane / 8, piece = lane % 8;
            const u32x4 v = *reinterpret_cast<const u32x4*>(area + row * 128 + ((piece ^ row) % 8) * 16);
            const uint32_t m = wm * WTM + 16 * decltype(j_c)::value + row, n = wn * WTN + 64 * decltype(half)::value + 8 * piece;
            const uint32_t off = m < m_left && n < n_left ? (m * (uint32_t)N + n) * 2 : 0x80000000u;
            __builtin_amdgcn_raw_buffer_store_b128(v, ybuf, (int)off, 0, 2);
          }
          laid();
        });
      });
    } else {
      constexpr int PIECES = WTN / 8, ROWS = 64 / PIECES, REGION = WTM * WTN * 2;
      static_assert(REGION * WGM * WGN <= NST * STAGE, "outputs fit the stages");
      asm volatile("" ::: "memory");
      wait_loads<0>();                                      // nothing lands in LDS behind this
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      uint8_t* region = lds + wave * REGION;
      static_for<0, TM>([&](auto j_c) __attribute__((always_inline)) {
        static_for<0, TN>([&](auto i_c) __attribute__((always_inline)) { lay(region + 16 * decltype(j_c)::value * WTN * 2, i_c, j_c, PIECES); });
      });
      laid();
      const int piece = lane % PIECES;
#pragma unroll
      for (int r = 0; r < WTM; r += ROWS) {
        const int row = r + lane / PIECES;
        const uint32_t m = wm * WTM + row, n = wn * WTN + 8 * piece;
        const u32x4 v = *reinterpret_cast<const u32x4*>(region + row * (WTN * 2) + ((piece ^ (row % 16)) % PIECES) * 16);
        if (m < m_left && n < n_left) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + (mb + m) * N + nb + n));
      }
    }
  };

  if (WALK && !bias) {                                     // (seen by all behind the first stage's barrier)
    for (int i = tid; i < 2 * BIAS / 4; i += NT) *reinterpret_cast<uint32_t*>(lds + NST * STAGE + WGM * WGN * AREA + 4 * i) = 0;
  }
  aim(load_at);
  int64_t mb = load_m, nb = load_n;                       // the tile that is multiplied
#pragma unroll
  for (int b = 0; b < NST; ++b) {
    static_for<0, LOADS>([&](auto t_c) __attribute__((always_inline)) { issue_one(t_c, b * STAGE); });
    if (b + 1 < blocks) load_k += 4096, load_s += s_step;  // (past the last block: that one again, not used)
    if (b == NST - 2) landed();
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kAhead; ++i) wr[i] = read(w_at, i);  // (in the loop's order, so that it waits for no more than it needs)
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    xr[j] = read(x_at, j);
    if (j == 0) read_scales();
    __builtin_amdgcn_sched_barrier(0);
  }
  uint32_t now = 0;                                       // place of the stage that is multiplied
  clear();
  for (int tile = 0;; ++tile) {
    // the loads are NST blocks ahead: of this tile, then of the next, or its last block again where there is none
    int b = 0;
    uint32_t load_step = 4096;
#pragma clang loop unroll(disable)
    for (int part_of = 0; part_of < 2; ++part_of) {
      const int stop = part_of == 0 ? blocks - NST : blocks;
      if (part_of == 1) {
        if (WALK && load_at + step < end) load_at += step, load_k = 0, aim(load_at);
        else load_step = 0, load_s -= load_k == (uint32_t)blocks * 4096 ? s_step : 0, load_k = (uint32_t)(blocks - 1) * 4096;
      }
#pragma clang loop unroll(disable)
      for (; b < stop; ++b) {
        const int to_next = now == (NST - 1) * STAGE ? -(NST - 1) * STAGE : STAGE;
        static_for<0, P>([&](auto u_c) __attribute__((always_inline)) {
          constexpr int u = decltype(u_c)::value, i = u / TM, j = u % TM, t = u - (P - kTail);
          if constexpr (t == 0) landed();
          __builtin_amdgcn_sched_barrier(0);
          part[u % kParts] = mfma128(wr[i % 4], xr[j]);
          if constexpr (u < kLag) {
            add(std::integral_constant<int, P - kLag + u>{}, by[TM - kLag + u]);
          } else {
            if constexpr (u - kLag < TM) by[u - kLag] = raw[u - kLag] * raw_w;
            add(std::integral_constant<int, u - kLag>{}, by[(u - kLag) % TM]);
          }
          if constexpr (t == 0) step_by(w_at[0], to_next), step_by(w_at[1], to_next);
          if constexpr (j == 0) wr[(i + kAhead) % 4] = read(w_at, (i + kAhead) % TN);
          if constexpr (i == TN - 1 && j == 0) step_by(x_at[0], to_next), step_by(x_at[1], to_next), step_by(ts_at, to_next), step_by(ws_at, to_next);
          if constexpr (i == TN - 1) xr[j] = read(x_at, j);
          if constexpr (i == TN - 1 && j == 0) read_scales();
          if constexpr (t >= 0)
            static_for<t * LOADS / kTail, (t + 1) * LOADS / kTail>([&](auto l_c) __attribute__((always_inline)) { issue_one(l_c, now); });
        });
        load_k += load_step, load_s += load_step ? s_step : 0;
        now += to_next;
      }
    }
    static_for<0, kLag>([&](auto u_c) __attribute__((always_inline)) {
      constexpr int u = decltype(u_c)::value;
      add(std::integral_constant<int, P - kLag + u>{}, by[TM - kLag + u]);
    });
    outputs(mb, nb, tile);
    if constexpr (!WALK) break;
    at += step;
    if (at >= end) break;
    mb = load_m, nb = load_n;
    clear();
  }
  wait_loads<0>();                                        // nothing lands in LDS behind the workgroup's end
}

// y = the sums of the parts of K, in their order, and the bias: 8 columns a thread.
__global__ void __launch_bounds__(256)
add_splits(const float* __restrict__ sums, int splits, const uint16_t* __restrict__ bias, uint16_t* __restrict__ y, int64_t values, int64_t N,
           int64_t first) {
  const int64_t at = ((first + blockIdx.x) * 256 + threadIdx.x) * 8;
  if (at >= values) return;
  float v[8], b[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) *reinterpret_cast<f32x4*>(v + 4 * i) = *reinterpret_cast<const f32x4*>(sums + at + 4 * i);
  for (int k = 1; k < splits; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(sums + k * values + at + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] += u[e];
    }
  if (bias) {
    widen8(*reinterpret_cast<const u32x4*>(bias + at % N), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
  }
  *reinterpret_cast<u32x4*>(y + at) = narrow8(v);
}

struct Call {
  const uint8_t* q;
  const float* s;
  const uint8_t* w;
  const float* sw;
  const uint16_t* bias;
  uint16_t* y;
  int64_t M, N, K;
  hipStream_t stream;
};

template <int BM, int BN, int WGM, int WGN, int NST, bool WALK>
hipError_t launch(const Call& c, int splits, float* sums) {
  const int64_t tiles_m = (c.M + BM - 1) / BM, tiles_n = (c.N + BN - 1) / BN;   // (fewer than 2^27 tiles)
  const int blocks = (int)(c.K / kScaleBlock), split_blocks = (blocks + splits - 1) / splits;
  auto run = [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL((block_tile<BM, BN, WGM, WGN, NST, WALK>), dim3((unsigned)count), dim3(64 * WGM * WGN), 0, c.stream, c.q, c.s, c.w, c.sw,
                       c.bias, c.y, c.M, c.N, (int)c.K, (uint32_t)tiles_m, (uint32_t)tiles_n, (uint32_t)first, split_blocks,
                       splits > 1 ? sums : nullptr);
    return hipGetLastError();
  };
  if (WALK) return run(0, std::min<int64_t>((tiles_m * tiles_n + 7) / 8, kCus / 8) * 8);
  const hipError_t e = in_launches(tiles_m * tiles_n * splits, 1, 64 * WGM * WGN, run);
  if (e != hipSuccess || splits == 1) return e;
  return in_launches((c.M * c.N + 2047) / 2048, 1, 256, [&](int64_t first, int64_t count) {
    hipLaunchKernelGGL(add_splits, dim3((unsigned)count), dim3(256), 0, c.stream, sums, splits, c.bias, c.y, c.M * c.N, c.N, first);
    return hipGetLastError();
  });
}

}  // namespace

size_t block_gemm_workspace(int64_t M, int64_t N, int64_t K) {
  if (block_few_fits(M, N, K)) return 0;
  const int splits = choose(M, N, K).splits;
  return splits == 1 ? 0 : (size_t)splits * M * N * sizeof(float);
}

hipError_t launch_block_gemm(const uint8_t* q, const float* s, const uint8_t* w, const float* sw, const uint16_t* bias, uint16_t* y, int64_t M,
                             int64_t N, int64_t K, float* sums, hipStream_t stream) {
  if (block_few_fits(M, N, K)) return launch_block_few(q, s, w, sw, bias, y, M, N, K, stream);
  const Choice c = choose(M, N, K);
  const Call call{q, s, w, sw, bias, y, M, N, K, stream};
  switch (c.tile) {
    case 0: return launch<256, 256, 4, 2, 2, true>(call, 1, nullptr);
    case 1: return launch<192, 256, 2, 2, 2, false>(call, c.splits, sums);
    case 2: return launch<128, 256, 2, 4, 3, false>(call, c.splits, sums);
    case 3: return launch<64, 256, 2, 4, 3, false>(call, c.splits, sums);
    case 4: return launch<192, 128, 2, 2, 3, false>(call, c.splits, sums);
    case 5: return launch<128, 128, 4, 2, 3, false>(call, c.splits, sums);
    case 6: return launch<64, 128, 2, 2, 3, false>(call, c.splits, sums);
    default: return launch<64, 64, 2, 1, 3, false>(call, c.splits, sums);
  }
}

}  // namespace w8a8
