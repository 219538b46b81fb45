// Rotary positions of queries and keys.
//
// What it computes: pairs (a, b) of the first `rotary` values of every head become A (a cos t - b sin t, b cos t + a sin
// t), t = p f_i for pair i of a token at position p; the rest of the head is copied, and so is a token that has no
// position (p < 0).  Pairs are the halves' (i, i + rotary / 2) or neighbours (2i, 2i + 1).
//
// Angles: f_i comes as a 64-bit fraction of a turn, so that the low 64 bits of p * turns_i are the exact fraction of the
// angle of whole turns, at any position; its upper 32 bits are taken (2^-32 of a turn), split into the nearest quarter
// turn and a rest of at most an eighth, and the rest's sine and cosine are series whose next terms are below 2^-28 of
// it.  Nothing is read but 64 bits a pair, and no table bounds the positions.
//
// A thread keeps one unit of 8 pairs (16 values, two 16-byte pieces) of a token, computes its 8 sines and cosines once,
// and turns that unit of one head after another.  Bound by memory: 8 x 1,502 tokens, 40 and 8 heads of 128, 295 MB in
// 55.9 us (5.3 TB/s); few tokens by the launch (4.2 us).
#include "decode.h"
#include "layer.h"
#include "layer_math.h"

namespace w8a8 {
namespace {

using namespace lm;

constexpr int kThreads = 256;

// Cosine and sine of `turn` / 2^32 turns.
__device__ __forceinline__ void cos_sin(uint32_t turn, float& c, float& s) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float t = (float)(int32_t)(turn - (quarter << 30)) * 0x1.921fb6p-30f;      // 2 pi / 2^32: |t| <= pi / 4
  const float u = t * t;
  float sn = __builtin_fmaf(u, 0x1.71de3ap-19f, -0x1.a01a02p-13f);                  // 1 / 9!, -1 / 7!
  sn = __builtin_fmaf(u, sn, 0x1.111112p-7f);                                       // 1 / 5!
  sn = __builtin_fmaf(u, sn, -0x1.555556p-3f);                                      // -1 / 3!
  sn = __builtin_fmaf(u * t, sn, t);
  float cs = __builtin_fmaf(u, -0x1.27e4fcp-22f, 0x1.a01a02p-16f);                  // -1 / 10!, 1 / 8!
  cs = __builtin_fmaf(u, cs, -0x1.6c16c2p-10f);                                     // -1 / 6!
  cs = __builtin_fmaf(u, cs, 0x1.555556p-5f);                                       // 1 / 4!
  cs = __builtin_fmaf(u, cs, -0.5f);
  cs = __builtin_fmaf(u, cs, 1.0f);
  const bool odd = quarter & 1;
  const float a = odd ? sn : cs, b = odd ? cs : sn;
  c = (quarter + 1) & 2 ? -a : a;                                                   // quarters 1 and 2
  s = quarter & 2 ? -b : b;                                                         // quarters 2 and 3
}

// `slots` of a workgroup work on units of dim / 16 threads each; a token has `parts` of them, which take its heads in
// turn.
template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
rope_rows(Rope r, int64_t first, int64_t rows, uint32_t parts, uint32_t slots) {
  const uint32_t units = r.dim / 16, slot = threadIdx.x / units, unit = threadIdx.x % units;
  if (slot >= slots) return;
  const uint32_t id = blockIdx.x * slots + slot, part = id % parts;   // (below 2^32, as a launch's threads are)
  const int64_t row = first + id / parts;
  if (row >= rows) return;
  const uint32_t seq = (uint32_t)row / (uint32_t)r.tokens, token = (uint32_t)row % (uint32_t)r.tokens;
  const int64_t p = max(r.lens[seq], 0) - r.tokens + token;
  const bool turned = (int)unit < r.rotary / 16 && p >= 0;
  float c[8], s[8];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cos_sin((uint32_t)(((uint64_t)p * r.turns[8 * unit + i]) >> 32), c[i], s[i]);
      c[i] *= r.amplitude;
      s[i] *= r.amplitude;
    }
  }
  // the unit's two pieces of a head: of the halves, or side by side (also behind the rotated part)
  const bool halves = !INTERLEAVED && (int)unit < r.rotary / 16;
  const int lo = (int)(halves ? 8 * unit : 16 * unit), hi = halves ? lo + r.rotary / 2 : lo + 8;
  for (int head = (int)part; head < r.q_heads + r.heads; head += (int)parts) {
    const bool is_q = head < r.q_heads;
    const int h = is_q ? head : head - r.q_heads;
    const uint16_t* x = (is_q ? r.q + row * r.ldq : r.k + row * r.ldk) + h * r.dim;
    uint16_t* y = (is_q ? r.q_out + row * r.ldq_out : r.k_out + row * r.ldk_out) + h * r.dim;
    u32x4 a = *reinterpret_cast<const u32x4*>(x + lo), b = *reinterpret_cast<const u32x4*>(x + hi);
    if (turned) {
      float u[8], v[8];
      widen8(a, u);
      widen8(b, v);
      if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u0 = u[2 * i], v0 = v[2 * i];
          u[2 * i] = __builtin_fmaf(u0, c[i], -u[2 * i + 1] * s[i]);
          u[2 * i + 1] = __builtin_fmaf(u[2 * i + 1], c[i], u0 * s[i]);
          v[2 * i] = __builtin_fmaf(v0, c[4 + i], -v[2 * i + 1] * s[4 + i]);
          v[2 * i + 1] = __builtin_fmaf(v[2 * i + 1], c[4 + i], v0 * s[4 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u0 = u[i];
          u[i] = __builtin_fmaf(u0, c[i], -v[i] * s[i]);
          v[i] = __builtin_fmaf(v[i], c[i], u0 * s[i]);
        }
      }
      a = narrow8(u);
      b = narrow8(v);
    }
    *reinterpret_cast<u32x4*>(y + lo) = a;
    *reinterpret_cast<u32x4*>(y + hi) = b;
  }
}

}  // namespace

hipError_t launch_rope(const Rope& r, hipStream_t stream) {
  const int all = r.q_heads + r.heads, slots = kThreads / (r.dim / 16);
  const int64_t rows = r.seqs * r.tokens;
  // One head a thread, two where there are many rows: 298 tokens of 48 heads of 128 4.2 us (5.8 with six heads a
  // thread), 1 x 1,502 8.2 (9.3 with one, 8.5 with six), 8 x 1,502 55.9 (56.3 with one, 60.1 with six, 4.9 TB/s then).
  const int parts = rows >= 1024 ? (all + 1) / 2 : all;
  // (a launch begins at a row: `parts` workgroups for every `slots` rows)
  return in_launches((rows + slots - 1) / slots, parts, kThreads, [&](int64_t first, int64_t count) {
    const int64_t left = (rows - first * slots) * parts, here = count * parts;
    const unsigned grid = (unsigned)(here * slots < left ? here : (left + slots - 1) / slots);
    if (r.interleaved)
      hipLaunchKernelGGL(rope_rows<true>, dim3(grid), dim3(kThreads), 0, stream, r, first * slots, rows, (uint32_t)parts, (uint32_t)slots);
    else
      hipLaunchKernelGGL(rope_rows<false>, dim3(grid), dim3(kThreads), 0, stream, r, first * slots, rows, (uint32_t)parts, (uint32_t)slots);
    return hipGetLastError();
  });
}

}  // namespace w8a8
