/*
 * w8a8.h -- C ABI of the MI355X (gfx950) W8A8 quantized projection library.
 *
 * The library implements the quantized decoder projection described on the
 * pages about quantized Clef checkpoints:
 *   - "CLEF Calibrated INT8 ConvRot" model card (Benefits list, notes under the
 *     latency table): activations of the INT8 text projections go through a
 *     rotation-plus-per-token-int8 quantizer, then an integer GEMM whose
 *     epilogue fuses the scales, the bias and the paired gate/up SwiGLU;
 *   - "Loading CLEF INT8" usage page: gate/up weights are packed into a single
 *     matrix when loaded; weights are immutable once loaded; fuse_mlp selects
 *     the paired gate/up epilogue;
 *   - "clef-flash-FP8" card (Quantization table, note after recipe.yaml): the
 *     FP8 W8A8 dynamic scheme, E4M3 weights with per-output-channel scales taken
 *     from the weights and E4M3 activations with per-token scales computed at
 *     run time.
 * Where the pages leave the arithmetic open, the library takes these readings:
 *   int8 scale s = amax/127 (fp32 IEEE division), code = round-half-even(y/s);
 *   fp8 scale s = amax/448, code = nearest OCP E4M3FN of clamp(y/s, +-448);
 *   a zero row has s = 0 and all-zero codes; the rotation is the normalized
 *   Sylvester Walsh-Hadamard transform of order 128 on each block of 128
 *   consecutive K elements, computed exactly and rounded once to fp32;
 *   the epilogue rounds once to bf16 (round half to even).
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers on the current HIP device.
 *     Tensors are dense, row-major, with the last dimension contiguous:
 *       x      bf16 [M, K]   (raw uint16 bit patterns)
 *       w      int8 [N, K]   or E4M3FN codes uint8 [N, K] (output-channel rows)
 *       q      int8 [M, K]   or E4M3FN codes uint8 [M, K]
 *       s_tok  fp32 [M],  s_ch fp32 [N]
 *       bias   bf16 [N]   (may be NULL: no bias)
 *       y      bf16 [M, N]
 *   - Every pointer must be 16-byte aligned.
 *   - The caller owns every buffer.  The library never allocates, frees or
 *     synchronizes; every call only enqueues kernels on `stream` (NULL is the
 *     default stream) and returns.  Calls are therefore safe to capture into
 *     a HIP graph.  Inputs are never written; outputs are fully overwritten;
 *     outputs must not alias inputs or the workspace.
 *   - All argument checks run on the host before anything is enqueued; on an
 *     error nothing is written and the status says why.  M == 0 is W8A8_OK and
 *     enqueues nothing;
 *     since it touches no memory, its pointers are not checked.  Faults inside
 *     kernels surface at the caller's next synchronization, as with any
 *     asynchronous HIP call.
 *   - Inputs must be finite; results for non-finite inputs are unspecified.
 *   - Shape limits: M >= 0; 1 <= K <= W8A8_MAX_K and K % 128 == 0 for the GEMM
 *     entry points (K % 32 == 0 for the quantizers alone; K % 128 == 0 whenever
 *     rot_block == 128); N >= 1 and N % 8 == 0; rot_block is 0 or 128.
 *     W8A8_MAX_K keeps every int8 accumulator (|acc| <= 127*127*K) inside int32.
 *   - Entry points are reentrant; the only global state is a per-device cache
 *     of the architecture check (the device must be gfx950).
 */
#ifndef W8A8_H
#define W8A8_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define W8A8_MAX_K 131072

typedef enum {
  W8A8_OK = 0,
  W8A8_ERR_NULL_POINTER = 1,       /* a required pointer is NULL (bias may be NULL) */
  W8A8_ERR_BAD_SHAPE = 2,          /* M < 0, N or K out of range or not a multiple as required */
  W8A8_ERR_MISALIGNED = 3,         /* a pointer is not 16-byte aligned */
  W8A8_ERR_BAD_ARGUMENT = 4,       /* a scalar argument outside its values (rot_block: 0 or 128), or the workspace is too small */
  W8A8_ERR_UNSUPPORTED_DEVICE = 5, /* no HIP device, or the current device is not gfx950 */
  W8A8_ERR_LAUNCH = 6,             /* the kernel launch itself failed (hipGetLastError) */
  W8A8_ERR_SCRATCH_TOO_SMALL = 7   /* w8a8_linear_packed_noalloc: the call needs more than
                                      W8A8_NOALLOC_MAX_WORKSPACE bytes of scratch */
} w8a8_status;

/* Human-readable name of a status code (static storage, never NULL). */
const char* w8a8_status_string(w8a8_status s);

/* ---- packed operand layout ---------------------------------------------------
 * A matrix of `rows` rows of K one-byte codes (K % 64 == 0) stored as blocks of
 * 32 rows x 64 bytes: block (r / 32, k / 64) starts at byte
 * ((r / 32) * (K / 64) + k / 64) * 2048 and holds row r % 32 of the block at
 * byte 64 * (r % 32) within it.  The row count is rounded up to a multiple of
 * 32.  Each 32-row, 64-byte piece of a GEMM stage is then one contiguous 2 KiB
 * read.  Weights are immutable once loaded ("Loading CLEF INT8" page, as with
 * the load-time gate/up packing), so a loader packs them once with
 * w8a8_pack_weight and calls the *_packed whole-path entry points. */

/* Bytes of the packed form of `rows` x K codes: ceil(rows / 32) * 32 * K
 * (0 for rows <= 0 or K <= 0). */
size_t w8a8_packed_bytes(int64_t rows, int64_t K);

/* Row-major codes w [rows, K] (int8 or E4M3FN, any one-byte codes) -> the packed
 * layout in w_packed (w8a8_packed_bytes(rows, K) bytes, caller-owned; padding
 * rows are written as zeros).  K % 64 == 0, 64 <= K <= W8A8_MAX_K.  For the
 * SwiGLU entry points pack the whole [2N, K] gate/up matrix in one call. */
w8a8_status w8a8_pack_weight(const void* w, int64_t rows, int64_t K, void* w_packed,
                             hipStream_t stream);

/* Bytes of device workspace the whole-path entry points need for M tokens of
 * K features: the int8 (or E4M3FN) codes of x in the packed layout
 * (w8a8_packed_bytes(M, K) bytes) followed by the fp32 scales [M], each part
 * starting on a 256-byte boundary.  Returns 0 for M <= 0 or K <= 0. */
size_t w8a8_workspace_bytes(int64_t M, int64_t K);

/* ---- stage 1: per-row dynamic symmetric quantizer ----------------------------
 * Per-token activation quantizer of the ConvRot INT8 path (INT8 ConvRot card,
 * latency-table notes) and of the FP8 dynamic scheme (clef-flash-FP8 card,
 * Quantization table).  For each row m of x: optionally rotate each block of
 * 128 (rot_block == 128), take amax = max|y|, s_tok[m] = amax/127 (int8) or
 * amax/448 (fp8), then q = round-half-even(y/s) clamped to +-127 (int8) or
 * the nearest E4M3FN value of clamp(y/s, +-448) (fp8).  Applied to the rows of
 * a weight matrix W [N, K] the same call gives the per-output-channel weight
 * codes and scales (weight scales computed straight from the weights, note
 * after the FP8 card's recipe.yaml). */
w8a8_status w8a8_quantize_act(const uint16_t* x, int64_t M, int64_t K, int rot_block,
                              int8_t* q, float* s_tok, hipStream_t stream);
w8a8_status w8a8_quantize_act_fp8(const uint16_t* x, int64_t M, int64_t K, int rot_block,
                                  uint8_t* q, float* s_tok, hipStream_t stream);
/* The same quantizers writing the codes in the packed layout (K % 64 == 0;
 * q_packed holds w8a8_packed_bytes(M, K) bytes; its padding rows are left
 * untouched).  One set of packed activation codes can feed several packed
 * GEMMs -- e.g. projections that share their input. */
w8a8_status w8a8_quantize_act_packed(const uint16_t* x, int64_t M, int64_t K, int rot_block,
                                     int8_t* q_packed, float* s_tok, hipStream_t stream);
w8a8_status w8a8_quantize_act_fp8_packed(const uint16_t* x, int64_t M, int64_t K, int rot_block,
                                         uint8_t* q_packed, float* s_tok, hipStream_t stream);

/* ---- stage 2 alone: acc[m][n] = sum_k q[m][k] * w[n][k], exact int32 ----------
 * The raw integer contraction (diagnostic / test entry point). acc is int32 [M, N].
 * The _packed form takes both code matrices in the packed layout (q_packed of M
 * rows, w_packed of N rows) and runs the same kernel, tile choice and K loop as
 * w8a8_gemm_dequant_packed, so it exposes the accumulators that epilogue sees. */
w8a8_status w8a8_gemm_i32(const int8_t* q, const int8_t* w, int32_t* acc,
                          int64_t M, int64_t N, int64_t K, hipStream_t stream);
w8a8_status w8a8_gemm_i32_packed(const int8_t* q_packed, const int8_t* w_packed, int32_t* acc,
                                 int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- stages 2+3: integer GEMM with the fused dequant epilogue ---------------
 * y[m][n] = bf16( acc[m][n] * s_tok[m] * s_ch[n] + bias[n] ), computed from the
 * exact int32 accumulator in fp32 with a single final rounding (INT8 ConvRot
 * card, Benefits list: scales and bias fused into the GEMM). */
w8a8_status w8a8_gemm_dequant(const int8_t* q, const float* s_tok, const int8_t* w, const float* s_ch,
                              const uint16_t* bias, uint16_t* y,
                              int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- stages 2+3': integer GEMM with the paired gate/up SwiGLU epilogue -------
 * w is the packed [2N, K] weight (gate rows 0..N-1, up rows N..2N-1, as packed
 * at load time on the "Loading CLEF INT8" page), s_ch and bias (nullable) are
 * [2N].  With g and u the unrounded dequantized values of rows n and N+n,
 * y[m][n] = bf16( silu(g) * u ), y is [M, N]. */
w8a8_status w8a8_gemm_swiglu(const int8_t* q, const float* s_tok, const int8_t* w_gateup,
                             const float* s_ch, const uint16_t* bias, uint16_t* y,
                             int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- fp8 stages 2+3: E4M3FN x E4M3FN GEMM (fp32 accumulation) + dequant ------
 * y[m][n] = bf16( (sum_k dec(q[m][k]) * dec(w[n][k])) * s_tok[m] * s_ch[n] + bias[n] ).
 * The fp32 summation order is fixed per output element and does not depend on
 * M, so results are independent of how rows are batched. */
w8a8_status w8a8_fp8_gemm_dequant(const uint8_t* q, const float* s_tok, const uint8_t* w,
                                  const float* s_ch, const uint16_t* bias, uint16_t* y,
                                  int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- stages 2+3 on packed operands ---------------------------------------------
 * w8a8_gemm_dequant / w8a8_gemm_swiglu / w8a8_fp8_gemm_dequant with both code
 * matrices in the packed layout: q_packed from w8a8_quantize_act*_packed (M
 * rows), the weight from w8a8_pack_weight (N rows, or 2N gate/up rows).  Same
 * arithmetic and results as the row-major forms. */
w8a8_status w8a8_gemm_dequant_packed(const int8_t* q_packed, const float* s_tok, const int8_t* w_packed,
                                     const float* s_ch, const uint16_t* bias, uint16_t* y, int64_t M,
                                     int64_t N, int64_t K, hipStream_t stream);
w8a8_status w8a8_gemm_swiglu_packed(const int8_t* q_packed, const float* s_tok,
                                    const int8_t* w_gateup_packed, const float* s_ch,
                                    const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                    hipStream_t stream);
w8a8_status w8a8_fp8_gemm_dequant_packed(const uint8_t* q_packed, const float* s_tok,
                                         const uint8_t* w_packed, const float* s_ch,
                                         const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                                         int64_t K, hipStream_t stream);

/* ---- unfused gate/up: SwiGLU of separately projected gate and up -------------
 * The "Loading CLEF INT8" page's fuse_mlp=False setting disables the paired
 * gate/up epilogue: gate and up are then ordinary linears (for example one
 * w8a8_linear onto the 2N packed rows, giving [M, 2N]) and this call combines
 * their bf16 outputs: y[m][n] = bf16( silu(gate[m][n]) * up[m][n] ), evaluated
 * in fp32 (g / (1 + exp(-g)) * u) with one round to nearest even.  gate and up
 * are bf16 [M, N] whose rows are `ld` elements apart (ld >= N; ld = 2N and
 * up = gate + N for the halves of a [M, 2N] projection); y is dense [M, N].
 * N % 8 == 0, ld % 8 == 0, pointers 16-byte aligned; y must not overlap the
 * inputs. */
w8a8_status w8a8_swiglu(const uint16_t* gate, const uint16_t* up, int64_t ld, uint16_t* y,
                        int64_t M, int64_t N, hipStream_t stream);

/* ---- whole paths: quantize x into the workspace, then GEMM + epilogue --------
 * `workspace` must hold w8a8_workspace_bytes(M, K) bytes (256-byte aligned is
 * best; 16-byte aligned is required) and is used as scratch for the quantized
 * activations and their scales; its contents afterwards are those codes (in
 * the packed layout) and scales.  Two kernels are enqueued on `stream` (the
 * quantizer, then the GEMM) -- or, for short int8 batches (M <= 512,
 * K <= 1024, at most 256 tiles of 32 tokens x 64 weight rows), one kernel
 * that quantizes each tile's rows itself, with the same codes, scales and
 * outputs.  The plain forms take the
 * row-major weight; the *_packed forms take the weight as written by
 * w8a8_pack_weight (same arithmetic, same results). */
w8a8_status w8a8_linear(const uint16_t* x, const int8_t* w, const float* s_ch, const uint16_t* bias,
                        uint16_t* y, int64_t M, int64_t N, int64_t K, int rot_block,
                        void* workspace, size_t workspace_bytes, hipStream_t stream);

w8a8_status w8a8_gateup_swiglu(const uint16_t* x, const int8_t* w_gateup, const float* s_ch,
                               const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K,
                               int rot_block, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

w8a8_status w8a8_fp8_linear(const uint16_t* x, const uint8_t* w, const float* s_ch,
                            const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K,
                            int rot_block, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

w8a8_status w8a8_linear_packed(const uint16_t* x, const int8_t* w_packed, const float* s_ch,
                               const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K,
                               int rot_block, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

w8a8_status w8a8_gateup_swiglu_packed(const uint16_t* x, const int8_t* w_gateup_packed,
                                      const float* s_ch, const uint16_t* bias, uint16_t* y, int64_t M,
                                      int64_t N, int64_t K, int rot_block, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

w8a8_status w8a8_fp8_linear_packed(const uint16_t* x, const uint8_t* w_packed, const float* s_ch,
                                   const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K,
                                   int rot_block, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* ---- the int8 whole path without a workspace ---------------------------------
 * For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): w8a8_linear_packed with
 * its workspace -- the packed activation codes and their scales -- taken from a
 * fixed device array inside the library instead of the caller.  Same kernels,
 * same arguments otherwise, same results byte for byte.  The array holds
 * W8A8_NOALLOC_MAX_WORKSPACE bytes on each device the library runs on, kept until
 * the process ends; a call whose w8a8_workspace_bytes(M, K) exceeds it returns
 * W8A8_ERR_SCRATCH_TOO_SMALL (checked after the shapes, before anything else)
 * and enqueues nothing.  This entry point allocates nothing (no hipMalloc, no
 * library allocation).  Every call on one device shares that device's array:
 * calls that overlap in time on one device (e.g. on two streams) race and give
 * undefined results; calls ordered on one stream are safe.  The array keeps the
 * last call's codes and scales; nothing in it needs clearing between calls. */
#define W8A8_NOALLOC_MAX_WORKSPACE (64u << 20)

w8a8_status w8a8_linear_packed_noalloc(const uint16_t* x, const int8_t* w_packed, const float* s_ch,
                                       const uint16_t* bias, uint16_t* y, int64_t M, int64_t N,
                                       int64_t K, int rot_block, hipStream_t stream);

/* ---- gate/up SwiGLU whose output is quantized for the next linear -----------
 * The down projection that follows the gate/up pair is an INT8 projection too,
 * so its input -- the SwiGLU output h [M, N] -- goes through the same per-token
 * activation quantizer as every INT8 projection's input (INT8 ConvRot card,
 * notes under the latency table), after the paired gate/up epilogue ("Loading
 * CLEF INT8", fuse_mlp):
 *   h = bf16(silu(g) * u)                    as w8a8_gateup_swiglu_packed;
 *   q_packed, s_tok = w8a8_quantize_act_packed(h, rot_out)   bit for bit.
 * Three kernels on `stream`: the quantizer of x (rotation rot_in), the gate/up
 * GEMM with the SwiGLU epilogue writing h into the workspace, the quantizer of
 * h.  The codes are w8a8_packed_bytes(M, N) bytes in the packed layout of a
 * [M, N] activation (padding rows untouched): the A operand of
 * w8a8_gemm_dequant_packed for the down projection (its K = N); s_tok is [M].
 * Shapes: the gate/up GEMM's (K % 128 == 0) and N % 64 == 0, N <= W8A8_MAX_K;
 * rot_out == 128 needs N % 128 == 0; rot_in and rot_out are 0 or 128
 * (W8A8_ERR_BAD_ARGUMENT otherwise). */

/* Workspace of w8a8_gateup_swiglu_quant_packed: w8a8_workspace_bytes(M, K)
 * (the codes and scales of x) followed by h, bf16 [M, N], on a 256-byte
 * boundary.  Afterwards it holds those values.  0 for M, N or K <= 0. */
size_t w8a8_swiglu_quant_workspace_bytes(int64_t M, int64_t N, int64_t K);

w8a8_status w8a8_gateup_swiglu_quant_packed(const uint16_t* x, const int8_t* w_gateup_packed,
                                            const float* s_ch, const uint16_t* bias, int64_t M,
                                            int64_t N, int64_t K, int rot_in, int rot_out,
                                            int8_t* q_packed, float* s_tok, void* workspace,
                                            size_t workspace_bytes, hipStream_t stream);

/* ---- few tokens: projections with 4-bit weights ---------------------------------
 * Single-token and small-batch decoding reads every weight for a handful of
 * tokens, so the weight bytes are the time.  Here a weight is a code in [-8, 7]
 * and each group of `group` consecutive columns (32, 64 or 128) of a row shares
 * one bf16 scale: w[n][k] = code * scale.  Row-major form:
 *   codes   uint8 [N, K / 2]: two codes a byte, the even column in the low half,
 *           each stored as code + 8
 *   scales  bf16 [N, K / group]
 * Shapes: 0 <= N <= 2^30, K % 128 == 0, 128 <= K <= W8A8_MAX_K; `group` other than
 * 32, 64 or 128 is W8A8_ERR_BAD_ARGUMENT. */

/* Rows of w bf16 [N, K] -> codes and scales: scale = bf16(amax / 7) of the group,
 * code = round-half-even(w / scale) clamped to +-7 (-8 is never produced); a group
 * of zeros has scale 0 and codes 0. */
w8a8_status w8a8_w4_quantize(const uint16_t* w, int64_t N, int64_t K, int group, uint8_t* codes,
                             uint16_t* scales, hipStream_t stream);

/* Packed form, rows rounded up to 16 (padding: codes 0, scales 0): blocks of 16
 * rows x 128 columns, block (n / 16, k / 128) at byte
 * ((n / 16) * (K / 128) + k / 128) * 1024.  Row r and column c of a block are in the
 * 32-bit word at byte (16 * (c / 8 % 4) + r) * 16 + 4 * (c / 32): element j = c % 8
 * at bit 4 * (j / 2) + 16 * (j % 2).  Scales: [N / 16][K / group][16].
 * w8a8_w4_pack lays a weight out once, at load time. */
size_t w8a8_w4_code_bytes(int64_t N, int64_t K);              /* 0 outside the limits */
size_t w8a8_w4_scale_bytes(int64_t N, int64_t K, int group);  /* 0 also for a bad group */
w8a8_status w8a8_w4_pack(const uint8_t* codes, const uint16_t* scales, int64_t N, int64_t K, int group,
                         uint8_t* codes_packed, uint16_t* scales_packed, hipStream_t stream);

/* y[m][n] = bf16( sum over groups of scale * sum(x * code) + bias[n] ), fp32 sums,
 * one rounding.  x bf16 [M, K], bias bf16 [N] or NULL, y bf16 [M, N].  N % 8 == 0,
 * N <= W8A8_W4_MAX_N, 0 <= M <= W8A8_W4_MAX_M, M * N <= 2^40.  Made for M up to 64; larger M is computed in blocks of
 * 32 or 64 tokens, each of which passes over the weight again.  A token's
 * result does not depend on the others in the call, nor on their number.  x is taken
 * as finite, with 144 * sum|x| over a group inside fp32 (the sums run over codes with
 * an offset that is taken out again); a token that is not spoils its own row only.  So a
 * group's rounding is that of sums up to 144 * sum|x|, about 2^-17 * sum|x| * scale, also
 * of elements whose codes are 0.  The
 * workspace holds fp32 partial sums where K is long and N small, so that K is cut,
 * of up to 1,024 tokens at a time; w8a8_w4_workspace_bytes is 0, and workspace may be
 * NULL, where it is not. */
#define W8A8_W4_MAX_M (1 << 20)
#define W8A8_W4_MAX_N ((1 << 28) - 32)
size_t w8a8_w4_workspace_bytes(int64_t M, int64_t N, int64_t K);
w8a8_status w8a8_w4_linear(const uint16_t* x, const uint8_t* codes_packed, const uint16_t* scales_packed,
                           const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, int group,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- few tokens: a paged cache of keys and values in 8 bits ---------------------
 * Pages of `page` tokens (16, 32, 64 or 128) for `heads` cache heads of `dim` values
 * (64 or 128):
 *   k_codes, v_codes  int8 [pages, heads, page, dim]
 *   k_scale, v_scale  fp32 [pages, heads]: value = code * scale of its page and head
 *   table             int32 [seqs, width]: the page of each block of a sequence
 *   lens              int32 [seqs]: tokens a sequence holds, those of the newest
 *                     append included
 * Token p of a sequence is row p % page of page table[p / page].  A negative
 * length counts as 0.  Positions follow the lengths as given, also past
 * width * page, where the table ends: new tokens there are dropped, queries
 * there see the keys that the table names.  Table entries
 * outside [0, pages) name no page: append drops the tokens that fall there, read
 * gives zeros, attention sees no keys there.  Which pages are whose is the
 * caller's: sequences may share pages that are only read, but two sequences of one
 * append must not write to the same page.
 * Limits: seqs <= W8A8_KV_MAX_SEQS, heads and q_heads <= W8A8_KV_MAX_HEADS, tokens <=
 * W8A8_KV_MAX_TOKENS, width * page <= W8A8_KV_MAX_LENGTH, pages < 2^31. */
#define W8A8_KV_MAX_SEQS (1 << 20)
#define W8A8_KV_MAX_HEADS 1024
#define W8A8_KV_MAX_TOKENS (1 << 20)
#define W8A8_KV_MAX_LENGTH (1 << 30)

/* The last `tokens` tokens of every sequence, rows k and v [seqs * tokens] of
 * [heads, dim] bf16 values, rows ldk and ldv elements apart (>= heads * dim, a
 * multiple of 8: slices of a wider projection), go to positions lens - tokens ..
 * lens - 1; those at negative positions are dropped.  For each page and head that
 * receives some: scale = max(old scale if the page holds earlier tokens of the
 * sequence, amax / 127 of the new values), held codes become
 * round-half-even(code * (old / new scale)), new ones round-half-even(x / scale).
 * A scale of a page that holds nothing from before is not read: a cache needs no
 * initialisation.  Values are taken as finite: a NaN or an infinity spoils the
 * codes of its page and head (of no other; attention of queries that see none of
 * that page is as without it).
 * (tokens / page + 2) * heads < 2^23, and that times seqs < 2^30.
 * Filling a page in one call rounds each value once; token by token, a page's
 * earlier codes are rounded again whenever a larger value arrives (each time by
 * at most half a step of the new scale). */
w8a8_status w8a8_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, int8_t* k_codes,
                           float* k_scale, int8_t* v_codes, float* v_scale, int64_t pages, const int32_t* table,
                           int64_t width, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t heads,
                           int64_t dim, int64_t page, hipStream_t stream);

/* The sequences as bf16: k, v [seqs, length, heads, dim] = bf16(code * scale), zeros
 * from a sequence's length on.  length * dim <= 2^35 - 2048, seqs * length * heads * dim < 2^42. */
w8a8_status w8a8_kv_read(const int8_t* k_codes, const float* k_scale, const int8_t* v_codes, const float* v_scale,
                         int64_t pages, const int32_t* table, int64_t width, const int32_t* lens, int64_t seqs,
                         int64_t length, int64_t heads, int64_t dim, int64_t page, uint16_t* k, uint16_t* v,
                         hipStream_t stream);

/* Attention of the last `tokens` tokens of every sequence over what it holds:
 * query i is at position p = lens - tokens + i and sees keys 0 .. p,
 *   y = sum_j exp(scale * q.k_j - max) v_j / sum_j exp(scale * q.k_j - max);
 * a query that sees no key (p < 0, an empty sequence) gives zeros.  Scales are not
 * negative, as append makes them; values of a page whose scale is below 2^-90 count
 * as zeros.  What lies in pages or rows that a sequence does not hold is not
 * used, NaN included.  q: rows
 * [seqs * tokens] of [q_heads, dim] bf16, ldq elements apart (>= q_heads * dim, a
 * multiple of 8); q_heads % heads == 0, query head a reads cache head
 * a / (q_heads / heads).  y bf16 [seqs, tokens, q_heads, dim], dense.  scale is
 * finite (usually dim^-0.5; W8A8_ERR_BAD_ARGUMENT otherwise).
 * Sequences are cut into pieces when there are too few queries to fill the GPU;
 * the pieces' partial results go through the workspace
 * (w8a8_kv_attention_workspace_bytes, which may be 0: then it may be NULL; 0 also
 * for arguments that the call refuses).  The cut depends on the shapes, not on
 * lens' values, and results do not vary from run to run. */
size_t w8a8_kv_attention_workspace_bytes(int64_t seqs, int64_t tokens, int64_t q_heads, int64_t heads, int64_t dim,
                                         int64_t page, int64_t width);
w8a8_status w8a8_kv_attention(const uint16_t* q, int64_t ldq, const int8_t* k_codes, const float* k_scale,
                              const int8_t* v_codes, const float* v_scale, int64_t pages, const int32_t* table,
                              int64_t width, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t q_heads,
                              int64_t heads, int64_t dim, int64_t page, float scale, uint16_t* y, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/* ---- around the projections: root-mean-square norm, after the residual's addition ----
 * For rows x [M, K] bf16, residual bf16 [M, K] or NULL, weight bf16 [K]:
 *   h = bf16(x + residual) (fp32 sum; h = x without a residual)
 *   z = h * weight,  r = 1 / sqrt(mean(h^2) + eps),  y = z * r
 * with fp32 sums.  `h`, if not NULL, receives h [M, K] (what the next addition takes); it may be the
 * residual's buffer or x's (in place).  Outputs:
 *   w8a8_rmsnorm               y bf16 [M, K]; it may be x's buffer
 *   ..._quantize               int8 codes, s_tok fp32 [M] = amax|y| / 127
 *   ..._quantize_fp8           E4M3FN codes, s_tok fp32 [M] = amax|y| / 448
 *   ..._quantize_block         E4M3FN codes, a scale for each 128 columns, amax|y| / 448 of those
 * The codes are those of w8a8_quantize_act* for the values z, which are common multiples of y: y is not
 * rounded to bf16 on the way.  rot_block == 128: codes of y turned by the normalized transform in blocks of
 * 128, in fp32.  Row-major codes are [M, K], their block scales [M, K / 128]; the _packed forms write the
 * packed layout (padding rows untouched), with block scales [K / 128][w8a8_block_scale_stride(M)].
 * A row of zeros gives zeros.  A row with a NaN or an infinity, or whose sum of h^2 leaves fp32's range
 * (one |h| of 2^64, or all of 2^64 / sqrt(K)), spoils its own row only.  A weight that is not finite spoils its
 * column of y in bf16, and every scale over that column, in all rows.
 * 1 <= K <= W8A8_MAX_K, K % 8 == 0 (codes: K % 32 == 0; packed: K % 64 == 0; rot_block or block scales:
 * K % 128 == 0); eps finite and positive (W8A8_ERR_BAD_ARGUMENT otherwise). */
w8a8_status w8a8_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps, uint16_t* h,
                         uint16_t* y, int64_t M, int64_t K, hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                  int rot_block, uint16_t* h, int8_t* q, float* s_tok, int64_t M, int64_t K,
                                  hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                         int rot_block, uint16_t* h, int8_t* q_packed, float* s_tok, int64_t M,
                                         int64_t K, hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                      int rot_block, uint16_t* h, uint8_t* q, float* s_tok, int64_t M, int64_t K,
                                      hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize_fp8_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                                             float eps, int rot_block, uint16_t* h, uint8_t* q_packed, float* s_tok,
                                             int64_t M, int64_t K, hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize_block(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, float eps,
                                        uint16_t* h, uint8_t* q, float* s, int64_t M, int64_t K, hipStream_t stream);
w8a8_status w8a8_rmsnorm_quantize_block_packed(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                                               float eps, uint16_t* h, uint8_t* q_packed, float* s, int64_t M,
                                               int64_t K, hipStream_t stream);

/* ---- around the attention: rotary positions of queries and keys ------------------
 * q rows [seqs * tokens] of [q_heads, dim] and k rows of [heads, dim], bf16, ldq and ldk elements apart
 * (>= heads * dim, a multiple of 8: slices of one projection), as w8a8_kv_append and w8a8_kv_attention take
 * them; row i of a sequence is at position p = lens - tokens + i (a negative length counts as 0).  The
 * first `rotary` values of each head are turned in pairs, (i, i + rotary / 2) or, with `interleaved`,
 * (2i, 2i + 1):
 *   (a, b) -> amplitude * (a cos t - b sin t, b cos t + a sin t),  t = p * f_i,
 * in fp32, rounded once; the rest of the head, and rows at p < 0, are copied.  turns[i] is
 * round(2^64 * f_i / (2 pi)) mod 2^64: frequencies as fractions of a turn, so that angles keep 2^-32 of a turn at
 * every position (f_i's own error, times p, comes on top).  q_out and k_out: rows of their own strides, or q and k
 * themselves (in place: same pointer and stride).  heads may be 0 (queries alone; k and k_out are not read then).
 * dim % 16 == 0, 16 <= dim <= 256; rotary % 16 == 0, 16 <= rotary <= dim; q_heads and heads up to
 * W8A8_KV_MAX_HEADS, q_heads >= 1; seqs and tokens as for the cache, seqs * tokens < 2^31; amplitude finite. */
w8a8_status w8a8_rope(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk, const uint64_t* turns, int64_t rotary,
                      int interleaved, float amplitude, const int32_t* lens, int64_t seqs, int64_t tokens, int64_t q_heads,
                      int64_t heads, int64_t dim, uint16_t* q_out, int64_t ldq_out, uint16_t* k_out, int64_t ldk_out,
                      hipStream_t stream);

/* ---- E4M3 projections with block scales ------------------------------------------
 * Codes E4M3FN; an activation's value is code * s of its token and 128 columns, a weight's code * s of its block of
 * 128 x 128 (rows past N are not counted).  scale = amax / 448 (fp32 IEEE division), code as w8a8_quantize_act_fp8's;
 * a block of zeros has scale 0 and codes 0.  A block with a NaN has a NaN for its scale (codes 0), one with an infinity an
 * infinite scale: a token with either gives no finite output (a NaN: NaNs only), and neither does a weight's block for the
 * rows that it belongs to; other tokens' and rows' outputs are what they are without it. */

/* Row stride of the scales that go with packed codes of M rows: M rounded up to a multiple of 32 (0 outside 1 .. 2^42). */
int64_t w8a8_block_scale_stride(int64_t M);

/* x bf16 [M, K] -> codes [M, K], s fp32 [M, K / 128]; packed: s [K / 128][w8a8_block_scale_stride(M)] (padding
 * untouched in both).  K % 128 == 0, M * K <= 2^42. */
w8a8_status w8a8_quantize_act_block(const uint16_t* x, int64_t M, int64_t K, uint8_t* q, float* s, hipStream_t stream);
w8a8_status w8a8_quantize_act_block_packed(const uint16_t* x, int64_t M, int64_t K, uint8_t* q_packed, float* s,
                                           hipStream_t stream);
/* w bf16 [N, K] -> codes [N, K] (lay them out with w8a8_pack_weight), s fp32 [ceil(N / 128), K / 128]. */
w8a8_status w8a8_quantize_weight_block(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* s, hipStream_t stream);

/* y[m][n] = bf16( sum_b s[b][m] * s_w[n / 128][b] * sum_{k in b} q[m][k] * w[n][k] + bias[n] ).  The inner sums run on
 * the E4M3 matrix instructions, which drop what lies 2^-13 below the largest of a group of their products (1.4e-5 of
 * the output's rms on normal values, 4e-5 with outliers of 20 times); the sum over blocks is fp32, rounded once
 * (and so is s * s_w, each block's factor).
 * Which form multiplies, and with it the order of the sum over blocks, depends on M, N and K.
 * M * N <= 2^40, N <= 2^28 - 32, M <= 2^30; scales that are not finite as above.  The workspace holds fp32
 * partial sums where the shape is short of tiles, so that K is cut; its size is 0, and workspace may be NULL, where it is not. */
size_t w8a8_fp8_block_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);   /* 0 also outside the limits */
w8a8_status w8a8_fp8_block_gemm_packed(const uint8_t* q_packed, const float* s, const uint8_t* w_packed, const float* s_w,
                                       const uint16_t* bias, uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream);

/* x is quantized into the workspace (packed codes and scales; a short call may leave it unused), then multiplied. M * K <= 2^42. */
size_t w8a8_fp8_block_workspace_bytes(int64_t M, int64_t N, int64_t K);        /* 0 for M <= 0 and outside the limits */
w8a8_status w8a8_fp8_block_linear_packed(const uint16_t* x, const uint8_t* w_packed, const float* s_w, const uint16_t* bias,
                                         uint16_t* y, int64_t M, int64_t N, int64_t K, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W8A8_H */
