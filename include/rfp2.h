/*
 * rfp2.h -- C ABI of the ROCmFP2 GEMV / GEMM library for AMD Instinct MI355X
 * (gfx950).
 *
 * The format and the method follow the page "ROCmFP2 codebook research
 * report" (llm.ciru.ai, 2026-07-13):
 *
 *   "01 · Storage": a block stores 32 weights in 10 bytes.  Bytes 0..7 are
 *     code bytes; byte j holds weights 4j..4j+3, weight 4j+i in bits
 *     2i..2i+1.  Byte 8 is the UE4M3 scale of weights 0..15, byte 9 the
 *     scale of weights 16..31.  2.50 bits per weight.
 *   "02 · Quantization": codes 00,01,10,11 mean -4,-1,+1,+4 times the scale
 *     of their half.  A scale byte b (legal 0x00..0x7E) has E = b >> 3,
 *     M = b & 7 and value M * 2^-10 (E == 0) or (8 + M) * 2^(E - 11).
 *     The quantizer starts near max|x|/4, tries legal scales, maps all 16
 *     values of the half to the nearest level (inner when |x/s| <= 2.5) and
 *     keeps the scale with the least squared error.
 *   "03 · Runtime": each code byte becomes four signed int8 lanes, which are
 *     multiplied four at a time with int8 (Q8_1-style) activations and
 *     accumulated in int32 per 16-weight half; the two weight scales and the
 *     activation scale are applied after the integer sum,
 *     d_a * (d_0 * S_0 + d_1 * S_1).  The multi-column kernel expands a
 *     block once and reuses it for every activation column.
 *
 * Conventions shared by every entry point:
 *   - Every data pointer is a DEVICE pointer owned by the caller (the library
 *     allocates nothing, frees nothing and keeps no state between calls
 *     beyond a per-device cache of the GPU's compute-unit count).
 *   - Inputs are never written.  Outputs are overwritten, not accumulated.
 *   - Every call only enqueues work on `stream` (0 = the null stream) and
 *     returns; nothing is synchronised.  Calls are thread-safe.
 *   - Matrices are row-major.  A stored weight matrix of N rows and K columns
 *     is N rows of K/32 blocks, back to back: N * K / 32 * 10 bytes, row n at
 *     byte n * K * 10 / 32.
 *   - Activations are q int8 [M][K] plus d fp32 [M][K/32]: column (token) m
 *     of the product uses q[m][k] * d[m][k/32].
 *   - Argument errors are checked on the host before anything is enqueued;
 *     the call then returns a negative status and launches nothing.
 *   - Data errors are loud on the device: a scale byte outside 0x00..0x7E
 *     makes every output that depends on it NaN.
 */
#ifndef RFP2_H
#define RFP2_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum rfp2_status {
  RFP2_OK = 0,
  RFP2_E_NULL = -1,   /* a required pointer is null                        */
  RFP2_E_SHAPE = -2,  /* a size is out of range (see each call)            */
  RFP2_E_ALIGN = -3,  /* a pointer is not aligned as the call requires     */
  RFP2_E_LAUNCH = -4  /* the HIP runtime reported an error for the launch  */
} rfp2_status;

#define RFP2_ABI_VERSION 1
#define RFP2_GEMV_MAX_M 8

/* ABI version of the loaded library (RFP2_ABI_VERSION). */
int rfp2_abi_version(void);

/* Static English text for a status code; never NULL. */
const char* rfp2_status_string(int status);

/*
 * rfp2_quantize_acts -- int8 activations, one fp32 scale per 32 values
 * ("03 · Runtime": the int8 activation operand and its scale).
 *   a  [M][K] fp32, 16-byte aligned.   q [M][K] int8, 4-byte aligned.
 *   d  [M][K/32] fp32, 4-byte aligned.
 * Per 32-value block: amax = max|a|, d = amax / 127 (IEEE fp32 division,
 * round to nearest even), q = round(a / d) with halves away from zero,
 * clamped to [-127, 127]; d == 0 gives q = 0.  A block holding a NaN or an
 * infinity gets d = NaN and q = 0.
 * Requires M >= 1, K >= 32, K % 32 == 0.
 */
rfp2_status rfp2_quantize_acts(const float* a, int64_t M, int64_t K,
                               int8_t* q, float* d, hipStream_t stream);

/*
 * rfp2_quantize_weights -- pack fp32 weights into ROCmFP2 blocks
 * ("02 · Quantization": how a block is chosen).
 *   x [N][K] fp32, 4-byte aligned.  w [N * K/32 * 10] bytes, 2-byte aligned.
 * Each 16-weight half gets the legal scale byte with the least squared
 * reconstruction error over all 127 legal bytes (errors summed in fp64 in
 * index order); on an exact tie the byte nearest to the start byte (the one
 * whose scale is nearest max|x|/4, the lower on a tie) wins, the lower one
 * first.  Codes: x < 0 negative, else positive; |x| <= 2.5 * s inner.
 * Non-finite weights give unspecified bytes.
 * Requires N >= 1, K >= 32, K % 32 == 0.
 */
rfp2_status rfp2_quantize_weights(const float* x, int64_t N, int64_t K,
                                  uint8_t* w, hipStream_t stream);

/*
 * rfp2_quantize_weights_imatrix -- rfp2_quantize_weights with the
 * importance-weighted error of "05 · Completed experiment": a candidate
 * scale's error is sum_i imp_i * sqrt(sigma^2 + x_i^2) * (x_i - xhat_i)^2
 * over the half, where imp_i is the importance of the value's input channel
 * and sigma^2 is the mean of x^2 over the half (the page leaves sigma
 * undefined; this is the reading taken).  Weights and errors are fp64, one
 * rounding per step, so the choice is reproducible.  The block layout,
 * codebook and codes are unchanged; only which scale wins can differ.
 *   importance [K] fp32, 4-byte aligned, finite and >= 0 (other values give
 *   unspecified bytes).  x, w and the limits as rfp2_quantize_weights.
 */
rfp2_status rfp2_quantize_weights_imatrix(const float* x, int64_t N, int64_t K,
                                          const float* importance, uint8_t* w,
                                          hipStream_t stream);

/*
 * rfp2_gemv -- y[m][n] = sum_k w[n][k] * q[m][k] * d[m][k/32] for a few
 * activation columns ("03 · Runtime": decode once, reuse for every column).
 *   w [N][K/32][10] bytes, 16-byte aligned.  q [M][K] int8, 16-byte aligned.
 *   d [M][K/32] fp32, 4-byte aligned.         y [M][N] fp32, 4-byte aligned.
 * Requires N >= 1, 1 <= M <= RFP2_GEMV_MAX_M, 256 <= K <= 32768,
 * K % 256 == 0 (a row is then a whole number of 80-byte groups and every row
 * starts 16-byte aligned).
 */
rfp2_status rfp2_gemv(const uint8_t* w, int64_t N, int64_t K,
                      const int8_t* q, const float* d, int64_t M,
                      float* y, hipStream_t stream);

/*
 * rfp2_gemm -- the same product for a batch of M >= 1 activation columns
 * (prompt batches), computed with i8 matrix-core instructions on int32
 * integer sums ("03 · Runtime" applied to a tile of columns).  The UE4M3
 * mantissas of a block's two scales are folded into its int8 weights, so
 * the block is one integer dot product with one power-of-two scale while
 * the two scale exponents differ by at most 2 (as int32 per-half partials
 * otherwise); every such scaled sum is exact and the activation scale is
 * applied to it with one rounding, then added with one more.
 * Layouts and alignment as rfp2_gemv.  Requires N >= 1, M >= 1,
 * 256 <= K <= 2^24, K % 256 == 0.
 */
rfp2_status rfp2_gemm(const uint8_t* w, int64_t N, int64_t K,
                      const int8_t* q, const float* d, int64_t M,
                      float* y, hipStream_t stream);

/*
 * rfp2_gemm_f16 -- the same product as rfp2_gemm, computed on the fp16
 * matrix cores.  Every reconstructed weight (level x UE4M3 scale) and every
 * int8 activation is exactly an fp16 number and every product is exact in
 * fp32, so each 32-weight block's sum s0*S0 + s1*S1 comes out of the matrix
 * core in fp32 (exact while the two scale exponents differ by at most 7;
 * beyond, the core's fp32 accumulation may round, each step within 2^-24 of
 * the running sum) and only the activation scale is applied afterwards: one
 * multiply-add per output and block instead of the int32 path's two.
 * Layouts, alignment and limits as rfp2_gemm.
 */
rfp2_status rfp2_gemm_f16(const uint8_t* w, int64_t N, int64_t K,
                          const int8_t* q, const float* d, int64_t M,
                          float* y, hipStream_t stream);

/*
 * rfp2_moe_gemv -- routed-expert GEMV for one token.
 *   w    E experts back to back, each [N][K/32][10] bytes; 16-byte aligned.
 *   ids  [top_k] int32 on the device: the experts to apply, in output order.
 *   q, d one activation column ([K] int8, [K/32] fp32).
 *   y    [top_k][N] fp32: row j = expert ids[j] applied to the token.
 *   err  nullable device int32: when an id lies outside [0, E) its row of y
 *        is set to NaN and 1 is written to *err (never cleared by the call).
 * Duplicate ids are legal.  Expert offsets are computed in 64 bits.
 * Requires E >= 1, N >= 1, 1 <= top_k <= 65535, 256 <= K <= 32768,
 * K % 256 == 0.
 */
rfp2_status rfp2_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                          const int32_t* ids, int64_t top_k,
                          const int8_t* q, const float* d,
                          float* y, int32_t* err, hipStream_t stream);

/*
 * rfp2_moe_gemv_tokens -- routed-expert GEMV for T tokens at once (e.g. the
 * tokens of a speculative-decoding verification batch).  Slot s = t * top_k
 * + j of token t is routed to expert ids[s]; the slots routed to one expert
 * are computed together, so each expert's rows are expanded once and reused
 * for every token routed to it ("Why AMD-friendly does not mean always
 * faster": expand a block once, reuse it across all activation columns).
 *   w    E experts back to back, each [N][K/32][10] bytes; 16-byte aligned.
 *   ids  [T][top_k] int32 on the device.
 *   q, d [T][K] int8 (16-byte aligned) and [T][K/32] fp32.
 *   y    [T][top_k][N] fp32: row s = expert ids[s] applied to token s / top_k.
 *   err  as rfp2_moe_gemv (an id outside [0, E) gives a NaN row and *err = 1).
 * Duplicate ids are legal.  T = 1 is rfp2_moe_gemv.  Each row of y is within
 * the fp32 bound of the product, but the order of its additions may differ
 * from rfp2_moe_gemv's for the same token.
 * Requires E >= 1, N >= 1, 1 <= T <= RFP2_GEMV_MAX_M, top_k >= 1,
 * T * top_k <= 64, 256 <= K <= 32768, K % 256 == 0.
 */
rfp2_status rfp2_moe_gemv_tokens(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                 const int32_t* ids, int64_t T, int64_t top_k,
                                 const int8_t* q, const float* d, float* y, int32_t* err,
                                 hipStream_t stream);

/*
 * rfp2_moe_sort -- the routed slots grouped by expert, the token order of a
 * prompt batch through the routed experts ("04 · Measured evidence" and
 * "07 · Recipe decision": the method's gain is prefill on large expert
 * tensors; a prefill product takes each expert's tokens together).
 *   ids     [S] int32 on the device: slot s (token s / top_k of a batch) is
 *           routed to expert ids[s].
 *   offsets [E+1] int32 (written): expert e's slots are
 *           order[offsets[e] .. offsets[e+1]); offsets[E] = the routed slots.
 *   order   [S] int32 (written up to offsets[E]): every slot whose id lies in
 *           [0, E), grouped by expert in expert order, increasing slot order
 *           inside an expert (the stable order: deterministic).
 *   err     nullable device int32: set to 1 when an id lies outside [0, E)
 *           (such slots are left out; never cleared by the call).
 * One workgroup; suited to the few thousand slots of a prompt batch.
 * Requires 1 <= S <= 2^24, 1 <= E <= 2048; all pointers 4-byte aligned.
 */
rfp2_status rfp2_moe_sort(const int32_t* ids, int64_t S, int64_t E, int32_t* offsets,
                          int32_t* order, int32_t* err, hipStream_t stream);

/*
 * rfp2_moe_gemm_workspace_bytes -- device bytes rfp2_moe_gemm needs as
 * workspace for E experts and T * top_k slots (0 when the sizes are out of
 * range).
 */
size_t rfp2_moe_gemm_workspace_bytes(int64_t E, int64_t T, int64_t top_k);

/*
 * rfp2_moe_gemm -- routed-expert products for a prompt batch of T tokens on
 * the matrix cores: the slots are sorted by expert (rfp2_moe_sort), then each
 * expert's slots are cut into tiles of 64 tokens and multiplied with that
 * expert's weights as rfp2_gemm_f16 multiplies a dense batch (exact fp16
 * operands, one rescale per output and block).
 *   w    E experts back to back, each [N][K/32][10] bytes; 16-byte aligned.
 *   ids  [T][top_k] int32 on the device; slot s = t * top_k + j.
 *   q, d [T][K] int8 (16-byte aligned) and [T][K/32] fp32.
 *   y    [T][top_k][N] fp32: row s = expert ids[s] applied to token s / top_k
 *        (NaN for an id outside [0, E), and *err = 1 as rfp2_moe_gemv).
 *   workspace  device memory of at least rfp2_moe_gemm_workspace_bytes(E, T,
 *        top_k) bytes, 256-byte aligned, owned by the caller; overwritten.
 *        Calls that share a workspace must not overlap in time.
 * Each output is computed independently of which other slots share its
 * tile, so y does not depend on the routing of the other tokens.
 * Requires 1 <= E <= 2048, N >= 1, T >= 1, top_k >= 1, T * top_k <= 2^24,
 * 256 <= K <= 2^24, K % 256 == 0.
 */
rfp2_status rfp2_moe_gemm(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                          const int32_t* ids, int64_t T, int64_t top_k, const int8_t* q,
                          const float* d, float* y, int32_t* err, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/*
 * rfp2_moe_gemm_noalloc -- rfp2_moe_gemm for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): the same sort and product kernels and the same
 * result, with the sorted slots kept in a device array that the library owns
 * instead of a caller workspace.  The call allocates nothing.
 *   w, ids, q, d, y, err and their layouts, alignment and limits as
 *   rfp2_moe_gemm; in addition rfp2_moe_gemm_workspace_bytes(E, T, top_k)
 *   must not exceed RFP2_MOE_GEMM_NOALLOC_MAX_BYTES (otherwise RFP2_E_SHAPE,
 *   nothing launched).  With 128 experts that allows up to 261,886 routed
 *   slots, e.g. 32,735 tokens at top-8.
 * The array (RFP2_MOE_GEMM_NOALLOC_MAX_BYTES bytes) is held by every GPU the
 * library runs on until the process ends; its device address is looked up on
 * the first call on each device (RFP2_E_LAUNCH if that fails).  All calls on
 * one GPU share it and it keeps the last call's contents: calls that overlap
 * in time on one GPU (several streams, several host threads) race and must be
 * serialised by the caller.
 */
#define RFP2_MOE_GEMM_NOALLOC_MAX_BYTES 1048576
rfp2_status rfp2_moe_gemm_noalloc(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                  const int32_t* ids, int64_t T, int64_t top_k,
                                  const int8_t* q, const float* d, float* y, int32_t* err,
                                  hipStream_t stream);

/*
 * rfp2_quant_gemv -- one token end to end: quantizes the fp32 activations a
 * exactly as rfp2_quantize_acts does, writing q and d, and computes
 * y = W * a as rfp2_gemv does from that q and d ("03 · Runtime": the int8
 * activation operand, its scale, then the product), in a single kernel
 * launch for most K and up to 128 MiB of weights (beyond, the two launches
 * are faster): each wave quantizes the activations it needs while its
 * weights stream in.  q and d are bit-identical to rfp2_quantize_acts.  y is
 * bit-identical to rfp2_gemv with M = 1 on them wherever the single launch
 * splits K as rfp2_gemv does; where rfp2_gemv's split gives a wave more than
 * 4 groups of 256 (K = 6144, 8192, 10240, 12288, 14336, 16384) and the call
 * reads at most 64 MiB, the single launch may split K over more waves or
 * more rows per workgroup, and y then sums in another order (same fp32
 * bound).
 *   w [N][K/32][10] bytes, 16-byte aligned.   a [K] fp32, 16-byte aligned.
 *   q [K] int8, 16-byte aligned (written).     d [K/32] fp32, 4-byte aligned
 *   (written).                                 y [N] fp32, 4-byte aligned.
 * Requires N >= 1, 256 <= K <= 32768, K % 256 == 0.
 */
rfp2_status rfp2_quant_gemv(const uint8_t* w, int64_t N, int64_t K, const float* a,
                            int8_t* q, float* d, float* y, hipStream_t stream);

/*
 * rfp2_quant_moe_gemv -- the routed-expert GEMV of rfp2_moe_gemv for one
 * token given in fp32, with the activation quantization of
 * rfp2_quantize_acts done inside the product launch (as rfp2_quant_gemv).
 * w, ids, y, err and the limits as rfp2_moe_gemv; a, q, d as
 * rfp2_quant_gemv.  q and d are bit-identical to rfp2_quantize_acts, and y
 * to rfp2_moe_gemv on them, with the same exception as rfp2_quant_gemv.
 */
rfp2_status rfp2_quant_moe_gemv(const uint8_t* w, int64_t E, int64_t N, int64_t K,
                                const int32_t* ids, int64_t top_k, const float* a,
                                int8_t* q, float* d, float* y, int32_t* err,
                                hipStream_t stream);

/*
 * Rotary positions, a paged key/value cache and the attention over it: what a
 * decode step does between its weight products.  The products' fp32 rows go
 * in, the attention's fp32 rows come out and feed rfp2_quant_gemv or
 * rfp2_quantize_acts.
 *
 * rfp2_rope_freqs -- the angle per position of each pair of a rotary
 * embedding, written to freqs [rot/2] (device fp64, 8-byte aligned):
 *   f_i = base^(-2i / rot), i = 0 .. rot/2 - 1, stretched for contexts longer
 *   than the model was made for:
 *   orig_len == 0   every f_i is divided by factor (linear interpolation);
 *   orig_len > 0    by parts: with r_i = orig_len * f_i / (2 pi) turns over
 *     the original length and g_i = clamp((r_i - low_turns) / (high_turns -
 *     low_turns), 0, 1), the result is (1 - g_i) * f_i / factor + g_i * f_i
 *     (slow pairs are interpolated, fast pairs are kept).
 *   factor == 1 leaves f_i as it is in either form.
 * Requires 2 <= rot <= 1024, rot even, base > 1, factor >= 1, orig_len >= 0,
 * and 0 <= low_turns < high_turns where orig_len > 0; all finite.
 */
rfp2_status rfp2_rope_freqs(int64_t rot, double base, double factor, double orig_len,
                            double low_turns, double high_turns, double* freqs,
                            hipStream_t stream);

/* Which two values of a head form pair i of `rot` rotated values. */
#define RFP2_ROPE_HALF 0        /* i and i + rot/2  */
#define RFP2_ROPE_INTERLEAVED 1 /* 2i and 2i + 1    */

/*
 * rfp2_rope -- rotary positions: the first rot values of every head are
 * rotated pair by pair, the rest is copied.  With a = pos[t] * freqs[i]:
 *   y1 = mscale * (x1 cos a - x2 sin a),  y2 = mscale * (x2 cos a + x1 sin a),
 * computed in fp64 and rounded once, so that far positions keep their angle.
 *   x   T rows of H heads of D fp32 values, row t at x + t * x_stride;
 *       y likewise with y_stride.  y == x with equal strides rotates in
 *       place; any other overlap is not allowed.  16-byte aligned.
 *   pos [T] int32 on the device (4-byte aligned), any value.
 *   freqs [rot/2] fp64 on the device, 8-byte aligned.
 * Requires T >= 1, H >= 1, 4 <= D <= 1024, D % 4 == 0, 2 <= rot <= D, rot
 * even, H * D <= 2^24, strides >= H * D and multiples of 4, a style of the
 * two above, mscale finite.
 */
rfp2_status rfp2_rope(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                      const int32_t* pos, const double* freqs, int64_t rot, int style,
                      double mscale, float* y, int64_t y_stride, hipStream_t stream);

/* What a cached value is held as. */
#define RFP2_KV_F16 0 /* IEEE half precision                                    */
#define RFP2_KV_I8 1  /* int8, one fp32 scale per 32 values of a token and head,
                         code and scale exactly as rfp2_quantize_acts gives them */

/*
 * rfp2_kv_cache -- a paged key/value cache.  The struct itself lives in HOST
 * memory and is read during the call; the pointers in it are device pointers
 * owned by the caller.  Token p of sequence s is row p % page_size of page
 * page_table[s * max_pages + p / page_size]; entries whose tokens no call
 * touches may hold anything.  With H = kv_heads, D = head_dim, P = page_size:
 *   k        [pages][H][P][D]        half or int8, 16-byte aligned
 *   v        [pages][H][P/8][D][8]   the same type, 16-byte aligned: eight
 *            tokens side by side for each value, the order in which the
 *            attention's matrix instructions sum over tokens
 *   k_scale, v_scale [pages][H][P/8][D/32][8] fp32, 16-byte aligned: the
 *            scale of 32 values, eight tokens side by side (RFP2_KV_I8; not
 *            read for RFP2_KV_F16)
 *   page_table [seqs][max_pages] int32, 4-byte aligned
 * Requires 1 <= kv_heads <= 1024, head_dim a multiple of 32 from 32 to 256,
 * page_size a power of two from 8 to 4096, 1 <= pages < 2^31, 1 <= seqs <=
 * 2^20, max_pages >= 1, max_pages * page_size < 2^31.  Offsets into the cache
 * are computed in 64 bits.
 */
typedef struct rfp2_kv_cache {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  const int32_t* page_table;
  int64_t seqs;
  int64_t max_pages;
  int64_t pages;
  int64_t page_size;
  int64_t kv_heads;
  int64_t head_dim;
  int32_t format;
} rfp2_kv_cache;

/*
 * rfp2_kv_write -- T tokens' keys and values into the cache.
 *   k, v  T rows of kv_heads heads of head_dim fp32 values, row t at
 *         k + t * k_stride and v + t * v_stride; 16-byte aligned.
 *   seq, pos [T] int32 on the device: token t is token pos[t] of sequence
 *         seq[t].  pos[t] < 0 marks padding: nothing is stored.
 *   err   nullable device int32: a token whose sequence, position or page lies
 *         outside the cache is not stored and 1 is written to *err (never
 *         cleared by the call).
 * RFP2_KV_F16 rounds to nearest even (beyond 65504: infinity).
 * A place should be named once in a call.  Named by several tokens it holds a
 * mixture: each code, half or scale is one token's, but the scale of a block may
 * be another's than its codes (nothing orders the stores).  Other places are not
 * affected.
 * Requires T >= 1, strides >= kv_heads * head_dim and multiples of 4.
 */
rfp2_status rfp2_kv_write(const rfp2_kv_cache* cache, const float* k, const float* v, int64_t T,
                          int64_t k_stride, int64_t v_stride, const int32_t* seq,
                          const int32_t* pos, int32_t* err, hipStream_t stream);

/*
 * rfp2_rope_kv_write -- rfp2_rope of T tokens' H query heads and kv_heads key
 * heads at positions pos, and rfp2_kv_write of the rotated keys and of the
 * values, in one launch (the row of one QKV product: q, k and v may be parts
 * of the same rows).  Bit-identical to the separate calls (but for places named
 * by several tokens, as in rfp2_kv_write).  q_out (row t at
 * q_out + t * q_out_stride) must not overlap q, k or v (equal to one of them it is
 * refused: lanes read their pairs while others write); it is written for
 * every token, padding too.  H == 0 with q == q_out == NULL rotates and
 * stores keys alone.
 * Requires what the two calls require, and rot <= head_dim.
 */
rfp2_status rfp2_rope_kv_write(const rfp2_kv_cache* cache, const float* q, const float* k,
                               const float* v, int64_t T, int64_t H, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, const int32_t* seq,
                               const int32_t* pos, const double* freqs, int64_t rot, int style,
                               double mscale, float* q_out, int64_t q_out_stride, int32_t* err,
                               hipStream_t stream);

/*
 * rfp2_kv_read -- T cached tokens back as fp32 (code * scale, or the half
 * value): the reverse of rfp2_kv_write, with the same arguments.  pos[t] < 0
 * gives a row of zeros; a token outside the cache gives a row of NaN and 1 is
 * written to *err.
 */
rfp2_status rfp2_kv_read(const rfp2_kv_cache* cache, int64_t T, const int32_t* seq,
                         const int32_t* pos, float* k, float* v, int64_t k_stride,
                         int64_t v_stride, int32_t* err, hipStream_t stream);

/*
 * rfp2_paged_attn -- attention of each sequence's newest tokens over its
 * cached tokens (its own keys and values already written).
 *   Sequence b (row b of the page table) holds lens[b] tokens; its queries are
 *   the tokens at positions lens[b] - new_tokens + t, t = 0 .. new_tokens - 1.
 *   The query at position p sees the cached positions j with j <= p and, where
 *   window > 0, j > p - window.  Query head h reads key/value head
 *   h / (H / kv_heads):
 *     y = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q.k_j - max).
 *   q   [B][new_tokens] rows of H heads of head_dim fp32 values, row i at
 *       q + i * q_stride; 16-byte aligned.
 *   y   [B][new_tokens][H][head_dim] fp32, 16-byte aligned, no overlap with q
 *       or the cache.  A query that sees nothing (lens[b] <= 0, or a position
 *       below 0) gives zeros.
 *   lens [B] int32 on the device; 4-byte aligned.
 *   err nullable device int32: a length beyond max_pages * page_size, or a
 *       visible token on a page outside the cache, gives NaN rows, and 1 is
 *       written to *err (never cleared by the call).
 *   workspace  device memory of at least rfp2_paged_attn_workspace_bytes(cache,
 *       B, new_tokens, H) bytes, 256-byte aligned, owned by the caller;
 *       overwritten.  Calls that share a workspace must not overlap in time.
 * Scores, weights and sums are held in fp32; the queries enter the matrix
 * cores as two half-precision numbers each (22 bits of the row's largest), scaled by a
 * power of two: scores and sums stay finite for int8 keys up to 2^104 and values up to
 * 2^87 in magnitude (halves end far below), beyond which results may be infinite or NaN.
 * A score of minus infinity (a half key beyond 65504) is a weight of 0, one of plus
 * infinity makes its row NaN.  The result
 * depends on nothing but the arguments (no atomics on values) and is the same
 * from call to call.  What lies in the cache beyond a sequence's length never
 * reaches an output.  Nothing is read back to the host, so the call can be
 * captured in a graph and replayed with longer sequences.
 * Requires 1 <= B <= min(1024, cache->seqs), B * max_pages * page_size <=
 * 2^36, 1 <= new_tokens <= RFP2_ATTN_MAX_NEW, H a multiple of kv_heads, H <= 1024, q_stride >= H *
 * head_dim and a multiple of 4, window >= 0, scale finite.
 */
#define RFP2_ATTN_MAX_NEW 8
size_t rfp2_paged_attn_workspace_bytes(const rfp2_kv_cache* cache, int64_t B,
                                       int64_t new_tokens, int64_t H);
rfp2_status rfp2_paged_attn(const rfp2_kv_cache* cache, const float* q, int64_t B,
                            int64_t new_tokens, int64_t H, int64_t q_stride,
                            const int32_t* lens, float scale, int64_t window, float* y,
                            int32_t* err, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

/*
 * The calls around the products of a feed-forward part, dense or routed: the
 * norm that adds to the residual stream and quantizes, the routing of tokens
 * to experts, the gate's activation between two products, and the experts'
 * weighted sum back onto the stream.  fp32 rows come in; what a product takes
 * next goes out (int8 activations exactly as rfp2_quantize_acts gives them
 * for the fp32 values, expert ids).  Inner arithmetic is fp64 with one
 * rounding to fp32: a value is the fp32 number next to the formula's, or the
 * other neighbour where the formula's lies within the fp64 error of their
 * middle, and codes and scales are the quantizer's of these.  That error is at
 * most 2^-43 of a value or of the sum of its terms' magnitudes (2^-40 in rows of
 * more than 16384 values, whose squares a thread adds by the hundreds and more;
 * 2^-41 where a gelu is below 2^-149 of its gate).  Infinities and NaN go through
 * the formulas (a block of 32 that holds one gets d = NaN, q = 0).
 *
 * rfp2_rms_norm -- the norm of each head (of a query or key before rfp2_rope):
 *   y = x * gain / sqrt(mean over the head of x^2 + eps).
 *   x, y  T rows of H heads of D values, row t at x + t * x_stride and
 *         y + t * y_stride; 16-byte aligned.  y == x with equal strides works
 *         in place; any other overlap is not allowed.
 *   gain  [D], the same for all heads; 16-byte aligned.
 * Requires T >= 1, H >= 1, 4 <= D <= 1024, D % 4 == 0, H * D <= 2^24, strides
 * >= H * D and multiples of 4, eps > 0 and finite.
 */
rfp2_status rfp2_rms_norm(const float* x, int64_t T, int64_t H, int64_t D, int64_t x_stride,
                          const float* gain, double eps, float* y, int64_t y_stride,
                          hipStream_t stream);

/*
 * rfp2_add_rms_norm -- a product's rows added to the residual stream, and the
 * norm of the sum as the next product's input:
 *   h = x + add,  y = h * gain / sqrt(mean over the row of h^2 + eps),
 *   q, d = rfp2_quantize_acts of y.
 *   x, add, h, y  T rows of K values, row t at x + t * x_stride and so on;
 *         16-byte aligned.  add may be NULL (h is then NULL too: the norm of
 *         x); h, y, and q with d may be NULL where they are not wanted, but
 *         not y and q both.  h and y may each be x or add with equal strides
 *         (not both the same one); any other overlap is not allowed.
 *   gain  [K], 16-byte aligned.
 *   q [T][K] int8, d [T][K/32] fp32, both 4-byte aligned (16 for q where a
 *         product reads it).
 * Requires T >= 1, 4 <= K <= 2^24, K % 4 == 0 (K % 32 == 0 with q), strides
 * (of what is there) >= K and multiples of 4, eps > 0 and finite.
 */
rfp2_status rfp2_add_rms_norm(const float* x, const float* add, int64_t T, int64_t K,
                              int64_t x_stride, int64_t add_stride, const float* gain, double eps,
                              float* h, int64_t h_stride, float* y, int64_t y_stride, int8_t* q,
                              float* d, hipStream_t stream);

/*
 * rfp2_moe_combine -- the routed experts' rows summed by their weights onto the
 * residual stream, with the norm that follows (rfp2_add_rms_norm's) in the same
 * pass:
 *   h = x + sum_j weights[t][j] * rows[t][j]   (fp64, rounded once).
 *   x, h, y, gain, q, d  as rfp2_add_rms_norm; x may be NULL (nothing is added
 *         to).  With gain NULL there is no norm (eps is not read), y, q and d are
 *         NULL and h is not; with a gain, h may be NULL but not y and q both.
 *         h and y may each be x with equal strides (not both).
 *   rows     [T][top_k][K] fp32, 16-byte aligned: what rfp2_moe_gemv,
 *         rfp2_moe_gemv_tokens and rfp2_moe_gemm write.
 *   weights  [T][top_k] fp32, 4-byte aligned.
 * A weight of 0 does not take out a row that holds NaN or infinity.
 * Requires 1 <= top_k <= 1024, T * top_k <= 2^30, the limits of
 * rfp2_add_rms_norm otherwise.
 */
rfp2_status rfp2_moe_combine(const float* x, const float* rows, const float* weights, int64_t T,
                             int64_t top_k, int64_t K, int64_t x_stride, const float* gain,
                             double eps, float* h, int64_t h_stride, float* y, int64_t y_stride,
                             int8_t* q, float* d, hipStream_t stream);

/* How a router's logits become scores. */
#define RFP2_ROUTE_SOFTMAX 0 /* p = exp(l) / sum over the experts of exp(l) */
#define RFP2_ROUTE_SIGMOID 1 /* p = 1 / (1 + exp(-l))                       */

/*
 * rfp2_moe_route -- the experts of each token and their weights, from the
 * router's logits: the ids that rfp2_moe_gemv and its kin take, the weights
 * that rfp2_moe_combine takes.
 *   logits [T] rows of E fp32, row t at logits + t * stride; 4-byte aligned.
 *   bias   nullable [E] fp32, 4-byte aligned: added to the scores for the
 *          choice only (a balance among the experts); finite.
 *   v_e = p_e + bias_e, or v_e = logits_e without a bias.  With groups > 1 the
 *   experts form `groups` runs of E / groups; a group counts by the sum of its
 *   group_top (1 or 2) largest v (by those that are not masked), and only the
 *   top_groups best groups stay.  The top_k largest v among what stays are
 *   chosen, in falling order; among equal groups or experts the lower comes
 *   first.  v and p are fp64, p within 2^-43 of the formula's: with a bias, scores
 *   that differ by less may come in either order (those of equal logits and biases
 *   are equal).  A sigmoid's logit, or one less the token's largest in a softmax,
 *   below -690 makes p 0; renorm goes by the chosen logits there, and its weights
 *   are the formula's however small the scores are.
 *   ids     [T][top_k] int32, 4-byte aligned.
 *   weights [T][top_k] fp32, 4-byte aligned: scale * p of the chosen, where
 *          renorm != 0 divided by the sum of the chosen p (0 where all are masked).
 *   err     nullable device int32: a token with a logit of NaN or plus infinity,
 *          or any bias that is not finite, gets ids of -1 and weights of NaN, and
 *          1 is written to *err (never cleared by the call).
 * A logit of minus infinity masks its expert: p = 0, and it is chosen only where
 * fewer than top_k others stay (with weight 0; the lower first).  A token whose
 * logits are all minus infinity gets valid ids and weights of 0.
 * Requires T >= 1, 1 <= E <= 2048, stride >= E, 1 <= top_k <= 64, groups from 1 to
 * 64 dividing E, 1 <= top_groups <= groups, top_k <= top_groups * (E / groups),
 * group_top 1, or 2 with a bias and E / groups >= 2, scale finite.
 */
rfp2_status rfp2_moe_route(const float* logits, int64_t T, int64_t E, int64_t stride,
                           const float* bias, int score, int64_t groups, int64_t group_top,
                           int64_t top_groups, int64_t top_k, int renorm, double scale,
                           int32_t* ids, float* weights, int32_t* err, hipStream_t stream);

/* The activation of a gate. */
#define RFP2_GATE_SILU 0 /* g / (1 + exp(-g))                                            */
#define RFP2_GATE_GELU 1 /* 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))            */

/*
 * rfp2_quantize_gated_acts -- act(gate) * up as int8 activations: what lies
 * between the gate and up products and the down product of a feed-forward part.
 *   gate, up  M rows of K fp32, row m at gate + m * gate_stride and up + m *
 *             up_stride (two halves of one product's rows, or two products);
 *             16-byte aligned.
 *   act       one of the two above.
 *   q [M][K] int8, d [M][K/32] fp32: rfp2_quantize_acts of the product's fp32
 *             values; 4-byte aligned, no overlap with gate or up.
 * Requires M >= 1, K >= 32, K % 32 == 0, K <= 2^24, strides >= K and multiples
 * of 4.
 */
rfp2_status rfp2_quantize_gated_acts(const float* gate, const float* up, int64_t M, int64_t K,
                                     int64_t gate_stride, int64_t up_stride, int act, int8_t* q,
                                     float* d, hipStream_t stream);

/*
 * rfp2_dequantize_acts -- the values that int8 activations stand for,
 * a = fl32(q * d): the reverse of rfp2_quantize_acts (a router or any other
 * reader of fp32 values can follow a call that wrote q and d alone).
 *   q, d as rfp2_quantize_acts writes them, 4-byte aligned; a [M][K] fp32,
 *   16-byte aligned, no overlap with q or d (refused: others still read them).
 * Requires M >= 1, K >= 32, K % 32 == 0, K <= 2^30.
 */
rfp2_status rfp2_dequantize_acts(const int8_t* q, const float* d, int64_t M, int64_t K, float* a,
                                 hipStream_t stream);

/*
 * rfp2_read_ceiling -- measurement helper, not part of the method: reads
 * `bytes` bytes of buf once with the plainest coalesced 16-byte loads
 * (thread t of the grid reads pieces t, t + T, t + 2T, ... of 16 bytes,
 * T = 256 * min(2048, ceil(bytes / 4096)) threads) and XORs the four words of
 * every piece it reads; a thread whose XOR equals `magic` writes it to
 * out[t], no other thread writes.  Its time is the ceiling for any kernel that
 * must read that many bytes (launch and ramp-up included), the yardstick the
 * products' effective bandwidth is reported against besides the HBM peak.
 *   buf  device bytes, 16-byte aligned.
 *   out  device uint32 [T] (RFP2_READ_CEILING_OUTPUTS at most); only the
 *        entries of threads whose XOR equals magic are written.
 * Requires bytes >= 16, bytes % 16 == 0.
 */
#define RFP2_READ_CEILING_OUTPUTS 524288
rfp2_status rfp2_read_ceiling(const uint8_t* buf, int64_t bytes, uint32_t magic, uint32_t* out,
                              hipStream_t stream);

/*
 * Inspection entry points.  They run the products' own device functions on
 * the register layouts the products use, so what they return is what the
 * products compute internally ("03 · Runtime": SPREAD / PERMUTE expand each
 * code byte into four int8 lanes, DOT4 sums each 16-weight half in int32).
 *
 * rfp2_debug_decode: the GEMV's decode.  The block stream is taken in 80-byte
 * groups of 8 blocks, as a GEMV lane holds them, and each block is decoded as
 * the GEMV decodes block j of its group (the odd blocks start at byte 2 of a
 * dword).  codes_out [N][K] int8: the lane each weight expands to;
 * scales_out [N][K/16] fp32: the scale of each half (NaN for an illegal
 * byte).  Requires N >= 1, K >= 32, K % 32 == 0; w 2-byte aligned, codes_out
 * and scales_out 4-byte aligned.
 *
 * rfp2_debug_half_dots: the GEMV's int32 sum of each 16-weight half against
 * the int8 activations (staged in the GEMV's lane order), sums_out
 * [M][N][K/32][2] int32.  Requires N >= 1, M >= 1, K >= 32, K % 32 == 0,
 * M * N * (K/32) <= 2^40; w 2-byte aligned, q 4-byte aligned.
 *
 * rfp2_debug_half_sums_mf: the same int32 half sums as computed by the
 * GEMV's matrix-core form of two to eight columns (v_mfma_i32_4x4x4_16b_i8
 * over quads of four rows at one 8-block group, one column's activations per
 * lane; "03 · Runtime": the half's int8 products summed in int32 before any
 * scale), sums_out [M][N][K/32][2] int32 as rfp2_debug_half_dots.  Requires
 * N >= 1, M >= 1, K >= 256, K % 256 == 0, M * N * (K/32) <= 2^40; w 2-byte
 * aligned, q 4-byte aligned.
 *
 * rfp2_debug_decode_f16: the fp16 value (level x scale) each weight takes in
 * the fp16 matrix-core products, h_out [N][K] as IEEE half-precision bit
 * patterns in natural order (NaN for both halves of a block with an illegal
 * scale byte).  form 0: the decode of rfp2_gemm_f16 (a thread expands both
 * halves of one block of a 20-byte pair); form 1: the decode of
 * rfp2_moe_gemm (a lane expands one half of a block straight into its
 * matrix-core operand).  Requires N >= 1, K >= 32, K % 32 == 0, form 0 or 1;
 * w and h_out 2-byte aligned.
 */
rfp2_status rfp2_debug_decode(const uint8_t* w, int64_t N, int64_t K,
                              int8_t* codes_out, float* scales_out,
                              hipStream_t stream);
rfp2_status rfp2_debug_half_dots(const uint8_t* w, int64_t N, int64_t K,
                                 const int8_t* q, int64_t M,
                                 int32_t* sums_out, hipStream_t stream);
rfp2_status rfp2_debug_half_sums_mf(const uint8_t* w, int64_t N, int64_t K,
                                    const int8_t* q, int64_t M,
                                    int32_t* sums_out, hipStream_t stream);
rfp2_status rfp2_debug_decode_f16(const uint8_t* w, int64_t N, int64_t K, int form,
                                  uint16_t* h_out, hipStream_t stream);

/*
 * rfp2_debug_decode_i8: the decode of rfp2_gemm (the int8 matrix-core
 * product), as its staging threads run it: blocks taken in dword-aligned
 * 20-byte pairs (the second block of a pair starts at byte 2 of a dword),
 * the scale mantissas folded into the two int8 operands.  Per block, in
 * natural weight order: wa_out [N][K] and wb_out [N][K] int8, the operands
 * whose weight k stands for wa[k] * sA + wb[k] * sB; scales_out
 * [N][K/32][6] fp32 = (s, -1.5*2^23*s, sA, -1.5*2^23*sA, sB,
 * -1.5*2^23*sB), where s = sA = sB when the block is one dot product and
 * s = -sB (negative: the split path) when its halves stay apart; all six
 * are NaN for a block with an illegal scale byte.
 * Requires N >= 1, K >= 32, K % 32 == 0; w 2-byte aligned, the outputs
 * 4-byte aligned.
 */
rfp2_status rfp2_debug_decode_i8(const uint8_t* w, int64_t N, int64_t K, int8_t* wa_out,
                                 int8_t* wb_out, float* scales_out, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* RFP2_H */
