/*
 * dg.h - C ABI of the MI355X (gfx950) FP8 block-scaled NT GEMM library.
 *
 * What the library computes (D = A . B^T with fine-grained scales):
 *
 *   D[m, n] = bf16( sum over 128-wide K slabs kb of
 *                   (sum_{k in slab} A[m, k] * B[n, k]) * sfa[m, kb] * sfb[n / 128, kb] )
 *
 * A and B hold OCP e4m3 codes (1 byte, largest finite 448).  A carries one
 * fp32 scale per row and 128-wide K slab; B one fp32 scale per 128 x 128
 * block.  The operation and its MoE layouts are the ones described on the
 * DeepGEMM pages: "DeepSeek open-source week day 3" (deepseek.csdn.net),
 * section "technical features" (FP8 GEMM with fine-grained scaling and a
 * second, higher-precision accumulation level; contiguous and masked grouped
 * layouts); "DeepGEMM: making LLM matrix multiplication fly" (pomoai.com),
 * sections "core functions" (block-wise scaling) and "technical details"
 * (the fp8_gemm_nt naming: both operands K-contiguous).  The 1x128 / 128x128
 * granularity, e4m3 and the bf16 output are readings of those pages.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every pointer argument is caller-owned DEVICE memory (hipMalloc'd or a
 *   torch CUDA tensor) on the current device.  The library never frees,
 *   keeps or allocates anything on behalf of a call's arguments.
 * - Every compute call is asynchronous on `stream` (0 = the null stream),
 *   performs no host<->device copy and no synchronisation, and reads no
 *   device value on the host; every one can be captured into a HIP graph
 *   (see the workspace rule below).
 * - Split-K workspace.  Dense calls (fp8, bf16, fp4, 4-bit weights) whose K is
 *   split over several workgroups, and attention calls whose keys are, keep
 *   fp32 partial results and arrival counters in a library-owned workspace,
 *   one per (device, stream).  Calls on one stream
 *   share it in stream order; calls on different streams never share one, so
 *   split-K calls may overlap in time on different streams.  A call that
 *   needs more than its stream's workspace holds makes a larger one (one
 *   hipMalloc, then a zero-fill kernel on `stream`; the library frees
 *   nothing, so it adds no hipFree synchronisation); the smaller block is
 *   retired, not freed, and stays
 *   allocated until the process ends, because a launch in flight or a graph
 *   captured earlier may still use it.  While `stream` is capturing a graph
 *   such a growth is refused with DG_ERR_WORKSPACE and nothing is enqueued:
 *   size the workspace first with dg_reserve_workspace(bytes, stream), bytes
 *   from dg_dense_workspace_size (dg_bf16_w4_workspace_size,
 *   dg_kv8_attention_workspace_size, dg_latent_attention_workspace_size).  A
 *   captured call keeps using the workspace its capture stream had; a replay must not overlap in time with other
 *   split-K work on that same workspace (replaying on the capture stream, or
 *   on any stream ordered with it, is safe).  dg_fp8_gemm_nt_noalloc uses a
 *   static per-GPU array instead and allocates nothing.
 * - Layouts are packed and row-major:
 *     A       [m][k]               (masked: [num_groups][max_m][k])
 *     B       [n][k]               (grouped: [num_groups][n][k])
 *     D       [m][n] bf16 bits     (masked: [num_groups][max_m][n])
 *     sfa     slab-major [k/128][ld], ld = dg_get_sfa_ld(m): sfa[kb*ld + row]
 *             (masked: [num_groups][k/128][dg_get_sfa_ld(max_m)])
 *     sfb     [ceil(n/128)][k/128] (grouped: [num_groups][ceil(n/128)][k/128])
 * - Preconditions checked on the host: non-null pointers, A/B/D/sfa/sfb
 *   16-byte aligned, k >= 128 and k % 128 == 0 (the bf16 and fp4 entry points
 *   state their own K rule), n >= 1, m >= 0.  m == 0 (or
 *   num_groups == 0 rows) is a successful no-op.  On a failed check nothing
 *   is enqueued, D is untouched and a status other than DG_OK is returned;
 *   dg_last_error_message() then describes the failure.
 * - D is overwritten (not accumulated) for valid rows only; every other
 *   element of D is left bit-for-bit untouched.
 * - No exception crosses this interface.  Every function may be called from
 *   several host threads at once (the workspace table is locked; the last
 *   error message is kept per thread).
 */
#ifndef DG_H
#define DG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* dg_stream_t; /* the same handle as hipStream_t */

typedef enum {
  DG_OK = 0,
  DG_ERR_INVALID_ARGUMENT = 1, /* null pointer, negative size, bad count        */
  DG_ERR_UNSUPPORTED_SHAPE = 2, /* k not a multiple of 128, m not aligned, ...  */
  DG_ERR_MISALIGNED = 3,        /* a pointer not 16-byte aligned                 */
  DG_ERR_NO_DEVICE = 4,         /* no usable gfx950 device                       */
  DG_ERR_HIP = 5,               /* a HIP runtime call or kernel launch failed     */
  DG_ERR_INTERNAL = 6,
  DG_ERR_WORKSPACE = 7          /* the stream's split-K workspace would have to
                                   grow while the stream is capturing a graph */
} dg_status;

/*
 * Dense FP8 NT GEMM: D[m][n] = A[m][k] . B[n][k]^T with 1x128 (A) and
 * 128x128 (B) fp32 block scales.  Rows m and columns n may be any size >= 0
 * and >= 1 respectively; a partial last 128-row block of B uses its own scale
 * row of sfb.  When the output tiles alone cannot fill the GPU (skinny m,
 * or few tiles, as in one GPU's shard of a larger GEMM), the K dimension is
 * split over several workgroups whose fp32 partial tiles meet in the
 * stream's split-K workspace (see the conventions above) and are added in a
 * fixed order, so results stay bit-for-bit reproducible.  For m <= 16, on
 * shapes whose 128-wide K slabs of 64-row tiles fill one run of at least 12
 * slabs per CU, a kernel that deals those slabs to the workgroups in equal
 * runs is used instead; every other shape takes the tiled kernels.  The
 * choice never changes a result beyond the split-K summation order.
 */
int dg_fp8_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                   uint16_t* d, int m, int n, int k, dg_stream_t stream);

/*
 * dg_fp8_gemm_nt for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, kernels and results as dg_fp8_gemm_nt (bit for bit), but
 * a split-K call takes its fp32 partial tiles and arrival counters from a
 * static array of the library, one per GPU (16 MiB of partials and 16384
 * counters, held until the process ends), instead of the stream's workspace;
 * the call never allocates, frees or synchronises.  Each call clears the
 * counters it uses with a small kernel on `stream` before the GEMM.  A call
 * that would need more scratch than the array holds returns
 * DG_ERR_UNSUPPORTED_SHAPE with nothing enqueued (the 64 x 2112 x 7168
 * decode shape takes 3.6 MiB).  All calls on one GPU share the array, so
 * calls of this entry point that overlap in time on one GPU (two streams, or
 * two threads) race and give wrong results; dg_fp8_gemm_nt has no such
 * limit.
 */
int dg_fp8_gemm_nt_noalloc(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                           uint16_t* d, int m, int n, int k, dg_stream_t stream);

/*
 * MoE grouped GEMM, contiguous layout ("DeepSeek open-source week day 3",
 * technical features, MoE item on the contiguous layout): the rows of all
 * experts are stacked in A (m rows), experts share n and k, and
 * m_indices[r] (device int32, m entries) names the expert whose B row r
 * uses.  Each aligned block of dg_get_m_alignment_for_contiguous_layout()
 * rows must belong to one expert; rows tagged outside [0, num_groups)
 * (padding, conventionally -1) are neither computed nor written, nor are
 * rows whose tag differs from the expert of their block.
 * m must be a multiple of that alignment (else DG_ERR_UNSUPPORTED_SHAPE).
 */
int dg_m_grouped_fp8_gemm_nt_contiguous(const uint8_t* a, const float* sfa, const uint8_t* b,
                                        const float* sfb, uint16_t* d, const int32_t* m_indices,
                                        int m, int n, int k, int num_groups, dg_stream_t stream);

/*
 * MoE grouped GEMM, masked layout ("DeepSeek open-source week day 3",
 * technical features, MoE item on the masked layout; PPIO's evaluation,
 * masked-layout section, decode use): every expert g owns a fixed
 * max_m x k slab of A and max_m x n slab of D; masked_m[g] (device int32,
 * num_groups entries, clamped on the device to [0, max_m]) says how many
 * leading rows are valid.  Only valid rows are computed and written, so the
 * shapes never change and the call suits graph capture.  expected_m is a
 * host-side hint of the typical valid count per expert (0 = unknown); it
 * only steers the tile choice and never changes results (every tile gives
 * the same bits).  Counts up to 48 pick 128-row tiles, which stream B
 * fastest while every expert fits 128 rows but slow down when one does not
 * (max_m <= 128 picks them in any case); counts up to 80 a 256-row tile
 * with the same streaming schedule; larger or unknown counts the schedule
 * that overlaps the fullest experts' MFMA work with their loads.
 */
int dg_m_grouped_fp8_gemm_nt_masked(const uint8_t* a, const float* sfa, const uint8_t* b,
                                    const float* sfb, uint16_t* d, const int32_t* masked_m,
                                    int num_groups, int max_m, int n, int k, int expected_m,
                                    dg_stream_t stream);

/*
 * MoE FC1 + SwiGLU on the masked layout, with h requantised for the second
 * GEMM: the single-GPU slice of the fused MoE kernel the pages describe
 * (the popular-press article on DeepGEMM, yeyulingfeng.com, section 04 on
 * Mega MoE: dispatch, the first GEMM, the SwiGLU activation, the second GEMM
 * and combine in one kernel; dispatch and combine across GPUs are not part of
 * this call).
 * B holds each expert's FC1 weight as [gate; up]: rows 0..inter-1 are the
 * gate projection, rows inter..2*inter-1 the up projection.  For expert g
 * and valid row m (m < clamp(masked_m[g], 0, max_m)):
 *
 *   gate[j] = FP8 GEMM of A[g][m] with B[g][j]           (as dg_m_grouped_fp8_gemm_nt_masked,
 *   up[j]   = FP8 GEMM of A[g][m] with B[g][inter + j]    but kept in fp32)
 *   h[j]    = silu(gate[j]) * up[j],   silu(x) = x / (1 + exp(-x))
 *
 * and h is quantised with the activation rule of dg_quantize_a_1x128 (per
 * row and 128-wide block of h: amax floored at 1e-4, s = amax / 448,
 * code = e4m3(h / s)), all in fp32.  Layouts:
 *     A   [num_groups][max_m][k] e4m3, sfa [num_groups][k/128][dg_get_sfa_ld(max_m)]
 *     B   [num_groups][2*inter][k] e4m3, sfb [num_groups][2*inter/128][k/128]
 *     hq  [num_groups][max_m][inter] e4m3 codes (output)
 *     hs  [num_groups][inter/128][dg_get_sfa_ld(max_m)] fp32 scales (output)
 * hq and hs are exactly the A operand of a masked GEMM with k = inter, so
 * the second layer reads them without a conversion pass.  inter must be a
 * positive multiple of 128 and k of 128; pointers 16-byte aligned
 * (masked_m 4-byte).  Rows past an expert's count, and the padding entries
 * of hs, are left untouched.  expected_m is a hint as for the masked GEMM.
 * Errors as for the other entry points; nothing is allocated.
 */
int dg_m_grouped_fp8_gemm_nt_masked_swiglu(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                                           uint8_t* hq, float* hs, const int32_t* masked_m, int num_groups,
                                           int max_m, int inter, int k, int expected_m, dg_stream_t stream);

/*
 * MoE FC1 + SwiGLU + FP8 requantisation on the contiguous layout: the
 * prefill side of dg_m_grouped_fp8_gemm_nt_masked_swiglu (the popular-press
 * article on DeepGEMM, yeyulingfeng.com, section on MoE: the contiguous
 * layout for prefill, the masked one for decode; section 04 on Mega MoE for
 * the fused FC1 and SwiGLU).  B holds each expert's FC1 weight as [gate; up]
 * as for the masked entry point, and for every row m whose tag
 * e = m_indices[m] lies in [0, num_groups):
 *
 *   gate[j] = FP8 GEMM of A[m] with B[e][j]           (as dg_m_grouped_fp8_gemm_nt_contiguous,
 *   up[j]   = FP8 GEMM of A[m] with B[e][inter + j]    but kept in fp32)
 *   h[j]    = silu(gate[j]) * up[j]
 *
 * quantised with the activation rule of dg_quantize_a_1x128, all in fp32.
 * Layouts:
 *     A   [m][k] e4m3, sfa [k/128][dg_get_sfa_ld(m)], m_indices [m] (-1 = padding)
 *     B   [num_groups][2*inter][k] e4m3, sfb [num_groups][2*inter/128][k/128]
 *     hq  [m][inter] e4m3 codes (output)
 *     hs  [inter/128][dg_get_sfa_ld(m)] fp32 scales (output)
 * hq and hs are exactly the A operand of a contiguous GEMM with k = inter
 * and the same m_indices.  m must be a multiple of the 128-row alignment
 * (every 128-row block holds one expert's rows and padding); inter a
 * positive multiple of 128, k of 128; pointers 16-byte aligned (m_indices
 * 4-byte).  Padding rows, rows with an out-of-range tag and the padding
 * entries of hs are left untouched.  Errors as for the other entry points;
 * nothing is allocated.
 */
int dg_m_grouped_fp8_gemm_nt_contiguous_swiglu(const uint8_t* a, const float* sfa, const uint8_t* b,
                                               const float* sfb, uint8_t* hq, float* hs, const int32_t* m_indices,
                                               int m, int inter, int k, int num_groups, dg_stream_t stream);

/*
 * BF16 NT GEMM: D[m][n] = bf16( sum_k A[m, k] * B[n, k] ) for bf16 A [m][k]
 * and B [n][k] (bit patterns in uint16), fp32 accumulation, no scales
 * ("DeepGEMM: making LLM matrix multiplication fly", pomoai.com, core
 * functions: BF16 GEMMs beside the FP8 ones).  The same tiles, LDS layout and
 * split-K as the FP8 dense GEMM run it on gfx950's bf16 MFMA
 * (v_mfma_f32_16x16x32_bf16).  k must be a positive multiple of 64 (one
 * 128-byte slab row); otherwise as dg_fp8_gemm_nt (m may be 0, n >= 1,
 * 16-byte aligned pointers, the split-K workspace note applies).
 */
int dg_bf16_gemm_nt(const uint16_t* a, const uint16_t* b, uint16_t* d, int m, int n, int k, dg_stream_t stream);

/*
 * FP4 NT GEMM ("DeepGEMM: making LLM matrix multiplication fly", pomoai.com,
 * core functions: FP4 named beside FP8 and BF16; its caveats warn that FP4
 * may cost accuracy).  The pages give FP4 no scaling rule, so the FP8 method
 * carries over with e2m1 operands:
 *
 *   D[m][n] = bf16( sum over slabs kb of
 *                   (sum_{k in kb} A[m, k] * B[n, k]) * sfa[m, kb] * sfb[n / 128, kb] )
 *
 * A [m][k/2] and B [n][k/2] hold e2m1 codes two per byte (element 2i in the
 * low nibble of byte i); sfa (slab-major, dg_get_sfa_ld(m)) and sfb
 * ([ceil(n/128)][k/128]) are the FP8 scale layouts.  k must be a positive
 * multiple of 256 (whole 128-byte rows); otherwise as dg_fp8_gemm_nt (m may
 * be 0, n >= 1, 16-byte aligned pointers, the split-K workspace note).
 */
int dg_fp4_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb, uint16_t* d,
                   int m, int n, int k, dg_stream_t stream);

/*
 * K-grouped GEMM ("DeepGEMM: making LLM matrix multiplication fly",
 * pomoai.com, core functions: the K-grouped family beside the M-grouped one,
 * for the irregular shapes of MoE training such as weight gradients, where
 * the tokens of each expert form a run of K).  The groups are concatenated
 * along K: group g owns the k_sizes[g] K columns that follow the groups
 * before it, and
 *
 *   D[g][m][n] = bf16( sum over group g's slabs kb of
 *                      (sum_{k in slab kb} A[m, k] * B[n, k]) * sfa[m, kb] * sfb[n / 128, kb] )
 *
 * with the dense layouts and scales for A [m][k], sfa (slab-major,
 * dg_get_sfa_ld(m)), B [n][k] and sfb [ceil(n/128)][k/128]; D is
 * [num_groups][m][n] bf16.  k_sizes is device int32 (num_groups entries),
 * read only on the device so that the call is graph-capturable: each size
 * must be a multiple of 128 and their sum at most k; on the device a
 * negative size counts as 0, the remainder below a multiple of 128 is
 * ignored, and a group is cut off at k.  A group with no K columns gets
 * D[g] = 0.  Every element of D is written.
 */
int dg_k_grouped_fp8_gemm_nt(const uint8_t* a, const float* sfa, const uint8_t* b, const float* sfb,
                             uint16_t* d, const int32_t* k_sizes, int num_groups, int m, int n, int k,
                             dg_stream_t stream);

/* Row alignment required of each expert's segment in the contiguous layout (128). */
int dg_get_m_alignment_for_contiguous_layout(void);

/* Leading dimension of the slab-major sfa layout for m rows: m rounded up to 4. */
int dg_get_sfa_ld(int m);

/*
 * Quantise an fp32 activation matrix x[m][k] to e4m3 codes q[m][k] with one
 * fp32 scale per row and 128-wide slab, written slab-major to
 * sfa[kb*dg_get_sfa_ld(m) + row] (entries for rows >= m are set to 0).
 * Per block: amax = max|x| (floored at 1e-4), s = amax / 448 (fp32, correctly
 * rounded), q = e4m3(x / s) rounded to nearest even and saturated at 448.
 */
int dg_quantize_a_1x128(const float* x, uint8_t* q, float* sfa, int m, int k, dg_stream_t stream);

/*
 * Quantise an fp32 weight matrix x[n][k] to e4m3 codes q[n][k] with one fp32
 * scale per 128 x 128 block, sfb[ceil(n/128)][k/128]; same rule as above;
 * the last row block may be partial.
 */
int dg_quantize_b_128x128(const float* x, uint8_t* q, float* sfb, int n, int k, dg_stream_t stream);

/*
 * FP4 quantisers: as dg_quantize_a_1x128 / dg_quantize_b_128x128 with e2m1
 * codes (range 6): per block amax (floored at 1e-4), s = amax / 6 (fp32,
 * correctly rounded), code = e2m1(x / s) rounded to nearest with ties to
 * even, saturated at 6.  q is [m][k/2] (resp. [n][k/2]) bytes, two codes per
 * byte, element 2i in the low nibble; the scale layouts are the FP8 ones.
 */
int dg_quantize_a_1x128_fp4(const float* x, uint8_t* q, float* sfa, int m, int k, dg_stream_t stream);
int dg_quantize_b_128x128_fp4(const float* x, uint8_t* q, float* sfb, int n, int k, dg_stream_t stream);

/*
 * ---- 4-bit weights with bf16 activations
 *
 * A weight matrix [n][k] in 4 bits with one bf16 scale for every row and group
 * of 32, 64 or 128 values along K:
 *
 *   w[n][k] = s[n][k / group] * (c[n][k] - z[n][k / group])
 *
 *   codes  [n][k/2] bytes, two codes per byte (element 2i in the low nibble)
 *   scales [n][k/group] bf16 bits
 *   zeros  [n][k/group] bytes 0..15: DG_W4_U4 only, NULL for DG_W4_E2M1
 *
 * DG_W4_E2M1: c is the e2m1 value of the code (as dg_fp4_gemm_nt), z = 0.
 * DG_W4_U4: c is the code itself, 0..15.
 * k must be a positive multiple of group; every pointer 16-byte aligned.
 */
typedef enum { DG_W4_E2M1 = 0, DG_W4_U4 = 1 } dg_w4_format;

/*
 * d[m][n] = bf16( sum_g s[n][g] * (sum_{k in g} c[n][k] a[m][k] - z[n][g] * sum_{k in g} a[m][k]) )
 * for bf16 a [m][k]: the projections of a decode step, where a handful of
 * tokens meet weights that are read once.  Products and sums are fp32 (the
 * scale meets the fp32 sum of its group, so no weight is rounded after
 * scaling), in one launch, with the same bits on every call.  Any m >= 0 (0: a
 * no-op) is computed.  The weights are read once for m <= 16; more rows read them
 * again for every 16 while the product is small, else for every 32 (m <= 32) or
 * 64, so a long prompt is better served by dg_dequantize_b_w4 and
 * dg_bf16_gemm_nt.  With m > 16, K may be split over workgroups: the call then
 * needs dg_bf16_w4_workspace_size bytes of the stream's workspace (see the
 * workspace rule above).
 *
 * DG_W4_U4 codes enter the products as 128 + c, and (128 + z) sum a is taken off
 * in fp32: an output carries fp32 roundings of terms up to 143 s |a|, for weights
 * of up to 15 s.  So rows of a whose sum of 143 |a| over a group passes fp32's
 * range give outputs that are not finite, and rows with an infinity NaN, whatever
 * the weights' signs.  DG_W4_E2M1 has no such limit.  NaN and infinities stay in
 * their row.
 */
int dg_bf16_w4_gemm_nt(const uint16_t* a, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
                       uint16_t* d, int m, int n, int k, int group, int format, dg_stream_t stream);

/* Bytes of the stream's workspace that dg_bf16_w4_gemm_nt takes for a shape on
 * the current device: 0 for m <= 16, and for more rows while the product is small. */
int dg_bf16_w4_workspace_size(int m, int n, int k, int group, int format, size_t* bytes);

/*
 * Quantise a weight matrix x[n][k] (bf16 bits if x_bf16, else fp32) into that
 * form; x must be finite, and for DG_W4_U4 hi - lo too.  Per row and group:
 *   DG_W4_E2M1: s = bf16(max(amax, 1e-4) / 6), code = e2m1(x / s), nearest, ties to even
 *   DG_W4_U4:   lo = min(x, 0), hi = max(x, 0), s = bf16(max(hi - lo, 1e-4) / 15),
 *               z = min(rint(-lo / s), 15), code = clamp(rint(x / s) + z, 0, 15)
 * in fp32 with correctly rounded divisions, against the scale as stored.
 */
int dg_quantize_b_w4(const void* x, int x_bf16, uint8_t* codes, uint16_t* scales, uint8_t* zeros, int n, int k,
                     int group, int format, dg_stream_t stream);

/* w[n][k] = bf16(s * (c - z)): the bf16 weights that codes stand for. */
int dg_dequantize_b_w4(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, uint16_t* w, int n, int k,
                       int group, int format, dg_stream_t stream);

/*
 * ---- An 8-bit key/value cache and the attention over it
 *
 * A pool of num_blocks blocks of `block` tokens (16, 32, 64 or 128) of h_kv
 * heads of d values (64, 128 or 256), in e4m3 codes with one fp32 scale for
 * each block and head, keys and values apart:
 *
 *   k_codes [num_blocks][h_kv][block][d]    k_scales [num_blocks][h_kv]
 *   v_codes [num_blocks][h_kv][d][block]    v_scales [num_blocks][h_kv]
 *
 * (values lie dimension by dimension).  block_table [batch][max_blocks] int32
 * names the block that holds tokens j * block .. j * block + block - 1 of each
 * sequence.  Entries that no token in question falls into are not read; tokens
 * whose entry lies outside [0, num_blocks), or past max_blocks, are neither
 * written nor seen.  Code arrays may pass 4 GiB.  An array without elements (no
 * blocks, no sequences, a table of no width) may be NULL.
 *
 * Packed tokens: q, k, v hold the rows of all sequences one after the other,
 * [total][heads][d] bf16 with *_stride elements (a multiple of 8) from token to
 * token, so slices of one projection's output serve as they are; cu [batch+1]
 * int32 holds the running sums of the sequences' rows, cu[0] = 0.  Lengths and
 * running sums live on the device and are read there only; rows outside
 * [0, total) and rows past the given longest sequence are ignored.
 *
 * dg_kv8_append puts k and v of the new tokens of every sequence behind the
 * ctx_lens[i] tokens that it has in the cache (max_new: the most new tokens of
 * one sequence).  Per block and head, over the new values that fall into it:
 *
 *   s' = max(s, smallest power of two p with amax <= 448 p)   amax floored at 1e-4
 *   code = e4m3(x / s'), nearest even
 *
 * with s the block's scale, or 0 if it held no token; if s' > s the block's
 * older codes become e4m3(c * s / s').  Powers of two lose nothing in either
 * step but below the smallest normal code.  amax counts finite values;
 * infinities saturate, NaN is stored as NaN.  A block that gets tokens must
 * belong to one sequence.  Bytes past a sequence's last token keep what they
 * held.  Nothing is allocated.
 */
int dg_kv8_append(const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, uint8_t* k_codes,
                  uint8_t* v_codes, float* k_scales, float* v_scales, const int32_t* block_table,
                  const int32_t* ctx_lens, const int32_t* cu_new, int batch, int total, int max_new, int h_kv, int d,
                  int block, int num_blocks, int max_blocks, dg_stream_t stream);

/*
 * Attention of the packed queries over the cache: for query i of the n_i of
 * sequence s, standing at position kv_lens[s] - n_i + i (its own key is in the
 * cache already, so one call serves single tokens, several tokens and prompts
 * behind a cached prefix), and head h reading key/value head h / (h_q / h_kv):
 *
 *   x[j] = scale * (q . k[j]),  out = sum_j softmax(x)[j] v[j],  lse = log sum_j e^x[j]
 *
 * with scale >= 0, over the tokens j it sees: those up to its own position if causal, all
 * kv_lens[s] otherwise, and of these the last `window` if window > 0 (causal
 * only).  A row that sees no token gets out = 0 and lse = -inf.  A NaN in a
 * key or value reaches the rows that see it and no others; what the cache
 * holds past kv_lens[s] reaches none.  Scales must be positive (a value scale
 * below 2^-64 counts as 2^-64), and the value scales that a row sees within
 * 2^100 of each other.
 * out is bf16 [total][h_q][d], lse fp32 [total][h_q] or NULL.  max_q is the
 * most queries of one sequence.  Scores, the softmax's running maximum and
 * sums and the output's accumulator are fp32; for the second product each
 * probability times its value scale is rounded to 11 bits or more (and, where
 * the value scales of a sequence are within 2^4 of each other, to steps of
 * 2^-31 of the row's largest).  Results do not depend on anything but the
 * arguments: the same call gives the same bits.
 * Needs dg_kv8_attention_workspace_size bytes of the stream's workspace (see
 * the workspace rule above: reserve it before capturing).  The work is shared
 * out on the device from the lengths it finds there, so a captured call stays
 * right, and balanced, as sequences grow.
 */
int dg_kv8_attention(const uint16_t* q, int64_t q_stride, const uint8_t* k_codes, const uint8_t* v_codes,
                     const float* k_scales, const float* v_scales, const int32_t* block_table,
                     const int32_t* kv_lens, const int32_t* cu_q, uint16_t* out, float* lse, float scale, int causal,
                     int window, int batch, int total, int max_q, int h_q, int h_kv, int d, int block, int num_blocks,
                     int max_blocks, dg_stream_t stream);

/* Bytes of the stream's workspace that dg_kv8_attention takes on the current device. */
int dg_kv8_attention_workspace_size(int d, size_t* bytes);

/*
 * ---- Latent attention: keys and values from one shared latent vector a token
 *
 * A token is a latent c of `latent` values (512 or 256) and a rope part r of
 * P = latent / 8 values, shared by all heads.  Absorbed, a head's key is (c, r)
 * and its value c; expanded, an up-projection of c gives each head a key part
 * and a value of D = latent / 4 values each, and its key is (key part, r).
 *
 * A paged cache holds, for num_blocks blocks of `block` tokens (16, 32, 64 or 128):
 *
 *   latent [num_blocks][block][latent]       bf16 if scales is NULL, else e4m3
 *   rope   [num_blocks][block][P]            bf16
 *   scales [num_blocks][block][latent / 128] fp32 powers of two, or NULL
 *
 * block_table, lengths, running sums and packed rows are those of the 8-bit
 * key/value cache above: tokens whose entry lies outside [0, num_blocks), or
 * past max_blocks, are neither written nor seen; rows outside [0, total) and
 * rows past the given longest sequence are ignored, and what would hold their
 * results keeps what it held.  Cache arrays may pass 4 GiB; an array without
 * elements may be NULL.
 *
 * dg_latent_append takes the latent and rope parts of new tokens, bf16 rows
 * with *_stride elements (a multiple of 8, at least the row) from token to token,
 * so slices of one projection's output serve as they are.  Token i of sequence s stands at
 * position ctx_lens[s] + i.  Into its place go
 *
 *   y = norm * c / sqrt(mean(c^2) + eps), or c if norm is NULL, in fp32: rounded
 *       to bf16, or, for each 128 values, with s the smallest power of two with
 *       amax <= 448 s (amax floored at 1e-4), e4m3(y / s), nearest even
 *   r turned by its position: (a, b) -> (a cos - b sin, a sin + b cos) in fp32,
 *       rounded to bf16, for pairs (r[2 i], r[2 i + 1]) if interleaved, else
 *       (r[i], r[i + P / 2]); cos and sin are angles[pos][i], angles[pos][P / 2 + i]
 *
 * with norm bf16 [latent] and angles fp32 [positions][P].  If q is not NULL,
 * the rope parts of the h_q query heads of each token (q_stride elements from
 * token to token, q_head_stride from head to head, strides as in
 * dg_latent_attention) are turned alike and written to q_out, which may be q
 * itself (else q_out overlaps no input); its rows must lie apart.  Tokens at positions outside [0, positions) are ignored;
 * no two tokens of a call may have the same place in the cache.  amax counts
 * finite values; infinities saturate, NaN is stored as NaN.  With a norm a NaN
 * makes the whole token NaN, and an infinity itself NaN and the rest of its
 * token 0.  At most 2^25 tokens a call.
 */
int dg_latent_append(const uint16_t* latent, int64_t latent_stride, const uint16_t* rope, int64_t rope_stride,
                     void* cache_latent, uint16_t* cache_rope, float* cache_scales, const int32_t* block_table,
                     const int32_t* ctx_lens, const int32_t* cu_new, const float* angles, int positions,
                     const uint16_t* norm, float eps, const uint16_t* q, int64_t q_stride, int64_t q_head_stride,
                     uint16_t* q_out, int64_t q_out_stride, int64_t q_out_head_stride, int interleaved, int batch,
                     int total, int max_new, int h_q, int latent_dim, int block, int num_blocks, int max_blocks,
                     dg_stream_t stream);

/*
 * Cached tokens as packed bf16 rows, latent [total][latent] and rope [total][P]:
 * row cu[s] + i is token starts[s] + i of sequence s (starts NULL: from 0 on).
 * e4m3 latents come out as the values they stand for.  Rows of tokens that the
 * table has no block for keep what they held.  At most 2^25 rows a call.
 */
int dg_latent_gather(const void* cache_latent, const uint16_t* cache_rope, const float* cache_scales,
                     const int32_t* block_table, const int32_t* starts, const int32_t* cu, uint16_t* latent,
                     uint16_t* rope, int batch, int total, int latent_dim, int block, int num_blocks, int max_blocks,
                     dg_stream_t stream);

/*
 * Absorbed attention of packed queries over the cache: for query i of the n_i of
 * sequence s, standing at position kv_lens[s] - n_i + i (its own token is in the
 * cache already), and each of the h_q heads,
 *
 *   x[j] = scale * (q . c[j] + q_rope . r[j]),  out = sum_j softmax(x)[j] c[j],  lse = log sum_j e^x[j]
 *
 * with scale >= 0, over the tokens j up to its own position if causal, all
 * kv_lens[s] otherwise.  A row that sees no token gets out = 0 and lse = -inf.
 * q [total][h_q][latent], q_rope [total][h_q][P] and out [total][h_q][latent]
 * are bf16, with any strides from token to token and from head to head that are
 * multiples of 8, from head to head 0 (one row for all heads) or at least the row;
 * out's rows must lie apart.  lse is fp32 [total][h_q] or NULL;
 * max_q is the most queries of one sequence (max_q * h_q at most 2^30).
 * A token whose latent or rope part is not finite can make the rows that see it
 * not finite, and no others; what the cache holds past kv_lens[s] reaches none.
 * Where its score is -inf its weight is 0, and 0 times an infinite latent makes
 * that channel of the row NaN and leaves the others.
 * Scores, the softmax's running reference and sums and the output's
 * accumulator are fp32; for the second product each probability is rounded to
 * bf16, in steps of 64 tokens that some row does not see wholly to two bf16
 * pieces.  The same call gives the same bits.  How many rows a workgroup takes goes
 * by max_q, h_q and the tokens that the table and the pool have room for, not by the
 * lengths, so a captured call keeps it: in a pool much larger than what its
 * sequences hold a short call takes longer, and last bits may differ from one pool
 * to another.  Needs
 * dg_latent_attention_workspace_size bytes of the stream's workspace (reserve
 * it before capturing); the work is shared out on the device from the lengths
 * it finds there.
 */
int dg_latent_attention(const uint16_t* q, int64_t q_stride, int64_t q_head_stride, const uint16_t* q_rope,
                        int64_t q_rope_stride, int64_t q_rope_head_stride, const void* cache_latent,
                        const uint16_t* cache_rope, const float* cache_scales, const int32_t* block_table,
                        const int32_t* kv_lens, const int32_t* cu_q, uint16_t* out, int64_t out_stride,
                        int64_t out_head_stride, float* lse, float scale, int causal, int batch, int total, int max_q,
                        int h_q, int latent_dim, int block, int num_blocks, int max_blocks, dg_stream_t stream);

/* Bytes of the stream's workspace that dg_latent_attention takes on the current device. */
int dg_latent_attention_workspace_size(int latent_dim, int max_q, int h_q, size_t* bytes);

/*
 * Expanded attention of packed prompts: for query i of the n_i of sequence s,
 * which has m_i tokens, standing at position m_i - n_i + i, and each head,
 *
 *   x[j] = scale * (q[0..D) . k[j] + q[D..D + P) . r[j]),  out = sum_j softmax(x)[j] v[j]
 *
 * q bf16 [total][heads][D + P] and kv bf16 [total_kv][heads][2 D] (key part,
 * then value; an up-projection's output as it stands), k_rope bf16 [total_kv][P],
 * with *_stride elements (a multiple of 8, at least the row, for kv and k_rope
 * less than 2^26) from token to token;
 * cu_q, cu_kv int32 [batch + 1] running sums; out bf16 [total][heads][D], lse
 * fp32 [total][heads] or NULL; head_dim D is 128 or 64, P = D / 2.  Masks, rows
 * that see nothing, precision and determinism as in dg_latent_attention; a
 * value that is not finite makes that dimension of the rows that see it not
 * finite and nothing else.  Needs no workspace.
 */
int dg_latent_expanded_attention(const uint16_t* q, int64_t q_stride, const uint16_t* kv, int64_t kv_stride,
                                 const uint16_t* k_rope, int64_t k_rope_stride, const int32_t* cu_q,
                                 const int32_t* cu_kv, uint16_t* out, float* lse, float scale, int causal, int batch,
                                 int total, int total_kv, int max_q, int heads, int head_dim, dg_stream_t stream);

/*
 * Size the split-K workspace of `stream` on the current device to hold at
 * least `bytes` of partial tiles (dg_dense_workspace_size gives a call's
 * need), so that later calls on that stream that fit allocate nothing and
 * can be captured.  Growing allocates one block and enqueues a zero-fill
 * kernel on `stream`; it does not synchronise the device.  Returns
 * DG_ERR_WORKSPACE, with nothing done, if it would have to grow while
 * `stream` is capturing.
 */
int dg_reserve_workspace(size_t bytes, dg_stream_t stream);

/* Operand types of the dense entry points, for dg_dense_workspace_size. */
typedef enum { DG_DTYPE_FP8 = 0, DG_DTYPE_BF16 = 1, DG_DTYPE_FP4 = 2 } dg_dtype;

/*
 * Bytes of split-K workspace that a dense call of this dtype and shape
 * (dg_fp8_gemm_nt, dg_bf16_gemm_nt or dg_fp4_gemm_nt, m x n, K of k values)
 * needs on the current device: 0 when the call does not split K.  Passing
 * it to dg_reserve_workspace for a stream before capturing such calls on
 * that stream keeps them from allocating.  Same shape checks as the GEMM calls (k a positive
 * multiple of 128, 64 or 256 for fp8, bf16 and fp4, m >= 0, n >= 1), an
 * unknown dtype is DG_ERR_INVALID_ARGUMENT, and *bytes is 0 on any error.
 */
int dg_dense_workspace_size(int dtype, int m, int n, int k, size_t* bytes);

/* Static text for a status code. */
const char* dg_status_string(int status);

/* Detail of the last failure on the calling thread ("" if none). */
const char* dg_last_error_message(void);

/*
 * Profiling hook: the next GEMM launch made on the calling thread records
 * `start_event` and `stop_event` (hipEvent_t handles created by the caller
 * with timing enabled; either may be NULL) at the start and end of the
 * kernel itself (hipExtLaunchKernel), so hipEventElapsedTime gives the
 * kernel's own duration without launch gaps.  One-shot: the hook clears
 * itself after that launch.  Not graph-capturable; for measurement only.
 */
int dg_profile_next_launch(void* start_event, void* stop_event);

/* Library version string. */
const char* dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_H */
