/*
 * qgemm.h -- C ABI of the packed-int4 weight GEMM library for AMD Instinct
 * MI355X (gfx950).
 *
 * It computes C[M,N] = A[M,K] . W[K,N] where W is held as 4-bit codes q in
 * [0,15], eight to a uint32, with one fp16 scale (and, asymmetric, one fp16
 * zero) per group of `group_size` consecutive k and per column n:
 *
 *   symmetric offset-binary  W[k,n] = (q[k,n] - 8) * scale[k/g, n]
 *   asymmetric               W[k,n] =  q[k,n] * scale[k/g, n] + zero[k/g, n]
 *
 * Sources (web pages, cited by title and section):
 *   [Marlin-Ada]  "Marlin INT4 on Ada - how it works" (TinyLoop docs):
 *                 "The core mismatch: symmetric vs asymmetric" (both formats,
 *                 delta = zero + 8*scale, C = C_sym + A_group_sum @ delta),
 *                 "The pipeline, end to end" (pack, group-sum and correction
 *                 stages), "How the dispatcher chooses" (K, N multiples of
 *                 128; group_size == K written as -1 for per-column scales).
 *   [HyperQwen]   "HyperQwen int8 tensor-core fix of the Marlin W4A8 negative
 *                 scale bug and per-layer activation quantization": the W4A8
 *                 path (int4 weights, per-token int8 activations, integer
 *                 accumulation) and the load-time sign fold of negative group
 *                 scales (scale -> -scale, code v -> 16 - v, clamped at 15).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers, row-major and contiguous, owned
 *     by the caller.  The library allocates no device memory and keeps no
 *     device state; scratch memory is a caller-provided workspace whose size
 *     qg_workspace_bytes() reports (0 for every path that needs none).
 *   - A W4A16 workspace starts with QG_W4A16_WS_COUNTER_BYTES bytes of
 *     split-K counters, then the fp32 partial sums (decode-size batches,
 *     M <= 80, where the split-K decode kernel runs) and the
 *     correction's group sums (QG_CORR_SEPARATE).  It must be zero-filled
 *     before its first use; every qgemm_w4a16 call leaves the counters at zero
 *     again, so one zero-filled workspace serves any sequence of qgemm_w4a16
 *     calls on one stream, whatever their shapes and flags.  Do not use it for
 *     anything else in between (group_sum_correction included).  Calls that
 *     may overlap in time (different streams or devices) must not share one.
 *   - fp16 tensors are passed as uint16_t (IEEE binary16 bit patterns).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).  All
 *     work is enqueued asynchronously; nothing is synchronised or read back.
 *   - Every argument is validated on the host BEFORE anything is launched; on
 *     error nothing is written and nothing is launched.  The return value is a
 *     QG_* status; qg_last_error() gives a per-thread description.  There is no
 *     internal fallback to another path: the caller decides what to do.
 *   - Shapes: K % 128 == 0 and N % 128 == 0 (the tile multiples the pages'
 *     dispatcher requires), M >= 1.  group_size must divide K and be 32, 64,
 *     a multiple of 128, or K; -1 is accepted as an alias of K (per-column
 *     scales), for every operation.
 *     pack_int4_weights, qgemm_w4a16 and qgemm_w4a8 also take any K, N >= 1
 *     ("tails"):
 *     group_size is then 32, 64, a multiple of 128 (the last group of g
 *     consecutive k may be partial: G = ceil(K / g)), K, or -1; see
 *     qg_padded_shape.
 *     Limits: K < 2^22 and ceil(K / g) * N * 2 < 2^31 (the kernels' 32-bit
 *     offsets; qgemm_w4a16_swiglu counts the pair's 2N), else
 *     QG_ERR_UNSUPPORTED.
 *   - A, C, scale, zero and delta must be 2-byte aligned; w_packed 16-byte
 *     aligned; A 16-byte aligned for the W4A16 GEMM, A_q 8-byte aligned for
 *     W4A8.
 *   - Calls on the same stream are ordered; concurrent calls on different
 *     streams that write the same output race (as any two kernels would).
 */
#ifndef QGEMM_H
#define QGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ---- */
#define QG_OK               0
#define QG_ERR_INVALID_ARG  1  /* NULL pointer, bad alignment, M < 1, ...        */
#define QG_ERR_UNSUPPORTED  2  /* shape or group size this library has no kernel for */
#define QG_ERR_WORKSPACE    3  /* workspace missing or smaller than required      */
#define QG_ERR_DEVICE       4  /* current device is not gfx950 / no device        */
#define QG_ERR_LAUNCH       5  /* the HIP runtime rejected a launch               */

/* ---- flags ---- */
/* pack_int4_weights: fold negative group scales into the codes (symmetric
 * packs only; ignored when zero != NULL).                                   */
#define QG_PACK_FOLD_NEG_SCALES 0x1u
/* qgemm_w4a16: add the asymmetric term with the two-stage
 * group_sum_correction (after an fp16 store of the symmetric product)
 * instead of fusing it into the GEMM epilogue.                              */
#define QG_CORR_SEPARATE        0x1u

/* Size of the counter region at the start of every non-empty W4A16
 * workspace (see the conventions above).                                    */
#define QG_W4A16_WS_COUNTER_BYTES 65536u

/* ---- operations, for qg_workspace_bytes ---- */
#define QG_OP_W4A16                 1
#define QG_OP_W4A8                  2
#define QG_OP_GROUP_SUM_CORRECTION  3
#define QG_OP_PACK                  4
#define QG_OP_W4A16_SWIGLU          5
#define QG_OP_FP8                   6
#define QG_OP_MOE_SORT              7  /* M = tokens, N = topk, num_experts  */
#define QG_OP_LORA                  8  /* M = tokens, group_size = rank, num_experts = adapters */

/* ---- element types, for the calls that take more than one ---- */
#define QG_DTYPE_F16                0
#define QG_DTYPE_BF16               1
#define QG_DTYPE_F32                2

/* 1 if HIP device `device` is a gfx950 GPU this library has kernels for,
 * else 0 (also 0 when the device does not exist).  The analogue of the pages'
 * runtime architecture gate ([Marlin-Ada], "How the dispatcher chooses").   */
int qg_device_supported(int device);

/* Static text for a QG_* status. Never NULL.                                */
const char *qg_status_string(int status);

/* Description of the last error on the calling thread ("" if none). The
 * pointer stays valid until the next library call on that thread.          */
const char *qg_last_error(void);

/* Padded shape of a pack of [K,N] codes with this group size (any K, N >= 1):
 * the packed weight holds K_padded * N_padded / 8 uint32, scale_out and
 * delta_out are [groups, N_padded] fp16.  K_padded = K rounded up to a whole
 * group (to 128 when group_size is K, -1, 32 or 64), N_padded = N rounded up to 128,
 * groups = K_padded / group_size (1 per column): ceil(K / group_size), except
 * that groups of 32 or 64 may add whole groups past K (zero scale and delta in
 * the pack; the input scale and zero keep ceil(K / group_size) rows).  Equal
 * to K, N, K/g for shapes
 * without tails.  Any output pointer may be NULL.  Returns a QG_* status.  */
int qg_padded_shape(int K, int N, int group_size, int *K_padded, int *N_padded, int *groups);

/* Bytes of workspace `op` needs for this shape (0 when none). Returns
 * (size_t)-1 when the arguments are invalid.                                */
size_t qg_workspace_bytes(int op, int M, int N, int K, int group_size,
                          int num_experts, unsigned flags);

/* ---- load-time repack ([Marlin-Ada] "The pipeline, end to end";
 *      [HyperQwen] negative group-scale section) ----
 * q         [K,N] uint8, one code (0..15) per byte; larger values are an
 *           error the kernel cannot report and give unspecified codes.
 * scale     [ceil(K / group_size), N] fp16.
 * zero      [ceil(K / group_size), N] fp16, or NULL for a symmetric weight.
 * flags     QG_PACK_FOLD_NEG_SCALES: for a symmetric weight, every (g,n) with
 *           scale < 0 (strictly; -0.0 is left alone) gets scale -> -scale and
 *           codes v -> min(16 - v, 15) over that group.
 * w_packed  [K_padded*N_padded/8] uint32 out, in this library's MFMA-operand
 *           tile order (private layout; the only consumers are the GEMMs);
 *           padding codes are 8.
 * scale_out [groups,N_padded] fp16 out (groups from qg_padded_shape): the
 *           (folded) scale, 0 in padded columns and padded groups.  May
 *           alias `scale` when N % 128 == 0 and groups == ceil(K / g).
 * delta_out [groups,N_padded] fp16 out, required iff zero != NULL (0 in
 *           padded columns and groups):
 *           delta = round_to_nearest_even_fp16(zero + 8*scale), with the
 *           pre-fold scale and the sum formed exactly.
 * Runs one or two kernels on `stream`. No workspace.                        */
int pack_int4_weights(const uint8_t *q, const uint16_t *scale, const uint16_t *zero,
                      int K, int N, int group_size, unsigned flags,
                      uint32_t *w_packed, uint16_t *scale_out, uint16_t *delta_out,
                      void *stream);

/* ---- W4A16 GEMM ([Marlin-Ada] "The core mismatch") ----
 * A        [M,K] fp16 activations.
 * w_packed, scale: from pack_int4_weights.
 * delta    [G,N] fp16 from pack_int4_weights for an asymmetric weight, or NULL
 *          for a symmetric one.
 * C        [M,N] fp16 out, OVERWRITTEN with A . W (fp32 accumulation, one
 *          rounding to fp16 at the end).  The weights enter the products
 *          exactly in the decode kernel for up to 16 rows and in the skinny
 *          and mid-batch kernels (codes as exact fp16 values, scales applied
 *          in fp32), and rounded once per element to fp16 in the decode
 *          kernel for 17 to 80 rows ((v-8)*scale + delta) and in the tiled
 *          kernels ((v-8)*scale), so |W| must stay within the fp16 range;
 *          QGEMM_LOG=1 names the kernel a call runs.
 * flags    0: the delta term sum_g a_sum[m,g]*delta[g,n] is added in fp32 in
 *          the GEMM epilogue (one launch).
 *          QG_CORR_SEPARATE: C is first stored as the symmetric product and
 *          then corrected in place by group_sum_correction (needs workspace).
 * Tails (K or N not a multiple of 128, from a tail pack): A is copied into
 *          the workspace with zero columns up to K_padded, the GEMM runs on
 *          the padded shape and its product is cropped into C; the delta term
 *          is fused; QG_CORR_SEPARATE is QG_ERR_UNSUPPORTED.
 * workspace/workspace_bytes: qg_workspace_bytes(QG_OP_W4A16, ...) bytes,
 *          256-byte aligned (NULL when that is 0).  For decode-size batches
 *          (M <= 16, and up to M = 80 on all but small weights) the K range
 *          is split over several workgroups whose fp32 partial sums meet in
 *          the workspace; the last to finish adds them in a fixed order, so
 *          results do not depend on timing.  A grid that would leave a few
 *          CUs one workgroup more than the rest splits its last column groups
 *          finer (or, when nothing else is split, only those), which also
 *          takes workspace.                                                 */
int qgemm_w4a16(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                const uint16_t *delta, uint16_t *C, int M, int N, int K,
                int group_size, unsigned flags, void *workspace,
                size_t workspace_bytes, void *stream);

/* ---- W4A16 GEMM without a workspace argument, for callers that cannot
 *      allocate device memory (code under HIP graph capture, tight serving
 *      loops, harnesses that forbid allocation) ----
 * Same arguments, checks, kernels and results as qgemm_w4a16 minus the
 * workspace: the scratch a call needs (split-K partial sums and counters,
 * the separate correction's group sums, a tail shape's padded A and C) is a
 * static device array of QG_NOALLOC_SCRATCH_BYTES bytes inside the library,
 * one per GPU, held until the process ends.  No device memory is allocated
 * or freed by the call.  A call whose scratch need
 * (qg_workspace_bytes(QG_OP_W4A16, ...)) exceeds QG_NOALLOC_SCRATCH_BYTES
 * returns QG_ERR_WORKSPACE before anything is launched.  The first call on a
 * device clears the scratch's counter region with a small kernel on
 * `stream`; every call leaves it at zero again.  Every call on a GPU uses
 * that GPU's one array, which keeps the last call's contents: calls that may
 * overlap in time on one GPU (different streams, threads or graphs) race and
 * must be ordered by the caller.                                            */
#define QG_NOALLOC_SCRATCH_BYTES 33554432u
int qgemm_w4a16_noalloc(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                        const uint16_t *delta, uint16_t *C, int M, int N, int K,
                        int group_size, unsigned flags, void *stream);

/* ---- SwiGLU of an MLP's gate and up projections in one call ([Marlin-Ada]
 *      "Gaps and follow-ups": the fused mlp_gate + mlp_up dispatch) ----
 * The pair is ONE packed weight of shape [K, 2N]: pack_int4_weights on the
 * codes [W_gate | W_up] (gate columns 0..N-1, up columns N..2N-1) and their
 * [G, 2N] scales (and zeros) concatenated the same way.
 * A        [M,K] fp16, 16-byte aligned.
 * w_packed, scale, delta: the pair's pack (delta NULL for symmetric weights).
 * H        [M,N] fp16 out, 16-byte aligned, OVERWRITTEN with
 *            H[m,n] = silu(G[m,n]) * U[m,n],  silu(x) = x / (1 + exp(-x)),
 *          G = A . W_gate and U = A . W_up with their delta terms fused.
 *          One launch for every M: the kernel holds G and U of the same
 *          output columns in fp32 and rounds H once.
 * N % 128 == 0 (the output width), K and group_size as for qgemm_w4a16.
 * flags    must be 0.
 * workspace/workspace_bytes: qg_workspace_bytes(QG_OP_W4A16_SWIGLU, M, N, K,
 *          group_size, 1, 0) bytes, 256-byte aligned (NULL when 0: every
 *          shape but the decode batches whose grid splits K, for all column
 *          groups or for the last ones only); it starts with the same
 *          counter region as a W4A16 workspace (zero-filled once, left at
 *          zero by every call), so one workspace of the larger size serves
 *          both kinds of call on one stream.                                */
int qgemm_w4a16_swiglu(const uint16_t *A, const uint32_t *w_packed, const uint16_t *scale,
                       const uint16_t *delta, uint16_t *H, int M, int N, int K, int group_size,
                       unsigned flags, void *workspace, size_t workspace_bytes, void *stream);

/* ---- asymmetric correction as its own two stages ([Marlin-Ada] "The
 *      pipeline, end to end", a_group_sum and correction_accum) ----
 * C[m,n] += sum_g a_sum[m,g] * delta[g,n],  a_sum[m,g] = sum_{k in g} A[m,k]
 * a_sum is formed in fp32 in the workspace; C is read, updated in fp32 and
 * rounded back to fp16 (ACCUMULATES into C, unlike the GEMMs).
 * workspace: qg_workspace_bytes(QG_OP_GROUP_SUM_CORRECTION, ...) bytes.     */
int group_sum_correction(const uint16_t *A, const uint16_t *delta, uint16_t *C,
                         int M, int N, int K, int group_size, void *workspace,
                         size_t workspace_bytes, void *stream);

/* ---- grouped W4A8 GEMM ([HyperQwen] "why int8 activation quantization
 *      (W4A8) is worth doing"; zero-point weights: its verification section,
 *      point 2) ----
 * A_q          [M_total,K] int8 per-token codes; a_scale [M_total] fp32
 *              (quantize_rows_int8 makes both from fp16 activations).
 * w_packed     E stacked packs (each K*N/8 uint32).
 * w_scale      E stacked [G,N] fp16 scales (the packs' scale_out).
 * w_delta      NULL for symmetric weights; for asymmetric (zero-point) ones
 *              the E stacked [G,N] fp16 deltas (the packs' delta_out,
 *              delta = zero + 8*scale).
 * expert_offsets  DEVICE int32[E+1], non-decreasing, offsets[0] = 0,
 *              offsets[E] = M_total: expert e owns rows offsets[e] ..
 *              offsets[e+1]-1.  NULL means one expert owning all rows (E must
 *              be 1).  Rows are clipped to [0, M_total) in the kernel.
 * max_rows_per_expert  the expected largest offsets[e+1]-offsets[e]; it only
 *              sizes the launch (ceil(max_rows_per_expert / 64) row blocks per
 *              expert, each taking every further 64-row block of its expert in
 *              turn), so a bound below the true count is slower, never wrong.
 * C            [M_total,N] fp16 out, overwritten:
 *              C[m,n] = a_scale[m] * sum_g (scale_e[g,n] * acc[m,g,n]
 *                                           + delta_e[g,n] * qsum[m,g])
 *              acc[m,g,n] = sum_{k in g} A_q[m,k] * (v_e[k,n] - 8)  (int32, exact)
 *              qsum[m,g]  = sum_{k in g} A_q[m,k]                    (int32, exact)
 *              (the delta term only with w_delta), in fp32, one rounding to
 *              fp16 at the end.
 * acc_debug    NULL, or [M_total,G,N] int32 out receiving acc exactly.
 * Tails (K or N not a multiple of 128, packs from pack_int4_weights of that
 *              shape: each [K_padded*N_padded/8], scales [G,N_padded]): A_q
 *              is copied with zero columns into the workspace, the product is
 *              formed on the padded shape and cropped into C; acc_debug is
 *              then QG_ERR_UNSUPPORTED.
 * workspace/workspace_bytes: qg_workspace_bytes(QG_OP_W4A8, M_total, N, K,
 *              group_size, E, 0) bytes, 256-byte aligned: 0 (pass NULL, 0)
 *              unless the shape has tails.  The first
 *              QG_W4A16_WS_COUNTER_BYTES bytes are never touched (they are
 *              the W4A16 split-K counters' place), so one zero-filled
 *              workspace may serve W4A16 and W4A8 calls in turn on one
 *              stream.                                                      */
int qgemm_w4a8(const int8_t *A_q, const float *a_scale, const uint32_t *w_packed,
               const uint16_t *w_scale, const uint16_t *w_delta,
               const int32_t *expert_offsets, int num_experts,
               int M_total, int max_rows_per_expert, int N, int K, int group_size,
               uint16_t *C, int32_t *acc_debug, void *workspace, size_t workspace_bytes,
               unsigned flags, void *stream);

/* ---- per-token int8 activation quantization, the input stage of
 *      qgemm_w4a8 ([HyperQwen] "why int8 activation quantization (W4A8) is
 *      worth doing": activations are quantized per token to int8) ----
 * A        [M,K] fp16 activations, 16-byte aligned; K % 8 == 0 (else
 *          QG_ERR_UNSUPPORTED).
 * A_q      [M,K] int8 out, 8-byte aligned; a_scale [M] fp32 out:
 *            a_scale[m] = max_k |A[m,k]| / 127
 *            A_q[m,k]   = clamp(round_half_even(A[m,k] / a_scale[m]), -127, 127)
 *          both divisions single IEEE binary32 operations (round to nearest
 *          even); a row of zeros gets a_scale 0 and codes 0.  The outputs
 *          are exactly qgemm_w4a8's A_q and a_scale.  Non-finite inputs give
 *          unspecified codes.
 * One kernel on `stream`. No workspace.                                     */
int quantize_rows_int8(const uint16_t *A, int M, int K, int8_t *A_q, float *a_scale,
                       void *stream);

/* ---- per-row, per-128-column fp8 quantization, the input stage of
 *      qgemm_fp8 ----
 * A        [M,K] fp16 or bf16 (dtype QG_DTYPE_F16 / QG_DTYPE_BF16)
 *          activations, 16-byte aligned; K % 16 == 0 (else
 *          QG_ERR_UNSUPPORTED).  With QG_QUANT_SWIGLU a [M,2K] gate/up pair
 *          (gate columns first), and x below is silu(gate) * up, in 64 bits
 *          wherever that decides a scale or a code; without it x = A.
 * A_q      [M,K] e4m3 codes out (OCP: largest value 448, no infinity),
 *          16-byte aligned; a_scale [M, ceil(K/128)] fp32 out.  For each row
 *          m and block b of 128 columns (the last may be partial):
 *            a_scale[m,b] = max |x| / 448
 *            A_q[m,k]     = e4m3(clamp(x[m,k] / a_scale[m,b], -448, 448))
 *          both quotients rounded once to binary32, the code rounded to the
 *          nearest (ties to even).  A block of zeros, of either sign, or
 *          of values so small that max |x| / 448 rounds to 0 gets scale 0
 *          and codes 0 (the byte 0x00); a block with a NaN, an infinity or
 *          an x beyond binary32's range gets a NaN scale and NaN codes, so
 *          every product with it is NaN.
 * M == 0 is a call that does nothing.  One kernel on `stream`, no workspace. */
#define QG_QUANT_SWIGLU 0x1u
int quantize_rows_fp8(const void *A, int dtype, int M, int K, unsigned flags, uint8_t *A_q,
                      float *a_scale, void *stream);

/* ---- block-scaled fp8 GEMM, dense or grouped by expert ----
 * A_q          [M_a,K] e4m3 codes, 16-byte aligned; a_scale [M_a, KB] fp32,
 *              KB = ceil(K/128): one scale per row and 128 columns
 *              (quantize_rows_fp8 makes both).
 * a_rows       NULL: row m of C takes row m of A (M_a == M_total).  Else
 *              DEVICE int32[M_total]: row m of C takes row a_rows[m] of A
 *              (moe_sort_rows' row_token: a token's row is quantized and
 *              stored once, however many experts read it).  Rows whose index
 *              lies outside [0, M_a) get zeros.  M_a * K must not exceed
 *              2^32 - 2^23 (else QG_ERR_UNSUPPORTED).
 * W            E stacked [N,K] e4m3 codes (k contiguous), 16-byte aligned;
 *              w_scale E stacked [ceil(N/128), KB] fp32: one scale per 128 x
 *              128 block.
 * expert_offsets  as for qgemm_w4a8: DEVICE int32[E+1], non-decreasing, or
 *              NULL for one expert that owns all rows.  Rows outside
 *              [offsets[0], offsets[E]) are left as they were.  The counts
 *              are read on the device: no bound on them is needed.
 * C            [M_total,N] fp16 or bf16 (dtype) out, overwritten:
 *                C[m,n] = sum_b a_scale[r,b] * w_scale_e[n/128,b] * P
 *                P      = sum_{k in b} A_q[r,k] * W_e[n,k],  r = a_rows[m]
 *              in fp32, one rounding at the end.  P comes from the e4m3
 *              matrix instruction, which adds eight products of consecutive
 *              k at a time, each cut to 2^-13 of the eight's largest power
 *              of two.
 * N >= 1 and K % 16 == 0 (the last block may be partial in both); K < 2^22,
 * ceil(N/128) * KB < 2^29.  M_total == 0 does nothing.
 * workspace/workspace_bytes: qg_workspace_bytes(QG_OP_FP8, M_total, N, K, 128,
 *              E, 0) bytes, 256-byte aligned: 0 (NULL) for every shape.
 * flags        must be 0.                                                   */
int qgemm_fp8(const uint8_t *A_q, const float *a_scale, const int32_t *a_rows, int M_a,
              const uint8_t *W, const float *w_scale, const int32_t *expert_offsets,
              int num_experts, int M_total, int N, int K, int dtype, void *C, void *workspace,
              size_t workspace_bytes, unsigned flags, void *stream);

/* ---- routing to experts ----
 * logits   [T,E] of dtype QG_DTYPE_F32, _F16 or _BF16; bias [E] fp32 or NULL.
 * score    s[t,e] = softmax over e of logits[t,:], or with QG_ROUTE_SIGMOID
 *          1 / (1 + exp(-logits[t,e])).
 * choice   c[t,e] = s[t,e] + bias[e] (the bias balances the load: it takes
 *          part in the choice, not in the weights).
 * groups   n_group > 1: the experts stand in n_group runs of E / n_group; a
 *          run's value is its largest choice, or with QG_ROUTE_GROUP_TOP2 the
 *          sum of its two largest; only experts of the topk_group runs with
 *          the largest values can be chosen.
 * ids      [T,topk] int32 out: the experts with the largest choices, largest
 *          first.  Choices and sums rank in 64 bits; without a bias the
 *          logits themselves rank the experts, and by their largest the
 *          groups (the order of the scores, also where those saturate).
 *          Equal ones go to the lowest index.
 * weights  [T,topk] fp32 out: s[t,ids], with QG_ROUTE_RENORMALIZE divided by
 *          their sum over the token's chosen experts (0 where that sum is 0),
 *          times `scaling`.  Computed in binary32, each within (41 + d) 2^-24
 *          of its size, d the distance of its logit from the token's largest
 *          (softmax), or 24 * 2^-24 (sigmoid).  A token with a
 *          score under 2^-120 among its chosen, or one whose order 32 bits
 *          leave open, has its weights from 64 bits, rounded once.
 * An expert whose logit is -infinity or NaN, or whose choice is, is masked: it
 * is never chosen, and slots left over hold id -1 and weight 0 (moe_sort_rows
 * drops them).  A logit of +infinity counts as the largest, in equal shares.
 * 1 <= E <= 1024, n_group <= 64 a divisor of E, 1 <= topk_group <= n_group,
 * 1 <= topk <= 64 and <= topk_group * E / n_group.  T == 0 does nothing.  One
 * kernel, no workspace.                                                     */
#define QG_ROUTE_SIGMOID        0x1u
#define QG_ROUTE_RENORMALIZE    0x2u
#define QG_ROUTE_GROUP_TOP2     0x4u
int moe_route(const void *logits, int dtype, const float *bias, int T, int E, int topk,
              int n_group, int topk_group, float scaling, unsigned flags, int32_t *ids,
              float *weights, void *stream);

/* ---- the routed slots, sorted by expert ----
 * ids      [T,topk] int32: the expert of each slot; ids outside [0,E) drop
 *          their slot.
 * The kept slots, ordered by expert and inside an expert by slot (t * topk +
 * j), become the rows 0 .. M-1 of a grouped product, M = expert_offsets[E]:
 * expert_offsets  [E+1] int32 out: expert e owns rows offsets[e] ..
 *          offsets[e+1]-1 (as qgemm_w4a8 and qgemm_fp8 take them).
 * row_token  [T*topk] int32 out: the token of each row; entries from M on are
 *          left as they were.
 * slot_row   [T,topk] int32 out: each slot's row, -1 for a dropped slot.
 * T * topk < 2^30, 1 <= E <= 1024.  T == 0 writes expert_offsets = 0.
 * workspace/workspace_bytes: qg_workspace_bytes(QG_OP_MOE_SORT, T, topk, 0, 0,
 *          E, 0) bytes, 256-byte aligned (NULL when 0: few slots).  It needs
 *          no initial value and keeps none between calls; its first
 *          QG_W4A16_WS_COUNTER_BYTES bytes are never touched.              */
int moe_sort_rows(const int32_t *ids, int T, int topk, int num_experts, int32_t *expert_offsets,
                  int32_t *row_token, int32_t *slot_row, void *workspace, size_t workspace_bytes,
                  void *stream);

/* ---- the experts' rows, weighted and summed back to their tokens ----
 * Y        [M_rows,N] fp16 or bf16 (dtype); slot_row [T,topk] int32 from
 *          moe_sort_rows; weights [T,topk] fp32 from moe_route.
 * out      [T,N] of Y's type, overwritten:
 *            out[t,n] = sum_j weights[t,j] * Y[slot_row[t,j], n]
 *          in fp32 in the order of j, one rounding at the end.  A slot whose
 *          row lies outside [0, M_rows) adds nothing, whatever its weight; a
 *          token with no slot left gets zeros.
 * 1 <= topk <= 64.  T == 0 does nothing.  One kernel, no workspace.         */
int moe_combine_rows(const void *Y, int dtype, const int32_t *slot_row, const float *weights,
                     int T, int topk, int M_rows, int N, void *out, void *stream);

/* ---- paged 4-bit key/value cache ----
 * A cache holds, for `num_pages` pages of `page_size` tokens (a power of two
 * from 32 to 1024), `heads` key/value heads of `head_dim` channels (64, 128 or
 * 256) in groups of `group` channels (32, 64 or 128, at most head_dim).  A
 * group of a token is 4-bit codes c with an fp16 scale s and an fp16 zero z
 * (the weights' asymmetric form), and stands for c * s + z.
 *   k, v        [num_pages, heads, page_size, head_dim/8] uint32, 16-byte aligned
 *   k_sz, v_sz  [num_pages, heads, head_dim/group, page_size, 2] fp16 (scale,
 *               zero), 16-byte aligned
 * Eight codes to a word:
 *   keys    a token's words are [4][head_dim/32]; nibble 4a + 2b + c (a, b, c 0
 *           or 1) of word (q, 2i + l) is channel
 *           32 (i + c head_dim/64) + 8 q + 4 l + 2 b + a.
 *   values  the words of 32 consecutive tokens (32 n .. 32 n + 31 of a page) are
 *           [head_dim/64][4][16][4]; nibble 4a + 2b + c of word (u, q, m, j) is
 *           channel 64 u + 16 j + m of token 16 c + 4 q + 2 b + a.
 * A batch is B sequences:
 *   kv_lens     [B] int32: the tokens of each, the new ones among them.
 *   page_table  [B, max_pages] int32: token t of sequence b is token t %
 *               page_size of page page_table[b, t / page_size].
 *   seq_offsets [B+1] int32, non-decreasing, or NULL (T == B): the rows
 *               seq_offsets[b] .. seq_offsets[b+1]-1 of the call's T rows are
 *               the LAST tokens of sequence b, in order (kv_lens[b] - n .. kv_lens[b] - 1);
 *               NULL: row b is the last token of sequence b.  Rows outside
 *               [seq_offsets[0], seq_offsets[B]) are left as they were.
 * All three stand on the device and are read there.  A token whose index is
 * negative or past the table, or whose page lies outside [0, num_pages), has no
 * place in the cache: it is not stored, reads as zeros and is never attended
 * to.  Two sequences may share pages that a call only reads.
 * max_pages * page_size <= 2^30.  T == 0 or B == 0 does nothing.            */

/* Keys and values of new tokens rotated, quantized and appended.
 * k, v     rows of [heads, head_dim] fp16 or bf16 (dtype), 16-byte aligned; row t
 *          starts ld_k (ld_v) elements after row t - 1, a multiple of 8 (so the
 *          parts of one projection's output can be passed as they lie).
 * q        NULL, or rows of [q_heads, head_dim] of the same type (ld_q):
 *          rotated into q_out [T, q_heads, head_dim] (16-byte aligned, contiguous), rounded once.
 * cos_sin  [max_pos, rot_dim] fp32, 16-byte aligned: the cosines of a position's
 *          rot_dim / 2 angles, then the sines; NULL with rot_dim 0: no rotation.
 *          rot_dim is a multiple of 16, at most head_dim; channels past it pass.
 * positions  [T] int32, or NULL: each token's index in its sequence.  A position
 *          outside [0, max_pos) makes the row's rotated channels NaN.
 * flags    0: angle i turns the channels (i, i + rot_dim/2);
 *          QG_KV4_INTERLEAVED: (2i, 2i + 1).
 *            a' = a cos - b sin,  b' = b cos + a sin
 *          in fp32, each product and each sum rounded once.
 * A group x of a token is stored with (fp32, fp16 roundings to nearest even)
 *            z = fp16(min x),  s = fp16((max x - min x) / 15),
 *            c = clamp(round_half_even((x - z) / s), 0, 15),  0 where s is 0.
 *          A group with a NaN or with values past fp16's range gets NaN scale
 *          and zero and codes 0, and so is NaN wherever it is seen: one of
 *          values in its own channels, one of keys in the rows that see it.
 * No two rows of a call may name the same place of the cache.  One kernel, no
 * workspace.                                                                */
#define QG_KV4_INTERLEAVED 0x1u
int kv4_append(const void *k, const void *v, const void *q, int dtype, int T, int ld_k, int ld_v,
               int ld_q, int q_heads, const int32_t *seq_offsets, const int32_t *kv_lens,
               const int32_t *page_table, int B, int max_pages, const int32_t *positions,
               const float *cos_sin, int rot_dim, int max_pos, unsigned flags, uint32_t *cache_k,
               uint32_t *cache_v, uint16_t *cache_k_sz, uint16_t *cache_v_sz, int num_pages,
               int heads, int page_size, int head_dim, int group, void *q_out, void *stream);

/* The rows of a batch back as values: k_out, v_out [T, heads, head_dim] of
 * dtype QG_DTYPE_F32, _F16 or _BF16, 16-byte aligned: c * s + z in fp32, rounded once.
 * One kernel, no workspace.                                                 */
int kv4_read(const uint32_t *cache_k, const uint32_t *cache_v, const uint16_t *cache_k_sz,
             const uint16_t *cache_v_sz, int num_pages, int heads, int page_size, int head_dim,
             int group, const int32_t *seq_offsets, const int32_t *kv_lens,
             const int32_t *page_table, int B, int max_pages, int T, int dtype, void *k_out,
             void *v_out, void *stream);

/* Attention of new tokens over the cache (which holds them already).
 * q        rows of [q_heads, head_dim] fp16 or bf16, 16-byte aligned, ld_q as
 *          above; q_heads a multiple of heads: query head j reads key/value
 *          head j / (q_heads / heads).
 * out      [T, q_heads, head_dim] of q's type, 16-byte aligned:
 *            out = sum_t p_t V_t,  p = softmax over the visible t of scale * q . K_t
 *          A token at position i (its index in the sequence) sees t <= i, and
 *          with window > 0 only t > i - window or t < sinks (the first tokens
 *          stay visible).  A row that sees nothing gets zeros.
 * scale    finite and > 0.
 * max_new  the expected largest number of rows of a sequence: it only picks the
 *          kernel, for all of a call's sequences.  Up to 16 rows of a key/value head
 *          (max_new * q_heads / heads) the waves of a workgroup share a sequence's tokens,
 *          and these are cut into parts; above, each wave walks all tokens of its own 32 rows
 *          (16 of 256 channels), in parts only where there are few rows.  So single tokens
 *          with long contexts are far slower beside a long run than in a call of
 *          their own: give them one.
 * max_pages, the table's width, also sizes the launch: a table far wider than the
 *          sequences need costs up to a third more time.
 * Scores, the softmax's maximum and sum and the accumulators are fp32; the
 * codes enter the products exactly, and so do a query's channels down to
 * 2^-17 of its largest (smaller ones within 2^-28 of that); p_t, against zeros
 * and in the sum, and p_t * s_t, against codes, are rounded to fp16 once each.
 * Results depend on the arguments alone, not on timing.
 * workspace  kv4_attend_workspace_bytes(...) bytes, 256-byte aligned (NULL when
 *          0); nothing is kept in it between calls.  One or two kernels.     */
size_t kv4_attend_workspace_bytes(int T, int max_new, int B, int q_heads, int heads, int head_dim,
                                  int max_pages, int page_size, int window, int sinks);
int kv4_attend(const void *q, int dtype, int T, int ld_q, int q_heads, int max_new,
               const int32_t *seq_offsets, const int32_t *kv_lens, const int32_t *page_table, int B,
               int max_pages, const uint32_t *cache_k, const uint32_t *cache_v,
               const uint16_t *cache_k_sz, const uint16_t *cache_v_sz, int num_pages, int heads,
               int page_size, int head_dim, int group, float scale, int window, int sinks,
               void *out, void *workspace, size_t workspace_bytes, unsigned flags, void *stream);

/* ---- low-rank adapters of many requests beside a shared projection ----
 *   Y[t] += scaling[a] * (X[t] . A[a]^T) . B[a]^T     for the tokens t of adapter a
 * X        [T,K], A [L,R,K], B [L,N,R], Y [T,N] (read and written), all fp16 or
 *          all bf16 (dtype), 16-byte aligned; K, N, R multiples of 8, R <= 512.
 * scaling  [L] fp32, or NULL for ones.
 * adapter_offsets [L+1], row_token [T], slot_row [T]: moe_sort_rows of the
 *          tokens' adapters (topk = 1, ids outside [0, L) for tokens without
 *          one): row m of adapter a's range is token row_token[m], if
 *          slot_row[row_token[m]] is m.  Tokens without a row keep their Y.
 * Both products and their sum with Y in fp32 (X . A^T enters the second as a sum
 * of two 16-bit values: 22 bits of a row's largest for fp16, 16 for bf16), one rounding to Y's
 * type.  Y must not overlap the other tensors.
 * workspace  qg_workspace_bytes(QG_OP_LORA, T, N, K, R, L, 0) bytes, 256-byte
 *          aligned; nothing is kept in it between calls.  T == 0 does nothing.
 *          Two kernels, or three where adapters have many rows each.         */
int lora_add(const void *X, const void *A, const void *B, const float *scaling,
             const int32_t *adapter_offsets, const int32_t *row_token, const int32_t *slot_row,
             int L, int T, int K, int N, int R, int dtype, void *Y, void *workspace,
             size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMM_H */
