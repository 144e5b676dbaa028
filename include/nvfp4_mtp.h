/*
 * nvfp4_mtp.h -- C ABI of the NVFP4 W4A16 MTP draft-head library (AMD gfx950).
 *
 * The library runs the hot path of a multi-token-prediction draft head whose
 * projection, expert and LM-head weights are NVFP4: a quantizer, a W4A16
 * decode GEMV, a W4A16 GEMM for prompt-sized row counts, an LM-head GEMV fused
 * with argmax, and a top-k MoE expert FFN.  The operations are the ones the
 * following pages describe (cited by page and item):
 *   [new.rs]      spark_model/layers/mtp_head/new.rs -- `MtpHead::new`
 *   [mtp_head.rs] metrale_model_layers/layers/mtp_head.rs -- module doc,
 *                 `MtpHead` fields, `MtpHead::gemv`, `quantize_proj`
 *   [v4_mtp.rs]   spark_model/layers/deepseek_v4_mtp.rs -- `forward_one`,
 *                 `argmax_grammar_masked`
 *   [prefill.rs]  spark_model/layers/qwen3_attention/prefill_weights.rs --
 *                 `w4a16_gemm_m128_dispatch`
 *
 * Conventions shared by every entry point:
 *  - All data pointers are DEVICE pointers unless a comment says "host".
 *    The caller owns every buffer; the library allocates nothing, keeps no
 *    state between calls and is safe to call from several host threads.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Every call only
 *    enqueues work on it and returns; it never synchronizes or reads back
 *    (moe_workspace_status, a host query, is the one exception).
 *  - Return value: NVFP4_OK (0) or a negative status.  Arguments are checked
 *    on the host before anything is enqueued; on failure nothing is enqueued
 *    and nvfp4_mtp_last_error() describes the problem.
 *  - bf16 data are passed as uint16_t bit patterns.
 *
 * NVFP4 weight layout (the pages show only the packed [N, K/2] code array;
 * the rest is the public NVFP4 format): a weight W[N][K] (out = in @ W^T, the
 * convention of [mtp_head.rs] `MtpHead::gemv` and [prefill.rs]) is stored as
 *   codes [N][K/2]  u8, two E2M1 codes per byte, even k in the low nibble;
 *   scales[N][K/16] u8, one E4M3FN scale per 16 consecutive k of a row,
 *                   row-major, no swizzle (bytes 0x7F/0xFF are invalid);
 *   global          one nvfp4_global, dequantized value
 *                   W^[n][k] = e2m1(code) * e4m3(scale) * global.dec.
 */
#ifndef NVFP4_MTP_H
#define NVFP4_MTP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Per-matrix global scale, 16 bytes, device resident.  Written by
 * nvfp4_quantize: amax = max |W|, enc = 2688 / amax (0 if amax == 0, at most
 * FLT_MAX), dec = amax / 2688 (2688 = 6 * 448, the largest E2M1 value times
 * the largest E4M3 value).  flags is reserved (written 0). */
typedef struct nvfp4_global {
    float dec;
    float enc;
    float amax;
    uint32_t flags;
} nvfp4_global;

/* Host-side descriptor of one NVFP4 matrix W[n][k] (device pointers inside).
 * codes must be 16-byte aligned, scales 2-byte aligned, global 4-byte
 * aligned; k % 32 == 0; n >= 0. */
typedef struct nvfp4_weight {
    const uint8_t *codes;         /* [n][k/2]  */
    const uint8_t *scales;        /* [n][k/16] */
    const nvfp4_global *global;   /* one struct */
    int32_t n;
    int32_t k;
} nvfp4_weight;

/* Host-side descriptor of a stack of NVFP4 routed experts (the NVFP4 MoE of
 * [new.rs] `MtpHead::new`: per expert a gate and an up projection
 * [inter][hidden] and a down projection [hidden][inter]).  Expert e's gate
 * codes start at gate_codes + e * inter * hidden / 2, its scales at
 * gate_scales + e * inter * hidden / 16, its global at gate_global[e]; the
 * same for up; down uses [hidden][inter] per expert. */
typedef struct nvfp4_moe_weights {
    int32_t num_experts;   /* E, 1..1024            */
    int32_t hidden;        /* H, % 32 == 0          */
    int32_t inter;         /* I, % 32 == 0          */
    const uint8_t *gate_codes, *gate_scales;
    const nvfp4_global *gate_global;
    const uint8_t *up_codes, *up_scales;
    const nvfp4_global *up_global;
    const uint8_t *down_codes, *down_scales;
    const nvfp4_global *down_global;
} nvfp4_moe_weights;

enum {
    NVFP4_OK = 0,
    NVFP4_ERR_ARG = -1,         /* null pointer or out-of-range scalar    */
    NVFP4_ERR_SHAPE = -2,       /* k % 32 != 0, m out of range, ...       */
    NVFP4_ERR_ALIGN = -3,       /* a pointer misses its alignment         */
    NVFP4_ERR_WORKSPACE = -4,   /* workspace missing or too small         */
    NVFP4_ERR_UNSUPPORTED = -5, /* shape the kernels do not handle        */
    NVFP4_ERR_HIP = -6,         /* kernel launch failed (message has why) */
    NVFP4_ERR_DEVICE = -7       /* a kernel reported a failure (workspace status) */
};

enum { NVFP4_OUT_F32 = 0, NVFP4_OUT_BF16 = 1 };

/* Bit 0 of lmhead_gemv_argmax's flags: compare bf16-rounded logits. */
#define NVFP4_ARGMAX_BF16_KEYS 1u

/*
 * nvfp4_quantize -- the two quantizer passes [new.rs] resolves in
 * `MtpHead::new` as `nvfp4_global_absmax` and `quantize_bf16_to_nvfp4` and
 * applies to every projection, router and expert matrix (`quantize_proj` in
 * [mtp_head.rs]).
 *   w_bf16  [n][k] bf16, row-major, 16-byte aligned; finite values (with a
 *           NaN or Inf the outputs are unspecified, nothing faults).
 *   codes   out [n][k/2] (16-byte aligned); scales out [n][k/16] (2-byte
 *           aligned); global out (one struct, 16-byte aligned).
 * Pass 1: amax = max |w|.  Pass 2, per 16-element block of a row:
 *   scale = E4M3_rne_sat(fl(fl(bmax * enc) / 6)), sf = its value;
 *   inv = sf > 0 ? min(fl(enc / sf), FLT_MAX) : 0;
 *   code = E2M1 nearest to fl(w * inv), ties to the even code, saturating
 *   at 6, sign = sign of the product.
 * Requires n >= 1, k >= 32, k % 32 == 0, n * k < 2^40.  Three launches
 * (clear, absmax, encode); no workspace.
 */
int nvfp4_quantize(const uint16_t *w_bf16, int32_t n, int32_t k, uint8_t *codes,
                   uint8_t *scales, nvfp4_global *global, void *stream);

/*
 * w4a16_gemv -- decode-row W4A16 GEMV, y[m][n] = sum_k x[m][k] * W^[n][k]
 * ([mtp_head.rs] `MtpHead::gemv` -> `w4a16_decode_gemv`; its doc of the
 * batched-M tiers: one pass over the weight serves all M rows).
 *   x_bf16  [m][w->k] bf16, 16-byte aligned; m in 1..8.
 *   y       [m][w->n], fp32 (y_dtype NVFP4_OUT_F32) or bf16 rounded to
 *           nearest-even from the fp32 sum (NVFP4_OUT_BF16); 4-byte aligned.
 * fp32 accumulation; one pass over codes and scales; one launch.  The
 * activations are staged in LDS: when round_up_pow2(m) * k * 2 exceeds
 * 155648 bytes the rows go in groups of the most that fit, one pass and
 * one launch per group (k * 2 <= 155648 is required).  Large weights
 * (enough 4-, 8- or 16-row units for every wavefront of the device) run on
 * the persistent streaming grid of lmhead_gemv_argmax with plain outputs;
 * either way each output is one fp32 sum.
 */
int w4a16_gemv(const uint16_t *x_bf16, int32_t m, const nvfp4_weight *w, void *y,
               int32_t y_dtype, void *stream);

/*
 * w4a16_gemv_grouped -- the same GEMV for `count` weights that share K and
 * the activations, in one launch: y[i][m][w[i]->n] = x * W^_i transposed,
 * for i < count.  The head's q, k and v projections read one normed hidden
 * state, as do an FFN's gate and up ([new.rs] `MtpHead::new` resolves the
 * `w4a16_gemv_qg` and dual `w4a16_gemv_fused` kernels next to the plain
 * GEMV; [prefill_weights.rs] installs a fused [q|k|v] weight for prefill).
 *   w       host array of `count` descriptors (1 <= count <= 8), all with the
 *           same k; a descriptor with n == 0 contributes nothing and its
 *           output pointer is not read.
 *   y       host array of `count` device pointers, each [m][w[i]->n] of
 *           y_dtype, 4-byte aligned.
 * Each output is the fp32-accumulated product of w4a16_gemv; the order of
 * the fp32 partial sums can differ from a call for that weight alone (the
 * tile shape is chosen for the summed row count).  Outputs must not
 * overlap.  Errors as w4a16_gemv, plus NVFP4_ERR_ARG for a bad
 * count or NULL arrays and NVFP4_ERR_SHAPE for mismatched k.
 */
int w4a16_gemv_grouped(const uint16_t *x_bf16, int32_t m, const nvfp4_weight *const *w,
                       void *const *y, int32_t count, int32_t y_dtype, void *stream);

/*
 * w4a16_gemm_m128 -- W4A16 GEMM for prompt-sized row counts, the
 * `w4a16_gemm_m128_dispatch` of [prefill.rs] in its lossless form (NVFP4 ->
 * bf16 dequantization, bf16 matrix products, fp32 accumulation; activations
 * are never quantized).  y[m][n] = sum_k x[m][k] * W^[n][k].
 *   x_bf16     [m][w->k] bf16, 16-byte aligned; m >= 1 (any m; work is tiled
 *              in 128- or 256-row blocks, a ragged last block is masked).
 *   y          [m][w->n] fp32 or bf16 (y_dtype), 4-byte aligned.
 *   workspace  NULL, or 16-byte aligned device scratch of at least
 *              w4a16_gemm_m128_workspace_bytes(m, w->n, w->k) bytes.  When
 *              the output tiles are too few to fill the device, or a last
 *              round of them would leave most of it idle, K of those tiles
 *              is cut into slices whose fp32 partial sums go to the
 *              workspace and are added in slice order by a second kernel
 *              (the same order on every call).  NULL: one pass over K.
 *              Nothing needs to be initialised; calls that overlap on one
 *              workspace race.
 * Any n >= 0; rows and columns outside the tiles are masked.  Errors:
 * NVFP4_ERR_WORKSPACE for a non-NULL workspace below the size needed, and
 * those of w4a16_gemv.
 */
size_t w4a16_gemm_m128_workspace_bytes(int32_t m, int32_t n, int32_t k);
int w4a16_gemm_m128(const uint16_t *x_bf16, int32_t m, const nvfp4_weight *w, void *y,
                    int32_t y_dtype, void *workspace, size_t ws_bytes, void *stream);

/*
 * lmhead_gemv_argmax -- LM-head GEMV over the first V vocabulary rows fused
 * with argmax: the draft-token selection of [v4_mtp.rs] `forward_one` (LM
 * head, then argmax) and of the NVFP4 LM head of [new.rs], with the reduced
 * vocabulary of [new.rs] / [v4_mtp.rs] (V = min(vocab_rows, w->n), 0 = all).
 * No logits tensor is written.
 *   h_bf16   [m][w->k] bf16, 16-byte aligned; m in 1..8.
 *   out_idx  [m] int32: the lowest index i < V whose key is the maximum,
 *            where key = logit (fp32), or the logit rounded to bf16 when
 *            flags & NVFP4_ARGMAX_BF16_KEYS.  The selection follows the
 *            ascending strict-greater scan of [v4_mtp.rs]
 *            `argmax_grammar_masked`: NaN never wins, -0 == +0, and if no
 *            key exceeds -inf the index is 0.
 *   out_max  [m] fp32: the fp32 logit of the selected row.
 *   workspace device scratch of at least
 *            lmhead_gemv_argmax_workspace_bytes(m, V) bytes (V = the number
 *            of rows scored), 256-byte aligned.  It holds a ticket counter
 *            and per-row packed maxima that must be zero before the first
 *            call (zero-fill the buffer once); each call returns them to
 *            zero (and lmhead_gemv_argmax_fc's call count, which only
 *            advances).  A workspace serves one call at a time: calls that
 *            overlap on one workspace race, and can leave the ticket off
 *            zero, which makes later calls wrong; zero-fill it again after
 *            such an overlap.
 * Rows with equal codes and scales produce bit-identical logits.  One launch.
 */
size_t lmhead_gemv_argmax_workspace_bytes(int32_t m, int32_t vocab_rows);
int lmhead_gemv_argmax(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w,
                       int32_t vocab_rows, int32_t *out_idx, float *out_max, void *workspace,
                       size_t ws_bytes, uint32_t flags, void *stream);

/*
 * lmhead_gemv_argmax_noalloc -- lmhead_gemv_argmax for callers that cannot
 * allocate device memory (code under graph capture, tight serving loops,
 * harnesses that forbid allocation): the same kernels and results, with the
 * workspace in a static array of the library, one copy of
 * NVFP4_NOALLOC_SCRATCH_BYTES per device, held until the process ends.  The
 * first call on a device looks the array up and clears its counters (a
 * kernel on `stream`); every call returns them to zero.  All calls on one
 * device share the array: calls that overlap on a device race (one at a
 * time per device, as with one workspace).  The grid is the device's
 * resident LM-head workgroups, each with m partials of 32 bytes; a grid
 * whose 512 + 32 * round_up(m) * workgroups bytes exceed the array is
 * refused with NVFP4_ERR_WORKSPACE (256 CUs need at most 131,584 bytes).
 * Allocates nothing (no hipMalloc, no allocating library routine).
 * Arguments, outputs and the other errors as lmhead_gemv_argmax.
 */
#define NVFP4_NOALLOC_SCRATCH_BYTES (1u << 20)
int lmhead_gemv_argmax_noalloc(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w,
                               int32_t vocab_rows, int32_t *out_idx, float *out_max, uint32_t flags,
                               void *stream);

/*
 * lmhead_gemv_argmax_logprob -- lmhead_gemv_argmax that also returns, per
 * activation row, the top-1 log-probability of the selected token: the
 * batched argmax of [mtp_head.rs] (`MtpHead` fields) that writes each row's
 * top-1 log-probability for the draft confidence stop.  In the same pass over
 * the weights (no extra bytes read) each slot keeps an online log-sum-exp of
 * the keys, merged with the argmax partials:
 *   out_logprob[i] = key[out_idx[i]] - log(sum over r < V of exp(key[r]))
 * in fp32, with the keys of lmhead_gemv_argmax (fp32 logits, or their bf16
 * rounding with NVFP4_ARGMAX_BF16_KEYS).  A NaN or +inf key, or a vocabulary
 * whose keys are all -inf, gives NaN.  All other arguments, the workspace
 * (the same size) and the errors as lmhead_gemv_argmax; out_logprob [m] fp32,
 * 4-byte aligned, must not be NULL.  One launch.
 */
int lmhead_gemv_argmax_logprob(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w,
                               int32_t vocab_rows, int32_t *out_idx, float *out_max,
                               float *out_logprob, void *workspace, size_t ws_bytes,
                               uint32_t flags, void *stream);

/*
 * lmhead_gemv_argmax_masked -- lmhead_gemv_argmax restricted to the tokens a
 * grammar allows: the device-side form of the masked argmax of [v4_mtp.rs]
 * `argmax_grammar_masked`, which needs no logits readback.
 *   allow_mask    device uint32 [m][mask_words]: token r is allowed for
 *                 activation row i when bit r % 32 of word r / 32 of row i is
 *                 set; tokens past the mask are not allowed.  4-byte aligned.
 *   out_logprob   NULL, or [m] fp32: the top-1 log-probability over the
 *                 allowed tokens (key[idx] minus the log-sum-exp of the
 *                 allowed keys); NaN when no allowed key has finite mass.
 * A disallowed token is scored as a -inf key, so the scan of
 * lmhead_gemv_argmax applies: the lowest-index maximum among the allowed
 * tokens, and index 0 (with row 0's logit in out_max) when nothing allowed
 * exceeds -inf, including an empty allowed set -- the pad draft of the scan.
 * Workspace, errors and the other arguments as lmhead_gemv_argmax.  One
 * launch; the mask word of each 32-row tile is loaded with its weights.
 */
int lmhead_gemv_argmax_masked(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w,
                              int32_t vocab_rows, const uint32_t *allow_mask, int32_t mask_words,
                              int32_t *out_idx, float *out_max, float *out_logprob,
                              void *workspace, size_t ws_bytes, uint32_t flags, void *stream);

/*
 * lmhead_gemv_argmax_fc -- the end of one draft step and the start of the
 * next: lmhead_gemv_argmax, then the next step's fc over the chosen
 * tokens' embedding rows, y = w4a16_gemv_embed(out_idx, table, x_rest, fc)
 * ([v4_mtp.rs] `propose` feeds each draft into the next step's input;
 * [mtp_head.rs] `MtpHead` fields: `embed_from_argmax`, the fc).
 *   h_bf16 ... flags          as lmhead_gemv_argmax (out_idx, out_max are
 *                             its outputs, bit for bit).
 *   table_bf16, table_vocab, hidden, x_rest_bf16, fc, y, y_dtype
 *                             as w4a16_gemv_embed with idx = out_idx.
 * At one row with K = 2048 and an fc of k = 2048 or 4096, and when the LM
 * head's grid can take every fc row (wavefronts 1..7 of each workgroup, two
 * rows each: 14 rows a workgroup, 3584 on 256 CUs), one launch: the
 * LM head's workgroups load their fc rows while its end chain runs, wait
 * (bounded, about a second) for the last workgroup to publish the id in the
 * workspace, gather its embedding row and finish the fc.  y then sums each
 * row in another order than w4a16_gemv_embed (equal up to fp32 rounding;
 * bit for bit on exactly representable sums), and is NaN if that wait gave
 * up.  The whole grid must be resident at once (the persistent LM-head grid
 * is sized so).  Otherwise the two calls, in order.  The workspace is
 * lmhead_gemv_argmax's; every call advances a count in it.
 */
int lmhead_gemv_argmax_fc(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w, int32_t vocab_rows,
                          int32_t *out_idx, float *out_max, void *workspace, size_t ws_bytes, uint32_t flags,
                          const uint16_t *table_bf16, int32_t table_vocab, int32_t hidden,
                          const uint16_t *x_rest_bf16, const nvfp4_weight *fc, void *y, int32_t y_dtype,
                          void *stream);

/*
 * embed_from_argmax -- the draft tokens' embedding rows, gathered on the
 * device: the `embed_from_argmax` step of [mtp_head.rs] (`MtpHead` fields),
 * which feeds the next draft step and stores the draft id in device memory
 * for deferred readback, so that a chain of draft steps needs no host round
 * trip ([v4_mtp.rs] `propose` feeds each draft into the next step).
 *   idx         device int32 [m] (e.g. out_idx of lmhead_gemv_argmax).
 *   table_bf16  device bf16 [vocab][hidden], 16-byte aligned; hidden % 8 == 0.
 *   out_bf16    device bf16, row i at out_bf16 + i * out_stride (elements;
 *               out_stride >= hidden, a multiple of 8), 16-byte aligned --
 *               e.g. the first half of the next step's fc input row.
 *   id_log      NULL, or device int32 [m]: receives idx (the chain's record).
 * An index outside [0, vocab) gives a zero row (id_log still records it).
 * m == 0 does nothing.  One launch.
 */
int embed_from_argmax(const int32_t *idx, int32_t m, const uint16_t *table_bf16, int32_t vocab,
                      int32_t hidden, uint16_t *out_bf16, int64_t out_stride, int32_t *id_log,
                      void *stream);

/*
 * lmhead_gemv_argmax_embed -- the LM head's argmax with the embedding gather
 * of the selected tokens done by its last workgroup: one launch for the tail
 * of a draft step and the head of the next (the gather of embed_from_argmax
 * without a kernel boundary or a second read of the index).
 *   allow_mask, mask_words   as lmhead_gemv_argmax_masked, or NULL / 0.
 *   out_logprob              NULL, or as lmhead_gemv_argmax_logprob.
 *   table_bf16, table_vocab, hidden, out_embed, out_stride, id_log
 *                            as embed_from_argmax (table_vocab may differ
 *                            from the head's rows; hidden % 8 == 0).
 * out_idx, out_max, the workspace and the errors as lmhead_gemv_argmax.
 */
int lmhead_gemv_argmax_embed(const uint16_t *h_bf16, int32_t m, const nvfp4_weight *w,
                             int32_t vocab_rows, const uint32_t *allow_mask, int32_t mask_words,
                             int32_t *out_idx, float *out_max, float *out_logprob,
                             const uint16_t *table_bf16, int32_t table_vocab, int32_t hidden,
                             uint16_t *out_embed, int64_t out_stride, int32_t *id_log,
                             void *workspace, size_t ws_bytes, uint32_t flags, void *stream);

/*
 * w4a16_gemv_embed -- w4a16_gemv whose activation rows begin with the
 * embedding rows of the tokens in idx, read by the GEMV itself: the next
 * draft step's fc over [embed(draft token) | hidden state] with the gather of
 * embed_from_argmax ([mtp_head.rs] `MtpHead` fields; [v4_mtp.rs] `propose`
 * feeds each draft into the next step) folded into its activation loads, so
 * the embedding row is fetched while the weights stream and no kernel
 * writes it.  Activation row i, element kk: table[idx[i]][kk] for kk <
 * hidden (a zero row for an id outside [0, table_vocab)), x_rest[i][kk -
 * hidden] for kk >= hidden.
 *   idx          device int32 [m] (e.g. out_idx of lmhead_gemv_argmax).
 *   table_bf16   device bf16 [table_vocab][hidden], 16-byte aligned;
 *                hidden a positive multiple of 32, at most w->k.
 *   x_rest_bf16  device bf16 [m][w->k - hidden], 16-byte aligned (NULL
 *                when hidden == w->k).
 *   m, w, y, y_dtype, stream, the kernels and the other errors as
 *                w4a16_gemv; the result equals w4a16_gemv of the
 *                concatenated rows bit for bit.
 */
int w4a16_gemv_embed(const int32_t *idx, const uint16_t *table_bf16, int32_t table_vocab,
                     int32_t hidden, const uint16_t *x_rest_bf16, int32_t m, const nvfp4_weight *w,
                     void *y, int32_t y_dtype, void *stream);

/*
 * moe_w4a16_gemv -- routed-expert MoE FFN for decode rows: the
 * `moe_topk_softmax` -> `moe_silu_mul` -> weighted-sum chain named in
 * [new.rs] `MtpHead::new`, on NVFP4 experts.
 *   x_bf16         [m][H] bf16, 16-byte aligned; m in 1..8.
 *   router_logits  [m][E] fp32 (the router projection's output).
 *   top_k          1..min(E, 16).
 *   y              out [m][H] fp32: sum_j w[j] * down_e(j)(a_j), summed
 *                  in fp32 in an order fixed by the routing (the same
 *                  inputs give the same bits).
 *   topk_ids       out [m][top_k] int32: experts by descending logit, the
 *                  lower id first among equal logits.
 *   topk_w         out [m][top_k] fp32: softmax over the selected logits.
 *   workspace      at least moe_w4a16_gemv_workspace_bytes(m, top_k, e),
 *                  256-byte aligned, zero-filled before its first use (it
 *                  holds ticket and column counters, which every call
 *                  returns to zero, per-call tagged hand-off words and a
 *                  sticky status word: see moe_workspace_status).  One
 *                  call at a time per workspace.
 * Per selected expert: g = gate x, u = up x (fp32),
 * a = bf16_rne(silu(g) * u), d = down a (fp32).  The gate/up weights are
 * read once per (row, slot) pair, the down weights once per distinct expert.
 * Requires H, I % 32 == 0
 * and round_up(m, 1|2|4|8) * max(H, I) * 2 <= 159744 bytes of LDS (H up to
 * 9984 at m = 8); NVFP4_ERR_UNSUPPORTED otherwise.  One launch at one
 * token when the down pass's activation rows fit in LDS and the whole grid
 * is resident at once (decode at the usual shapes); else gate/up (with the
 * routing), then the down pass with the combine.
 */
size_t moe_w4a16_gemv_workspace_bytes(int32_t m, int32_t top_k, const nvfp4_moe_weights *e);
int moe_w4a16_gemv(const uint16_t *x_bf16, int32_t m, const float *router_logits,
                   int32_t top_k, const nvfp4_moe_weights *e, float *y, int32_t *topk_ids,
                   float *topk_w, void *workspace, size_t ws_bytes, void *stream);

/*
 * moe_w4a16_gemv_trace -- moe_w4a16_gemv in its one-launch form with phase
 * timestamps, for profiling the one-token latency chain; the outputs are
 * those of moe_w4a16_gemv bit for bit.  Not a second computation: the same
 * kernel, given a trace buffer.
 *   m              1 (NVFP4_ERR_UNSUPPORTED otherwise, and when the call
 *                  would not take the one-launch form).
 *   trace          device uint64[trace_words], 8-byte aligned, at least
 *                  moe_w4a16_gemv_trace_words(m, top_k, e) words (0 when m
 *                  != 1); out: event ev of workgroup b at trace[ev * G + b],
 *                  G = ceil(I / 16) * top_k gate/up workgroups followed by
 *                  ceil(H / 8) down workgroups, each the GPU's 100 MHz
 *                  constant clock (s_memrealtime) read by the workgroup's
 *                  first thread.  Gate/up events: 0 start, 1 routing done,
 *                  2 activations stored, 3 counted in its column (the last
 *                  of a column: after issuing the release).  Down events:
 *                  0 start, 1 weight loads issued, 2 go word seen,
 *                  3 activations staged, 4 sums done, 5 output written.
 *                  Unused slots are left as they were.
 *   the other arguments and errors as moe_w4a16_gemv.
 */
size_t moe_w4a16_gemv_trace_words(int32_t m, int32_t top_k, const nvfp4_moe_weights *e);
int moe_w4a16_gemv_trace(const uint16_t *x_bf16, int32_t m, const float *router_logits,
                         int32_t top_k, const nvfp4_moe_weights *e, float *y, int32_t *topk_ids,
                         float *topk_w, void *workspace, size_t ws_bytes, uint64_t *trace,
                         size_t trace_words, void *stream);

/*
 * moe_layer_w4a16 -- the complete MoE layer of the draft head: the NVFP4
 * router (`moe_gate`, quantized next to the experts in [new.rs]
 * `MtpHead::new`), the routed experts of moe_w4a16_gemv and the shared
 * expert with its sigmoid `shared_expert_gate`, blended as the pages'
 * `moe_weighted_sum_blend`:
 *   router_logits = router x  (fp32 out [m][E]),
 *   y = sum_j w[j] * down_e(j)(a_j) + sigmoid(g . x) * down_s(a_s),
 *   a_s = bf16(silu(gate_s x) * up_s x),
 * with g = shared_gate_w_bf16 ([H] bf16) or, when it is NULL, a factor 1.
 *   router        [E][H] NVFP4 (n = num_experts, k = hidden).
 *   shared_gate, shared_up   [I][H] NVFP4; shared_down [H][I] NVFP4 (the
 *                 routed experts' width I).
 *   y, topk_ids, topk_w      as moe_w4a16_gemv.
 *   workspace     at least moe_layer_w4a16_workspace_bytes(m, top_k, e),
 *                 256-byte aligned, zero-filled before its first use.
 * Three launches: one grouped GEMV (router, shared gate, shared up), the
 * routing with the routed gate/up and the shared activations, and the down
 * pass over the routed experts and the shared one.  Requires, besides the
 * limits of moe_w4a16_gemv, (m * top_k + m) * I * 2 <= 153600 bytes (the
 * activation rows the down pass keeps in LDS); NVFP4_ERR_UNSUPPORTED
 * otherwise.
 */
size_t moe_layer_w4a16_workspace_bytes(int32_t m, int32_t top_k, const nvfp4_moe_weights *e);
int moe_layer_w4a16(const uint16_t *x_bf16, int32_t m, const nvfp4_weight *router, int32_t top_k,
                    const nvfp4_moe_weights *e, const nvfp4_weight *shared_gate,
                    const nvfp4_weight *shared_up, const nvfp4_weight *shared_down,
                    const uint16_t *shared_gate_w_bf16, float *y, int32_t *topk_ids, float *topk_w,
                    float *router_logits, void *workspace, size_t ws_bytes, void *stream);

/*
 * moe_workspace_status -- reads and clears the sticky status word of a
 * moe_w4a16_gemv / moe_layer_w4a16 workspace.  In the one-launch path the
 * down workgroups wait (bounded, about a second) for the gate/up workgroups
 * of the same launch, released through per-workgroup go words that carry
 * a per-call tag (a release left over from an earlier call never satisfies
 * a later wait).  If a wait gives up, or a go word holds a value no call
 * writes (the workspace was overwritten), that down workgroup writes NaN
 * rows into y and sets bit 0 (timeout) or bit 1 (overwritten) of this
 * word; the call itself has already returned NVFP4_OK.
 *   workspace  the MoE workspace (device), ws_bytes its size.
 *   status     host uint32: receives the bits (0 after clean calls).
 * Synchronizes `stream` (not allowed during graph capture:
 * NVFP4_ERR_UNSUPPORTED).  Returns NVFP4_OK when no bit was set, else
 * NVFP4_ERR_DEVICE with the reason in nvfp4_mtp_last_error(); an
 * overwritten workspace must be zero-filled again before its next use.
 */
int moe_workspace_status(void *workspace, size_t ws_bytes, uint32_t *status, void *stream);

/* ---- attention of the draft step: rotary positions and an 8-bit cache ----
 *
 * The steps between q|k|v and o in the draft step ([new.rs] `MtpHead::new`
 * resolves handles for them; the pages give no formulas, so the definitions here
 * are the library's own).
 *
 * Strided rows of heads (host descriptor): element d of head h of row r is
 * data[r * row_stride + h * head_stride + d], strides in elements (a
 * head_stride of 2 * dim reads the q halves of a gated q projection in
 * place).  data 16-byte aligned, both strides multiples of 8, head_stride >=
 * dim, row_stride >= 0.  Outputs of two rows or more: also row_stride >= (heads -
 * 1) * head_stride + dim (token by token), or row_stride >= dim and head_stride >=
 * (rows - 1) * row_stride + dim (head by head): no two share an element. */
typedef struct nvfp4_head_rows {
    uint16_t *data;       /* bf16 */
    int64_t row_stride, head_stride;
    int32_t heads, dim;
} nvfp4_head_rows;

/* Rotary positions (host descriptor).  Pair i < rot_dim / 2 of a row at
 * position p turns by the angle p * inv_freq[i] (computed in fp64, so far
 * positions keep their phase): (x, y) -> (x cos - y sin, x sin + y cos) *
 * mscale.  The pair is (i, i + rot_dim / 2) or, with interleaved != 0,
 * (2i, 2i + 1); elements from rot_dim on are copied.  Scaling for long
 * contexts is in the table and mscale.  rot_dim: a positive multiple of 16,
 * at most the rows' dim; inv_freq: device fp64 [rot_dim / 2], 8-byte aligned,
 * radians per position. */
typedef struct nvfp4_rope {
    const double *inv_freq;
    int32_t rot_dim;
    int32_t interleaved;
    float mscale;
} nvfp4_rope;

/* A paged 8-bit KV cache (host descriptor, device pointers).  Codes are
 * E4M3FN; scale byte b stands for 2^(b - 127) (bytes above 246 read as 246, so
 * that every value is finite in bf16), one per (page, head) and for K and V
 * each; kv8_append writes 17 to 246.  V lies transposed inside its page, so that
 * the attention's matrix operands load straight from it.
 * codes 16-byte aligned; page_tokens 16, 32, 64 or 128; head_dim 64, 128, 192
 * or 256; kv_heads >= 1; num_pages >= 1. */
typedef struct nvfp4_kv8_cache {
    uint8_t *k_codes;     /* [num_pages][kv_heads][page_tokens][head_dim] */
    uint8_t *k_scales;    /* [num_pages][kv_heads] */
    uint8_t *v_codes;     /* [num_pages][kv_heads][head_dim][page_tokens] */
    uint8_t *v_scales;    /* [num_pages][kv_heads] */
    int32_t num_pages, page_tokens, kv_heads, head_dim;
} nvfp4_kv8_cache;

/* A ragged batch over such a cache (host descriptor, device pointers, 4-byte
 * aligned).  Sequence b owns rows [cu_rows[b], cu_rows[b + 1]) of the call's
 * `rows` rows: the last n_b of its kv_lens[b] tokens, row i at position
 * kv_lens[b] - n_b + i.  Token t lies in page block_table[b][t / page_tokens].
 *   max_rows    host bound of n_b: rows of a sequence past it are not
 *               computed.
 *   max_kv_len  host bound of kv_lens, or 0 for max_pages * page_tokens; a
 *               longer sequence is still handled, less evenly split.
 * Values on the device that make no sense are bounded there: row ranges are
 * cut to [0, rows), lengths to [0, max_pages * page_tokens]; rows at negative
 * positions and tokens whose page id is outside [0, num_pages) are not
 * written, not read (zero rows) and not attended to. */
typedef struct nvfp4_kv8_seqs {
    const int32_t *cu_rows;       /* [batch + 1] */
    const int32_t *kv_lens;       /* [batch] */
    const int32_t *block_table;   /* [batch][max_pages] */
    int32_t batch, rows, max_rows, max_pages, max_kv_len;
} nvfp4_kv8_seqs;

/*
 * rope_qk -- rotary positions of q and k rows.
 *   q, q_out    rows before and after (the same shape; q_out may be q itself:
 *               then only the rotated elements are written; otherwise the
 *               two must not overlap).  NULL with q_out NULL: no q.
 *   k, k_out    the same for k; at least one of q and k.
 *   rows        rows of each (0 does nothing).
 *   positions   device int32 [rows], 4-byte aligned, any values.
 * Products and sums in fp64, rounded to fp32 and that to bf16.  dim % 8 == 0.
 * One launch.
 */
int rope_qk(const nvfp4_head_rows *q, const nvfp4_head_rows *q_out, const nvfp4_head_rows *k,
            const nvfp4_head_rows *k_out, int32_t rows, const int32_t *positions, const nvfp4_rope *rope,
            void *stream);

/*
 * kv8_append -- quantises the rows' k and v into the cache at their positions.
 *   k, v   [rows][kv_heads][head_dim] head rows.
 * Per page and head, over the tokens of the page that this call writes: amax =
 * max of the finite |x|; e = the smallest exponent >= -110 with amax <= 448 *
 * 2^e, 119 at most (values above 448 * 2^119 = 2.98e38 saturate).  A page that
 * the call writes from its first token on takes e; a page it continues takes
 * max(e, its present exponent), and when that grows the page's earlier codes are
 * re-rounded to it.  code = E4M3 nearest to x * 2^-e (ties
 * to even, saturating at 448; infinities saturate, NaN stays NaN).  Powers of
 * two leave every kept value exact unless it falls among the subnormals.
 * Writing the same rows again gives the same page.  After a shortened
 * sequence the next call overwrites the dropped tokens.  A page written by
 * the call must belong to one sequence only, and no page may occur twice in a
 * sequence's written range (else its content is unspecified).  One launch.
 */
int kv8_append(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_head_rows *k,
               const nvfp4_head_rows *v, void *stream);

/*
 * rope_kv8_append -- rope_qk of q and k at the rows' positions in their
 * sequences, then kv8_append of the rotated k (rounded to bf16, as rope_qk
 * writes it) and v, in one launch: q_out and the cache are bit for bit those
 * of the two calls.  The rotated k is not stored in bf16.  q and q_out may
 * both be NULL.  Rows of q outside every sequence are not written; those at
 * negative positions turn by them.
 */
int rope_kv8_append(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_rope *rope,
                    const nvfp4_head_rows *q, const nvfp4_head_rows *q_out, const nvfp4_head_rows *k,
                    const nvfp4_head_rows *v, void *stream);

/*
 * kv8_read -- the cache's values back in bf16 (a code times a power of two:
 * exact for scale bytes from 17 on) for the last n_b tokens of each sequence.
 *   k_out, v_out   [rows][kv_heads][head_dim] head rows; one may be NULL.
 *                  Tokens whose page id is out of range and rows at negative
 *                  positions become zero rows; rows outside every sequence
 *                  are left as they were.
 * One launch.
 */
int kv8_read(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, const nvfp4_head_rows *k_out,
             const nvfp4_head_rows *v_out, void *stream);

/*
 * kv8_attention -- attention of the rows' q heads over the cache,
 * out = softmax(scale * q k^T) v, q head h reading kv head h / (q_heads /
 * kv_heads).  The row at position p sees the tokens t <= p and, with window >
 * 0, of those the last `window` (itself included) and the first `sinks`.  Call
 * it after the rows' own k and v are appended.
 *   q           [rows][q_heads][head_dim] head rows; q_heads a multiple of
 *               kv_heads.
 *   scale       any factor (below 2.3e38, times log2(e) finite in fp32; 0: a
 *               plain mean);
 *               window, sinks >= 0 (sinks without a window changes nothing).
 *   out         bf16, row r head h at out + r * out_row_stride + h * head_dim
 *               (the o projection's activation row), 16-byte aligned,
 *               out_row_stride a multiple of 8, >= q_heads * head_dim;
 *               must not overlap q.
 *               A row that sees no token becomes zero; rows outside every
 *               sequence are left as they were.
 *   workspace   kv8_attention_workspace_bytes(cache, seqs, q_heads) bytes,
 *               256-byte aligned; nothing to initialise; one call at a time
 *               per workspace.  The size depends only on the host fields of
 *               the descriptors.
 * Scores, softmax statistics and sums in fp32 (q k^T and its differences within a
 * row below 3.4e38); weights are rounded to bf16 for the product with v and for
 * their sum.  An average of finite values is finite; beside V pages with values
 * above 2^88, terms below 2^-86 may be lost.  What a row does not see never reaches
 * it, NaN included.  The result is the same on every call with the same arguments
 * on the same device.  One or two launches.  Where a sequence has more than 64 rows
 * a kv head, row tiles and key splits go by that sequence: single rows over long
 * caches are faster in a call of their own than beside a prompt chunk.
 */
size_t kv8_attention_workspace_bytes(const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, int32_t q_heads);
int kv8_attention(const nvfp4_head_rows *q, const nvfp4_kv8_cache *cache, const nvfp4_kv8_seqs *seqs, float scale,
                  int32_t window, int32_t sinks, uint16_t *out, int64_t out_row_stride, void *workspace,
                  size_t ws_bytes, void *stream);

/*
 * verify_drafts -- which drafted tokens stand, and the token after them, from
 * the target's logits and given random numbers (the step after [v4_mtp.rs]
 * `propose`; `after_verify` then trims the cache).  Sequence b owns rows
 * [cu_rows[b], cu_rows[b + 1]) of `rows` rows, n_b of them: row i holds the
 * target's logits after i of its n_b - 1 drafts, and draft_ids[row] the draft
 * that follows the row (not read for a sequence's last row).
 *   logits       [rows] x vocab of logits_dtype (NVFP4_OUT_F32 or
 *                NVFP4_OUT_BF16), row r at r * row_stride elements
 *                (row_stride >= vocab), aligned to its element.  vocab
 *                1..2^24.
 *   draft_logits NULL: the drafts were chosen outright (the LM head's argmax).
 *                Else the rows of the draft's logits, same type and stride
 *                draft_stride: the draft of row r was sampled from row r.
 *   max_rows     host bound of n_b, 1..64; a longer sequence is cut to it.
 *   temperature  NULL (1), or device fp32 [batch]: divides both models'
 *                logits; 0, below 0 or not finite means greedy.
 *   u_accept     device fp32 [rows], u_sample device fp32 [batch]: random
 *                numbers in [0, 1).
 *   kv_lens      NULL, or device int32 [batch]: cache lengths with the
 *                sequence's n_b rows appended.
 * With p the target's softmax of a row and q the draft's (1 at the draft for
 * outright drafts), draft d stands when u_accept * q(d) < p(d); greedily, when
 * it is the row's first maximum.  At the first row whose draft falls, the token
 * is drawn from max(p - q, 0), or from p after the last draft: the lowest i
 * whose running sum exceeds u_sample times the whole (greedily: the first
 * maximum; from p should the difference vanish everywhere).  Softmax, sums and
 * comparisons in fp64.  A draft id outside [0, vocab) falls.  A target row
 * without a finite sum (NaN, +inf, or nothing above -inf) is taken greedily by
 * the scan of lmhead_gemv_argmax; such a draft row counts as an outright draft.
 *   out_accepted [batch] int32: drafts that stand.
 *   out_tokens   [rows] int32: the standing drafts, the drawn token, then -1;
 *                rows outside every sequence or past max_rows are left as they
 *                were.
 *   out_next     [batch] int32: the drawn token (-1 for a sequence without
 *                rows).
 *   out_kv_lens  [batch] int32 (with kv_lens; may be kv_lens itself): the
 *                lengths without the rows of fallen drafts, kv_lens - n_b +
 *                accepted + 1.
 *   workspace    verify_drafts_workspace_bytes(batch, max_rows, vocab,
 *                draft_logits != NULL) bytes, 16-byte aligned; nothing to
 *                initialise; one call at a time per workspace.
 * int32 and fp32 arrays 4-byte aligned.  Two launches (few rows of outright
 * drafts) or four.
 */
size_t verify_drafts_workspace_bytes(int32_t batch, int32_t max_rows, int32_t vocab, int32_t with_draft_logits);
int verify_drafts(const void *logits, int32_t logits_dtype, int64_t row_stride, int32_t vocab, const void *draft_logits,
                  int64_t draft_stride, const int32_t *cu_rows, int32_t batch, int32_t rows, int32_t max_rows,
                  const int32_t *draft_ids, const float *temperature, const float *u_accept, const float *u_sample,
                  const int32_t *kv_lens, int32_t *out_accepted, int32_t *out_tokens, int32_t *out_next,
                  int32_t *out_kv_lens, void *workspace, size_t ws_bytes, void *stream);

/* Message of the last failing call on this host thread ("" if none); the
 * pointer stays valid until the next call on the same thread. */
const char *nvfp4_mtp_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MTP_H */
