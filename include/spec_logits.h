/*
 * spec_logits.h -- C ABI of the operators that stand between a model and the
 * verify / sampling calls of spec_verify.h, on MI355X (gfx950):
 *
 *   spec_logits_w4        logits from hidden states and a head of 4-bit weights
 *                         with group scales
 *   spec_process_logits   penalties for repeated tokens, biases and grammar
 *                         masks on logits, position by position of a draft
 *   spec_history_append,  the state of the penalties: which tokens a sequence
 *   spec_history_reset    holds, and how often
 *
 * A round of speculative decoding calls them in this order: the drafter's
 * hidden state -> spec_logits_w4 -> spec_process_logits -> spec_sample, once
 * per draft; the target's hidden states -> spec_logits_w4 ->
 * spec_process_logits -> spec_verify -> spec_history_append of its output
 * tokens.
 *
 * Conventions are those of spec_verify.h: device pointers are the caller's,
 * dense and row-major; work is enqueued on `stream` (a hipStream_t of the
 * current device, NULL = the default stream) and runs asynchronously, with no
 * host synchronisation and no allocation, so every call may be captured into a
 * HIP graph, and calls on different streams are independent as far as their
 * buffers are.  Argument errors are returned (SV_ERR_*) before
 * anything is enqueued.  Types are SV_BF16 and SV_FP32.  Bad data never makes
 * a kernel read or write outside the arrays; what it gives is said at each
 * call.
 */
#ifndef SPEC_LOGITS_H
#define SPEC_LOGITS_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (checked synchronously). */
#define SL_MAX_K 65536         /* contraction length of spec_logits_w4           */
#define SL_MAX_ROWS (1 << 20)  /* rows of one call                               */
#define SL_MAX_DRAFT 64        /* draft tokens per sequence                      */
#define SL_MAX_BIAS 1024       /* bias entries per sequence                      */
#define SL_MAX_MASKS (1 << 20) /* rows of the mask table                         */

/*
 * out[r][n] = round( sum_g scales[n][g] * sum_{k in group g} (w[n][k] - zeros[n][g]) * hidden[r][k] ).
 *
 *  hidden   [R][K] bf16 or fp32 (hidden_dtype), 16-byte aligned.
 *  weights  [N][K/2] bytes, 16-byte aligned: byte j of row n holds w[n][2j] in its low and
 *           w[n][2j+1] in its high four bits, each 0..15.
 *  scales   [N][K/group] bf16 or fp32 (scale_dtype), aligned to its element; finite, below 2^124.
 *  zeros    [N][K/group] bytes, each 0..15 (the low four bits are used), or NULL: 8 everywhere.
 *  group    values of k that share a scale: 32, 64 or a multiple of 128; K is a multiple of it.
 *  R, K, N  R >= 0 and <= SL_MAX_ROWS (R == 0 is a no-op), 32 <= K <= SL_MAX_K, 1 <= N <= SV_MAX_VOCAB.
 *           R * N and R * K below 2^34 (SV_ERR_UNSUPPORTED beyond).
 *  out      [R][N] bf16 or fp32 (out_dtype), aligned to its element; overlaps no input (SV_ERR_ARG).
 *
 *  workspace  device buffer of spec_logits_w4_workspace_bytes(hidden_dtype, group, R, K) bytes,
 *           256-byte aligned (NULL where that is 0, as it is for few rows); it needs no
 *           preparation and holds nothing after the call.  Calls that share one must be ordered.
 *
 * The products w x are exact.  Sums are held in float32, those of the weights
 * and of the zero points apart within 256 values of k, and rounded once, to
 * nearest even, at the end: the error is that of a float32 product.  A row of
 * `hidden` with a NaN or an infinity gives a row of NaN (which the verify
 * reports as invalid); other rows are not affected.  A value of `hidden` beyond
 * 2^115 may give NaN too, because the sums inside a group are formed before its
 * scale.
 * Returns SV_OK or a negative code (nothing enqueued).
 */
size_t spec_logits_w4_workspace_bytes(int hidden_dtype, int group, int R, int K);
int spec_logits_w4(const void* hidden, int hidden_dtype, const uint8_t* weights, const void* scales, int scale_dtype,
                   const uint8_t* zeros, int group, int R, int K, int N, void* out, int out_dtype, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * The token history of S sequences (slots) over a vocabulary of V, in three
 * arrays that the caller owns and clears to zero once (all three; `ids` may
 * hold anything):
 *
 *  counts [S][V] int32: bit 31 set if the token is in the slot's prompt, the low 31 bits the
 *         number of times it was output; 0 for a token that the slot has never held.
 *  ids    [S][V] int32: ids[s][0..num[s]) are the tokens with counts[s][v] != 0, each once, in no
 *         particular order.
 *  num    [S] int32.
 *
 * spec_history_append adds tokens to slots: with prompt != 0 as prompt tokens
 * (bit 31), else as output tokens (one count for each time).
 *  slots   [B] int32, or NULL: sequence b is slot b (then B <= S).  A slot outside [0, S) is
 *          skipped.  A slot may appear more than once: its tokens all arrive.
 *  tokens  [B][T] int32.  A token outside [0, V) is skipped, so that the verify's out_tokens,
 *          padded with -1, go in as they are.
 * 1 <= T <= 2^24, B >= 0, S >= 0, 1 <= V <= SV_MAX_VOCAB.
 *
 * spec_history_reset empties slots: clears the counts of the tokens that the
 * slot lists and sets num to 0.  slots as above (a repeated slot is emptied once).
 *
 * Calls on one history must be ordered.  Returns SV_OK or a negative code.
 */
int spec_history_append(int32_t* counts, int32_t* ids, int32_t* num, int S, int V, const int32_t* slots,
                        const int32_t* tokens, int B, int T, int prompt, void* stream);
int spec_history_reset(int32_t* counts, const int32_t* ids, int32_t* num, int S, int V, const int32_t* slots, int B,
                       void* stream);

/*
 * The adjustments of a sampler's logits before temperature, top-k and top-p,
 * for J positions of each of B sequences.  Row (b, j) sees the history of its
 * slot and, after it, the first (first + j) draft tokens of b, as if they had
 * been output: position j of a verify follows x_1..x_j.  With c(v) the number
 * of times v was output and seen(v) = (v in the prompt or c(v) > 0):
 *
 *   z1 = seen(v) ? (z > 0 ? z / repetition : z * repetition) : z
 *   z2 = (z1 - frequency * c(v)) - (c(v) > 0 ? presence : 0)
 *   z3 = z2 + sum of the biases given for v
 *   out = mask allows v ? z3 : -inf
 *
 * formed in float32, each operation rounded by itself, and rounded once to the
 * logits' type.  A token that none of them touches keeps its bits.
 *
 *  logits      [B][J][V] bf16 or fp32, aligned to its element (16-byte alignment takes the
 *              wide path).
 *  out         [B][J][V], same type: `logits` itself (in place) or no overlap with it
 *              (SV_ERR_ARG).  In place, only what changes is written.
 *  counts, ids, num, S: a history as above, or NULL, NULL, NULL, 0: no history.
 *  slots       [B] int32 or NULL (slot b; then B <= S).  A slot outside [0, S) has no history.
 *              Slots may repeat (the candidates of one sequence share its history).
 *  draft_tokens [B][draft_stride] int32 or NULL (no drafts); first + J - 1 <= draft_stride and
 *              <= SL_MAX_DRAFT.  A token outside [0, V) is skipped.
 *  first       drafts that row 0 sees, >= 0.
 *  repetition, presence, frequency: [B] float, each may be NULL (1, 0, 0).
 *  bias_ids    [B][NB] int32, bias_values [B][NB] float, or both NULL with NB = 0; NB <= SL_MAX_BIAS.
 *              An id outside [0, V) is skipped (pad with -1).  The values of a repeated id are
 *              added up, in order.
 *  masks       [M][(V+31)/32] uint32: bit v % 32 of word v / 32 set if the mask allows v; and
 *  mask_rows   [B][J] int32: the mask of each row, -1 for none; or both NULL with M = 0.
 *  rows        [B] int32 or NULL: only rows j < rows[b] are used; the others are neither read nor
 *              written.
 * B * J <= SL_MAX_ROWS; B == 0 is a no-op; 1 <= V <= SV_MAX_VOCAB; 1 <= J.
 *
 * A repetition that is not positive and finite, a presence or frequency that
 * is not finite, or a mask row outside [-1, M) makes the rows concerned NaN,
 * which spec_verify and spec_sample report as invalid, as they do a row whose
 * mask allows nothing (only -inf).  A bias may be -inf (a ban).
 * Returns SV_OK or a negative code (nothing enqueued).
 */
int spec_process_logits(const void* logits, void* out, int dtype, const int32_t* counts, const int32_t* ids,
                        const int32_t* num, int S, const int32_t* slots, const int32_t* draft_tokens,
                        int draft_stride, int first, const float* repetition, const float* presence,
                        const float* frequency, const int32_t* bias_ids, const float* bias_values, int NB,
                        const uint32_t* masks, int M, const int32_t* mask_rows, const int32_t* rows, int B, int J,
                        int V, void* stream);

/* Static description of a return code (for SV_ERR_HIP, the last HIP error of this thread). */
const char* spec_logits_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_LOGITS_H */
