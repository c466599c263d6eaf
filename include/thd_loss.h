/*
 * thd_loss.h -- losses on packed token streams, with their gradients (C ABI of
 * libthdcp, MI355X / gfx950).
 *
 * What a packed batch trains on, next to the layout transform of thd_cp.h:
 * rows are token positions (in natural or zigzag order, one rank's share or
 * every rank's), labels and masks are the streams thd_roll_labels and
 * thd_roll_labels_zigzag write, documents the slots of cu_seqlens_padded.
 *
 *   thd_token_logprobs            log-probability of each row's label
 *   thd_token_logprobs_backward   its gradient with respect to the logits
 *   thd_policy_loss               clipped policy loss with a KL term + gradient
 *   thd_distill_topk              distillation from a teacher's top logits + gradient
 *   thd_preference_loss           preference loss over document pairs + gradient
 *
 * Conventions of thd_cp.h hold: device pointers, a hipStream_t passed as void*,
 * no call waits for the GPU, allocates or frees; argument errors are returned,
 * errors in device data go to a device status word.  Further:
 *  - logits are row-major [rows][vocab] of dtype THD_BF16, THD_FP16 or
 *    THD_FP32, `row_stride` elements from one row to the next (>= vocab);
 *    pointers need the element's alignment only.  A gradient has the logits'
 *    dtype and a stride of its own; it may be the logits' own buffer (same
 *    pointer and stride: the gradient replaces the logits), any other overlap
 *    is THD_ERR_ALIAS.  It is rounded once, from 32 bits, to nearest even, and
 *    is stored fastest where its rows start at the same place within 16 bytes
 *    as the logits' rows;
 *  - sums and softmax statistics are held in 32 bits (64 in the preference
 *    loss), and no result depends on timing;
 *  - mask: uint8 [rows] or NULL (every row counts).  A row with mask 0 has loss,
 *    log-probability and gradient 0; its logits, label and other values are not
 *    read into any result, whatever they hold;
 *  - a label of an unmasked row outside [0, vocab) (distillation: a column
 *    outside [-1, vocab)) makes that row's results NaN and the status word
 *    THD_ERR_LABEL; other rows are not affected.  Without one the status word
 *    is THD_OK; status may be NULL;
 *  - columns at -inf are left out of the softmax; a row of nothing but -inf, or
 *    holding NaN or +inf, gives NaN;
 *  - workspace: at least thd_loss_workspace_bytes(...) bytes, 8-byte aligned;
 *    NULL where that is 0.  Its contents do not matter and are not kept.
 */
#ifndef THD_LOSS_H
#define THD_LOSS_H

#include <stdint.h>

#include "thd_cp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------- */
#define THD_BF16 0
#define THD_FP16 1
#define THD_FP32 2

/* ---- limits -------------------------------------------------------------- */
#define THD_MAX_VOCAB 268435456     /* 2^28 columns: a row of 1 GiB in 32 bits */
#define THD_MAX_TOPK  256           /* teacher columns per row */
#define THD_MAX_PAIRS 65536         /* document pairs per call */

/*
 * thd_loss_workspace_bytes -- workspace of thd_token_logprobs (targets = 0),
 * thd_policy_loss (targets = 1) and thd_distill_topk (targets = k); -1 for
 * sizes those calls refuse.  Not 0 only where rows are so few that each is cut
 * into parts over several workgroups.  Host-only arithmetic.
 */
int64_t thd_loss_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype, int32_t targets);

/*
 * thd_token_logprobs -- for each row z with label y:
 *   logp = z_y - lse,  lse = ln sum_v exp(z_v).
 * labels: int64 [rows]; logp, lse: float [rows] (outputs; 0 in masked rows).
 * One pass over the logits; one launch and one for the status word, or two
 * where the rows are cut into parts.
 */
int thd_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                       const int64_t* labels, const uint8_t* mask, float* logp, float* lse, int32_t* status,
                       void* workspace, int64_t workspace_bytes, void* stream);

/*
 * thd_token_logprobs_backward -- gradient of sum_t dlogp[t] logp[t]:
 *   dlogits[t][v] = dlogp[t] ([v = y_t] - exp(z_v - lse_t)),
 * with lse as thd_token_logprobs wrote it (NaN makes the row NaN).  The softmax is
 * taken against lse as it is given, a 32-bit number: the label's element is off by
 * up to about 2^-24 (|lse| + 4) |dlogp|, which is all of it for a label within that
 * of certainty (thd_policy_loss keeps the relative precision of 1 - q_y).  One
 * launch.
 */
int thd_token_logprobs_backward(const float* dlogp, const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                int64_t row_stride, const int64_t* labels, const float* lse, const uint8_t* mask,
                                void* dlogits, int64_t grad_stride, void* stream);

/*
 * thd_policy_loss -- clipped policy loss with a KL term.  With logp as above,
 * r = exp(logp - old_logp), u = ref_logp - logp:
 *   loss = w (-min(r A, min(max(r, 1 - clip_low), 1 + clip_high) A)
 *             + kl_coef (exp(u) - u - 1))
 * and dlogits[t][v] = d loss[t] / d logits[t][v].  The gradient flows through r
 * where the minimum takes the unclipped branch or both are equal.
 * old_logp, advantages: float [rows].  ref_logp: float [rows], may be NULL when
 * kl_coef is 0 (it is not read then).  weights: float [rows] w, NULL: 1.
 * 0 <= clip_low <= 1, clip_high >= 0, all three finite.
 * loss, logp: float [rows] (outputs).  The logits are read once and the
 * gradient written once (rows cut into parts, and what of a row is beyond a
 * compute unit's registers and LDS, from 26624 16-byte words on, are read
 * twice).
 */
int thd_policy_loss(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                    const int64_t* labels, const uint8_t* mask, const float* old_logp, const float* ref_logp,
                    const float* advantages, const float* weights, double clip_low, double clip_high, double kl_coef,
                    float* loss, float* logp, void* dlogits, int64_t grad_stride, int32_t* status, void* workspace,
                    int64_t workspace_bytes, void* stream);

/*
 * thd_distill_topk -- distillation from the k largest logits of a teacher.  With
 * tau = temperature, p = softmax(teacher / tau) over the row's k given columns
 * and q = softmax(z / tau) over the whole vocabulary:
 *   loss = tau^2 w sum_i p_i (ln p_i - ln q_{id_i})
 *   dlogits[v] = tau w (q_v - sum_i p_i [id_i = v]).
 * teacher_logits: [rows][k] of teacher_dtype, teacher_ids: [rows][k] int32
 * (id_bytes 4) or int64 (id_bytes 8), rows teacher_stride elements apart in
 * both.  An id of -1, or a teacher logit of -inf, has no part in the sum; a row
 * without any part is as a masked one.  An id may occur more than once.
 * 1 <= k <= THD_MAX_TOPK, temperature > 0 and finite, log2(e) / temperature finite
 * in 32 bits (temperatures from 4.3e-39 on).
 * weights: float [rows] w, NULL: 1.  loss: float [rows] (output).
 */
int thd_distill_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                     const void* teacher_logits, int32_t teacher_dtype, const void* teacher_ids, int32_t id_bytes,
                     int32_t k, int64_t teacher_stride, const uint8_t* mask, const float* weights, double temperature,
                     float* loss, void* dlogits, int64_t grad_stride, int32_t* status, void* workspace,
                     int64_t workspace_bytes, void* stream);

/*
 * thd_preference_workspace_bytes -- workspace of thd_preference_loss (8-byte
 * aligned): 8 bytes per 512 tokens and per slot.  -1 for sizes it refuses.
 */
int64_t thd_preference_workspace_bytes(int64_t total_tokens, int32_t n_slots);

/*
 * thd_preference_loss -- preference loss over pairs of documents of one packed
 * stream in natural (token) order.  With S_d the sum of logp - ref_logp over
 * document d's unmasked tokens, for pair i = (chosen, rejected):
 *   rewards[i] = (beta S_chosen, beta S_rejected),  D = their difference
 *   loss[i] = scale ((1 - e) ln(1 + exp(-D)) + e ln(1 + exp(D)))
 * and dlogp[t] = d (sum of the losses) / d logp[t], 0 for masked tokens and
 * documents in no pair; it is what thd_token_logprobs_backward takes.
 * logp, ref_logp (NULL: 0), dlogp: float [total_tokens]; mask uint8
 * [total_tokens] or NULL; cu_seqlens_padded int32 [n_slots + 1];
 * pairs int32 [n_pairs][2] of slot numbers, a slot in any number of pairs, (-1,
 * -1) for an unused entry (loss and rewards 0); e = label_smoothing in [0, 1].
 * status: THD_OK, the first failing boundary rule (THD_ERR_CU_START,
 * THD_ERR_CU_MONOTONE, THD_ERR_CU_TOTAL: nothing else is written then), or
 * THD_ERR_PAIR if a pair names no slot: its loss and rewards are NaN and it has
 * no part in dlogp.  Two launches.
 * Cost: a few bytes a token for documents of up to some 100000 tokens in a few
 * pairs each.  Beyond, each 512 tokens of a document add up the partial sums of
 * both documents of each of its pairs again, and every piece of a document within
 * 512 tokens looks through all pairs: the time grows with the square of a
 * document's length times its pairs, and with documents times pairs.
 */
int thd_preference_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                        const int32_t* cu_seqlens_padded, int32_t n_slots, int64_t total_tokens,
                        const int32_t* pairs, int32_t n_pairs, double beta, double label_smoothing, double scale,
                        float* loss, float* rewards, float* dlogp, int32_t* status, void* workspace,
                        int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* THD_LOSS_H */
