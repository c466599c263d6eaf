/*
 * thd_attention.h -- attention inside the documents of a packed stream, with
 * its gradient (C ABI of libthdcp, MI355X / gfx950).
 *
 *   thd_attention            output and log-sum-exp of each query row
 *   thd_attention_backward   gradients of queries, keys and values
 *
 * For a query at position i of its document and its keys j, all of the same
 * document:
 *   z_j = scale q.k_j, or cap tanh(scale q.k_j / cap)        (cap > 0)
 *   p_j = exp(z_j - lse),  lse = ln sum_j exp(z_j),  out = sum_j p_j v_j
 * over the keys it sees: j <= i (causal) or the whole document, and with a
 * window w > 0 those with |i - j| < w.  No token of another document and no pad
 * is ever seen or read into any result.
 *
 * Queries are the whole stream (cp_size 1), or the rows that rank `rank` of
 * cp_size holds in the zigzag layout of thd_cp.h: total_tokens / cp_size rows,
 * of each document the chunks rank and 2 cp_size - 1 - rank.  Keys and values
 * are the whole stream in token order, as gathered over the ranks; their
 * gradients are this rank's part of the sum over ranks.
 *
 * Conventions of thd_cp.h hold: device pointers, a hipStream_t passed as void*,
 * no call waits for the GPU, allocates or frees; argument errors are returned,
 * errors in device data go to a device status word.  Further:
 *  - q, out, dout, dq: [rows][heads][dim], k, v, dk, dv:
 *    [total_tokens][kv_heads][dim] of THD_BF16 or THD_FP16.  A head's elements
 *    are contiguous, rows and heads at strides of their own (multiples of 8
 *    elements), pointers 16-byte aligned: views of one projection's output
 *    need no copy.  dim is a multiple of 8 up to THD_MAX_HEAD_DIM, heads a
 *    multiple of kv_heads (query head h reads key head h / (heads / kv_heads));
 *  - lse: float [heads][rows];
 *  - cu_seqlens_padded: int32 [n_slots + 1]; cu_seqlens: real boundaries, or
 *    NULL (no slot has pads).  The pads of a slot are the tail of its padded range.
 *    A pad's row of out and of every gradient is 0, its lse -inf;
 *  - status (or NULL): THD_OK, or the first failing rule: THD_ERR_CU_START,
 *    THD_ERR_CU_MONOTONE (either list), THD_ERR_CU_TOTAL, THD_ERR_CU_DIVISIBLE
 *    (cp_size > 1), THD_ERR_REAL_GT_PADDED.  On such an error nothing else is
 *    written;
 *  - sums, softmax statistics and scores are held in 32 bits; probabilities and
 *    the scores' gradients are rounded to the tensors' type as factors of the
 *    matrix products; each result is rounded once.  No result depends on timing;
 *  - a value that is not finite reaches the rows of its own document only (of
 *    that document also rows that do not see it: its probability 0 times it);
 *  - workspace: thd_attention_workspace_bytes bytes, 16-byte aligned.  Its
 *    contents do not matter and are not kept.
 */
#ifndef THD_ATTENTION_H
#define THD_ATTENTION_H

#include <stdint.h>

#include "thd_cp.h"
#include "thd_loss.h" /* element types */

#ifdef __cplusplus
extern "C" {
#endif

#define THD_MAX_HEAD_DIM 128
#define THD_MAX_STREAM   2147418112 /* tokens: 2^31 - 2^16 */
#define THD_SCALE_LOG2   100   /* scales are 2^-100 to 2^100 */
#define THD_CAP_LOG2     64    /* caps are 2^-64 and up */

/* One tensor: device address, elements from row to row and from head to head. */
typedef struct thd_heads {
  void* data;
  int64_t row_stride;
  int64_t head_stride;
} thd_heads;

/* What a forward call and its backward call have in common (host memory). */
typedef struct thd_attention_shape {
  int32_t dtype;       /* THD_BF16 or THD_FP16 */
  int32_t heads, kv_heads, dim;
  int32_t causal;      /* 0 or 1 */
  int32_t window;      /* 0: none */
  int32_t cp_size, rank;
  int32_t n_slots;
  int64_t total_tokens; /* up to THD_MAX_STREAM */
  double scale;        /* 2^-THD_SCALE_LOG2 to 2^THD_SCALE_LOG2 */
  double cap;          /* 0: none; else from 2^-THD_CAP_LOG2 on; 1.45 cap and scale / cap finite in
                          32 bits, scale / cap not 0 there */
  const int32_t* cu_seqlens_padded;
  const int32_t* cu_seqlens;
} thd_attention_shape;

/*
 * thd_attention_workspace_bytes -- workspace of thd_attention (backward = 0) and
 * thd_attention_backward (backward = 1); -1 for a shape those calls refuse.
 * Host-only arithmetic; boundary pointers are not looked at.
 */
int64_t thd_attention_workspace_bytes(const thd_attention_shape* shape, int32_t backward);

/*
 * thd_attention -- out and lse.  No output may overlap an input or another output
 * (THD_ERR_ALIAS).  Two launches: one lays out the documents' tiles, one computes.
 */
int thd_attention(const thd_attention_shape* shape, const thd_heads* q, const thd_heads* k, const thd_heads* v,
                  const thd_heads* out, float* lse, int32_t* status, void* workspace, int64_t workspace_bytes,
                  void* stream);

/*
 * thd_attention_backward -- gradients of sum(dout * out) with respect to q, k and
 * v, with out and lse as thd_attention wrote them.  The gradients may be views of
 * one buffer whose rows interleave, as long as no two share an element.  Three
 * launches, one more for THD_FP16, and one more where a group of heads is dealt out
 * over workgroups (long documents, few key heads), with sums of its parts in the
 * workspace.
 */
int thd_attention_backward(const thd_attention_shape* shape, const thd_heads* q, const thd_heads* k,
                           const thd_heads* v, const thd_heads* out, const float* lse, const thd_heads* dout,
                           const thd_heads* dq, const thd_heads* dk, const thd_heads* dv, int32_t* status,
                           void* workspace, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* THD_ATTENTION_H */
