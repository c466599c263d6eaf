/*
 * thd_params.h -- embedding table and gradients of a training step on packed
 * streams (C ABI of libthdcp, MI355X / gfx950).
 *
 *   thd_embedding            rows of the table for the stream's token ids
 *   thd_embedding_backward   the table's gradient
 *   thd_gradient_norm        norm of many gradients together
 *   thd_clip_gradients       the gradients, scaled down to a largest norm
 *
 * Conventions of thd_cp.h hold: device pointers, a hipStream_t passed as void*,
 * no call waits for the GPU, allocates or frees; argument errors are returned,
 * errors in device data go to a device status word (or NULL).  No result depends
 * on timing.  Tensors need the element's alignment only; 16-byte aligned rows are
 * fastest.
 */
#ifndef THD_PARAMS_H
#define THD_PARAMS_H

#include <stdint.h>

#include "thd_cp.h"
#include "thd_loss.h" /* element types, THD_MAX_VOCAB */

#ifdef __cplusplus
extern "C" {
#endif

#define THD_MAX_WIDTH   1048576   /* elements of a table row */
#define THD_MAX_TENSORS 65536     /* gradients per call */

/*
 * thd_embedding -- out[t] = scale table[ids[t]], rounded once.
 *
 * ids: int64 [rows]; mask: uint8 [rows] or NULL, rows with mask 0 are 0 and their
 * ids are not looked at (mask[0] of thd_roll_labels marks a stream's tokens).
 * table: [vocab][width] of dtype THD_BF16, THD_FP16 or THD_FP32, rows `table_stride`
 * elements apart (>= width); out: [rows][width] of the same dtype, rows `out_stride`
 * apart.  scale is finite in 32 bits.  An id that is no row of the table makes its
 * row NaN and the status word THD_ERR_TOKEN; without one it is THD_OK.  One launch,
 * and one before it for the status word above 8192 rows of less than 4096 bytes.
 */
int thd_embedding(const int64_t* ids, const uint8_t* mask, int64_t rows, const void* table, int32_t dtype,
                  int64_t vocab, int64_t width, int64_t table_stride, double scale, void* out, int64_t out_stride,
                  int32_t* status, void* stream);

/*
 * thd_embedding_workspace_bytes -- workspace of thd_embedding_backward, 16-byte
 * aligned: 16 bytes a row, partial sums of runs of one token that pass the borders of
 * units of 16 to 128 sorted rows (8 bytes for each element of a row and unit, rows in
 * whole eights of elements), and up to 0.5 MiB.  -1 for sizes the call refuses.  Host-only arithmetic.
 */
int64_t thd_embedding_workspace_bytes(int64_t rows, int64_t vocab, int64_t width);

/*
 * thd_embedding_backward -- dtable[v] = scale sum of drows[t] over the rows t with
 * ids[t] = v and mask not 0, in 32 bits in the rows' order within units of 16 to 128
 * sorted rows (the more and the wider the rows, the longer), those sums in order, rounded
 * once.
 *
 * drows: [rows][width] of dtype, rows `row_stride` elements apart; dtable:
 * [vocab][width] of out_dtype, which is dtype or THD_FP32, rows `table_stride` apart.
 * accumulate 0: every row of dtable is written (0 without a token); 1: the sums are
 * added to what dtable holds and rows without a token are not touched (a table that
 * has gradients from elsewhere, too).  An id that is no row of the table has no part,
 * and the status word is THD_ERR_TOKEN; without one it is THD_OK.
 * The rows are sorted by token: one launch up to 8192 rows, beyond two for each 9
 * bits of vocab, and two launches for the sums.
 */
int thd_embedding_backward(const void* drows, int32_t dtype, const int64_t* ids, const uint8_t* mask, int64_t rows,
                           int64_t vocab, int64_t width, int64_t row_stride, double scale, int32_t accumulate,
                           void* dtable, int32_t out_dtype, int64_t table_stride, int32_t* status, void* workspace,
                           int64_t workspace_bytes, void* stream);

/*
 * thd_gradients_workspace_bytes -- workspace of the two calls below, 8-byte aligned;
 * -1 for a number of tensors they refuse.
 */
int64_t thd_gradients_workspace_bytes(int32_t n_tensors);

/*
 * thd_gradient_norm -- *norm = |scale| sqrt(sum of the squares of all elements of all
 * tensors): squares of 16 bytes of elements summed in 32 bits (in 64 where 32 cannot
 * hold them), those sums in 64.
 *
 * grads, elements, dtypes: host arrays of n_tensors entries (0 to THD_MAX_TENSORS):
 * device address, number of elements (0 and up) and element type of each contiguous
 * tensor; types may differ.  norm: device float.  status: THD_ERR_NORM if the norm is
 * not finite (in 32 bits), else THD_OK.  One launch for each 96 tensors, and one more.
 */
int thd_gradient_norm(const void* const* grads, const int64_t* elements, const int32_t* dtypes, int32_t n_tensors,
                      double scale, float* norm, int32_t* status, void* workspace, int64_t workspace_bytes,
                      void* stream);

/*
 * thd_clip_gradients -- outs[i] = f grads[i], f = scale min(1, max_norm / (norm + 1e-6)),
 * each element rounded once.
 *
 * norm_in NULL: norm is that of thd_gradient_norm for these tensors, and is written to
 * *norm; else it is *norm_in (device float, e.g. joined over ranks whose tensors are
 * parts of a whole), and norm, if not NULL, receives it.  A norm that is not finite makes
 * every output 0 and the status word THD_ERR_NORM: a step with it moves no weight by
 * these gradients, and nothing that is not finite is left in them.
 * outs: host array of device addresses, out_dtypes: each the tensor's own type or
 * THD_FP32.  An output may be its own gradient of the same type (scaled in place; with
 * f = 1 it is left alone); any other overlap is THD_ERR_ALIAS.  max_norm > 0 (infinite:
 * f = scale), scale finite in 32 bits.  Two launches for each 96 tensors, one with
 * norm_in, and one between for more than 64 MiB.
 */
int thd_clip_gradients(const void* const* grads, void* const* outs, const int64_t* elements, const int32_t* dtypes,
                       const int32_t* out_dtypes, int32_t n_tensors, double max_norm, double scale,
                       const float* norm_in, float* norm, int32_t* status, void* workspace, int64_t workspace_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* THD_PARAMS_H */
