// C ABI of the loss operators: host-side argument checks and stream-ordered
// launches.  See include/thd_loss.h for the contract of each call.
#include <cmath>

#include "thd_loss_internal.h"

namespace {

struct Range {
  const void* p;
  int64_t bytes;
};

bool meet(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const auto x = reinterpret_cast<uintptr_t>(a.p);
  const auto y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + static_cast<uint64_t>(b.bytes) && y < x + static_cast<uint64_t>(a.bytes);
}

// No output may meet an input or another output.
template <size_t N, size_t M>
bool apart(const Range (&outs)[N], const Range (&ins)[M]) {
  for (size_t i = 0; i < N; ++i) {
    for (size_t j = i + 1; j < N; ++j)
      if (meet(outs[i], outs[j])) return false;
    for (size_t j = 0; j < M; ++j)
      if (meet(outs[i], ins[j])) return false;
  }
  return true;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int element_bytes(int32_t dtype) {
  switch (dtype) {
    case THD_BF16:
    case THD_FP16: return 2;
    case THD_FP32: return 4;
    default: return 0;
  }
}

bool sizes_ok(int64_t rows, int64_t vocab, int32_t dtype) {
  return rows >= 0 && rows <= INT32_MAX && vocab >= 1 && vocab <= THD_MAX_VOCAB && element_bytes(dtype) != 0;
}

// Bytes from the first to the last element of a row-major matrix; -1 if the
// stride does not fit.
int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t stride, int64_t element) {
  if (rows == 0) return 0;
  if (stride < cols || stride > (INT64_MAX / 16 - cols) / rows) return -1;
  return ((rows - 1) * stride + cols) * element;
}

struct Layout {
  thdcp::LossParts parts;
  int64_t bytes;
};

Layout loss_layout(void* workspace, int64_t rows, int64_t vocab, int32_t dtype, int32_t targets) {
  Layout l{};
  const auto n = static_cast<int32_t>(rows);
  const auto v = static_cast<int32_t>(vocab);
  l.parts = targets == 0 ? thdcp::logp_parts(n, v, dtype) : thdcp::loss_parts(n, v, dtype);
  if (l.parts.parts == 1) return l;
  const int64_t stats = rows * l.parts.parts * static_cast<int64_t>(sizeof(float2));
  l.bytes = stats + rows * (targets > 1 ? targets : 1) * static_cast<int64_t>(sizeof(float));
  l.parts.stats = static_cast<float2*>(workspace);
  l.parts.targets = reinterpret_cast<float*>(static_cast<char*>(workspace) + stats);
  return l;
}

int check_workspace(const Layout& l, const void* workspace, int64_t workspace_bytes) {
  if (l.bytes == 0) return THD_OK;
  return workspace && workspace_bytes >= l.bytes && aligned(workspace, 8) ? THD_OK : THD_ERR_ARG;
}

hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

int launched(hipError_t e) { return e == hipSuccess ? THD_OK : THD_ERR_HIP; }

// The one-pass kernels' status word: written by a workgroup of the launch that
// looks through all targets where they are few, else set to THD_OK by a launch
// before and by the rows that fail.
int prepare_status(thdcp::LossArgs& a, int64_t targets, void* stream) {
  if (!a.status) return THD_OK;
  a.scan = targets <= thdcp::kScanTargets;
  return a.scan ? THD_OK : launched(thdcp::launch_status_init(a.status, as_stream(stream)));
}

int init_status(int32_t* status, void* stream) {
  return status ? launched(thdcp::launch_status_init(status, as_stream(stream))) : THD_OK;
}

}  // namespace

extern "C" {

int64_t thd_loss_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype, int32_t targets) {
  if (!sizes_ok(rows, vocab, dtype) || targets < 0 || targets > THD_MAX_TOPK) return -1;
  return loss_layout(nullptr, rows, vocab, dtype, targets).bytes;
}

int thd_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                       const int64_t* labels, const uint8_t* mask, float* logp, float* lse, int32_t* status,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (!sizes_ok(rows, vocab, dtype)) return THD_ERR_ARG;
  if (rows == 0) return init_status(status, stream);
  const int64_t bytes = matrix_bytes(rows, vocab, row_stride, element_bytes(dtype));
  if (bytes < 0 || !logits || !labels || !logp || !lse || !aligned(logits, element_bytes(dtype))) return THD_ERR_ARG;
  const Layout l = loss_layout(workspace, rows, vocab, dtype, 0);
  if (check_workspace(l, workspace, workspace_bytes) != THD_OK) return THD_ERR_ARG;
  const Range outs[] = {{logp, rows * 4}, {lse, rows * 4}, {status, 4}, {workspace, l.bytes}};
  const Range ins[] = {{logits, bytes}, {labels, rows * 8}, {mask, rows}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::LogitRows r{logits, nullptr, row_stride, 0, static_cast<int32_t>(rows), static_cast<int32_t>(vocab), dtype};
  thdcp::LossArgs a{};
  a.mask = mask;
  a.labels = labels;
  a.logp = logp;
  a.lse = lse;
  a.status = status;
  if (l.parts.parts == 1) {
    const int rc = prepare_status(a, rows, stream);
    if (rc != THD_OK) return rc;
  }
  return launched(thdcp::launch_token_logprobs(r, a, l.parts, as_stream(stream)));
}

int thd_token_logprobs_backward(const float* dlogp, const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                                int64_t row_stride, const int64_t* labels, const float* lse, const uint8_t* mask,
                                void* dlogits, int64_t grad_stride, void* stream) {
  if (!sizes_ok(rows, vocab, dtype)) return THD_ERR_ARG;
  if (rows == 0) return THD_OK;
  const int es = element_bytes(dtype);
  const int64_t in_bytes = matrix_bytes(rows, vocab, row_stride, es);
  const int64_t out_bytes = matrix_bytes(rows, vocab, grad_stride, es);
  if (in_bytes < 0 || out_bytes < 0 || !dlogp || !logits || !labels || !lse || !dlogits || !aligned(logits, es) ||
      !aligned(dlogits, es))
    return THD_ERR_ARG;
  const bool in_place = dlogits == logits && grad_stride == row_stride;
  const Range outs[] = {{dlogits, out_bytes}};
  const Range ins[] = {{logits, in_place ? 0 : in_bytes}, {labels, rows * 8}, {mask, rows}, {dlogp, rows * 4},
                       {lse, rows * 4}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::LogitRows r{logits, dlogits, row_stride, grad_stride, static_cast<int32_t>(rows),
                     static_cast<int32_t>(vocab), dtype};
  thdcp::LossArgs a{};
  a.mask = mask;
  a.labels = labels;
  a.lse_in = lse;
  a.dlogp = dlogp;
  return launched(thdcp::launch_logp_backward(r, a, as_stream(stream)));
}

int thd_policy_loss(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                    const int64_t* labels, const uint8_t* mask, const float* old_logp, const float* ref_logp,
                    const float* advantages, const float* weights, double clip_low, double clip_high, double kl_coef,
                    float* loss, float* logp, void* dlogits, int64_t grad_stride, int32_t* status, void* workspace,
                    int64_t workspace_bytes, void* stream) {
  if (!sizes_ok(rows, vocab, dtype)) return THD_ERR_ARG;
  // the kernels hold the clip's ends and the coefficient in 32 bits
  const auto kl = static_cast<float>(kl_coef);
  if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0) || !std::isfinite(static_cast<float>(clip_high)) ||
      !std::isfinite(kl))
    return THD_ERR_ARG;
  if (rows == 0) return init_status(status, stream);
  const int es = element_bytes(dtype);
  const int64_t in_bytes = matrix_bytes(rows, vocab, row_stride, es);
  const int64_t out_bytes = matrix_bytes(rows, vocab, grad_stride, es);
  if (in_bytes < 0 || out_bytes < 0 || !logits || !labels || !old_logp || !advantages || !loss || !logp || !dlogits ||
      (kl != 0.0f && !ref_logp) || !aligned(logits, es) || !aligned(dlogits, es))
    return THD_ERR_ARG;
  const Layout l = loss_layout(workspace, rows, vocab, dtype, 1);
  if (check_workspace(l, workspace, workspace_bytes) != THD_OK) return THD_ERR_ARG;
  const bool in_place = dlogits == logits && grad_stride == row_stride;
  const Range outs[] = {{dlogits, out_bytes}, {loss, rows * 4}, {logp, rows * 4}, {status, 4}, {workspace, l.bytes}};
  const Range ins[] = {{logits, in_place ? 0 : in_bytes}, {labels, rows * 8}, {mask, rows}, {old_logp, rows * 4},
                       {kl != 0.0f ? ref_logp : nullptr, rows * 4}, {advantages, rows * 4},
                       {weights, rows * 4}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::LogitRows r{logits, dlogits, row_stride, grad_stride, static_cast<int32_t>(rows),
                     static_cast<int32_t>(vocab), dtype};
  thdcp::LossArgs a{};
  a.mask = mask;
  a.labels = labels;
  a.weights = weights;
  a.logp = logp;
  a.old_logp = old_logp;
  a.ref_logp = kl != 0.0f ? ref_logp : nullptr;
  a.advantages = advantages;
  a.low = static_cast<float>(1.0 - clip_low);
  a.high = static_cast<float>(1.0 + clip_high);
  a.ln_low = std::log1p(-clip_low);
  a.ln_high = std::log1p(clip_high);
  a.kl_coef = kl;
  a.loss = loss;
  a.status = status;
  if (l.parts.parts > 1) return launched(thdcp::launch_policy_parts(r, a, l.parts, as_stream(stream)));
  const int rc = prepare_status(a, rows, stream);
  if (rc != THD_OK) return rc;
  return launched(thdcp::launch_policy_rows(r, a, as_stream(stream)));
}

int thd_distill_topk(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                     const void* teacher_logits, int32_t teacher_dtype, const void* teacher_ids, int32_t id_bytes,
                     int32_t k, int64_t teacher_stride, const uint8_t* mask, const float* weights, double temperature,
                     float* loss, void* dlogits, int64_t grad_stride, int32_t* status, void* workspace,
                     int64_t workspace_bytes, void* stream) {
  if (!sizes_ok(rows, vocab, dtype) || element_bytes(teacher_dtype) == 0) return THD_ERR_ARG;
  if (k < 1 || k > THD_MAX_TOPK || (id_bytes != 4 && id_bytes != 8)) return THD_ERR_ARG;
  const auto tau = static_cast<float>(temperature);
  const auto inv = static_cast<float>(1.0 / temperature);
  // the kernels multiply logits by log2(e) / tau
  if (!(tau > 0.0f) || !std::isfinite(tau) || !std::isfinite(inv * 1.4426950408889634f) || !(inv > 0.0f))
    return THD_ERR_ARG;
  if (rows == 0) return init_status(status, stream);
  const int es = element_bytes(dtype);
  const int ts = element_bytes(teacher_dtype);
  const int64_t in_bytes = matrix_bytes(rows, vocab, row_stride, es);
  const int64_t out_bytes = matrix_bytes(rows, vocab, grad_stride, es);
  const int64_t t_bytes = matrix_bytes(rows, k, teacher_stride, ts);
  const int64_t id_total = matrix_bytes(rows, k, teacher_stride, id_bytes);
  if (in_bytes < 0 || out_bytes < 0 || t_bytes < 0 || id_total < 0 || !logits || !teacher_logits || !teacher_ids ||
      !loss || !dlogits || !aligned(logits, es) || !aligned(dlogits, es) || !aligned(teacher_logits, ts) ||
      !aligned(teacher_ids, id_bytes))
    return THD_ERR_ARG;
  const Layout l = loss_layout(workspace, rows, vocab, dtype, k);
  if (check_workspace(l, workspace, workspace_bytes) != THD_OK) return THD_ERR_ARG;
  const bool in_place = dlogits == logits && grad_stride == row_stride;
  const Range outs[] = {{dlogits, out_bytes}, {loss, rows * 4}, {status, 4}, {workspace, l.bytes}};
  const Range ins[] = {{logits, in_place ? 0 : in_bytes}, {teacher_logits, t_bytes}, {teacher_ids, id_total},
                       {mask, rows}, {weights, rows * 4}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::LogitRows r{logits, dlogits, row_stride, grad_stride, static_cast<int32_t>(rows),
                     static_cast<int32_t>(vocab), dtype};
  thdcp::LossArgs a{};
  a.mask = mask;
  a.weights = weights;
  a.teacher = teacher_logits;
  a.teacher_ids = teacher_ids;
  a.teacher_stride = teacher_stride;
  a.teacher_dtype = teacher_dtype;
  a.ids64 = id_bytes == 8;
  a.k = k;
  a.temperature = tau;
  a.inv_temperature = inv;
  a.loss = loss;
  a.status = status;
  if (l.parts.parts > 1) return launched(thdcp::launch_distill_parts(r, a, l.parts, as_stream(stream)));
  const int rc = prepare_status(a, rows * k, stream);
  if (rc != THD_OK) return rc;
  return launched(thdcp::launch_distill_rows(r, a, as_stream(stream)));
}

int64_t thd_preference_workspace_bytes(int64_t total_tokens, int32_t n_slots) {
  if (total_tokens < 0 || total_tokens > INT32_MAX || n_slots < 0 || n_slots == INT32_MAX) return -1;
  return 8 + 8 * (static_cast<int64_t>(thdcp::preference_tiles(static_cast<int32_t>(total_tokens))) + n_slots);
}

int thd_preference_loss(const float* logp, const float* ref_logp, const uint8_t* mask,
                        const int32_t* cu_seqlens_padded, int32_t n_slots, int64_t total_tokens,
                        const int32_t* pairs, int32_t n_pairs, double beta, double label_smoothing, double scale,
                        float* loss, float* rewards, float* dlogp, int32_t* status, void* workspace,
                        int64_t workspace_bytes, void* stream) {
  const int64_t need = thd_preference_workspace_bytes(total_tokens, n_slots);
  if (need < 0 || n_pairs < 0 || n_pairs > THD_MAX_PAIRS) return THD_ERR_ARG;
  if (!(label_smoothing >= 0.0 && label_smoothing <= 1.0) || !std::isfinite(beta) || !std::isfinite(scale))
    return THD_ERR_ARG;
  if (!cu_seqlens_padded || !workspace || workspace_bytes < need || !aligned(workspace, 8)) return THD_ERR_ARG;
  if ((total_tokens > 0 && (!logp || !dlogp)) || (n_pairs > 0 && (!pairs || !loss || !rewards))) return THD_ERR_ARG;
  const int64_t t = total_tokens, n = n_pairs;
  const Range outs[] = {{loss, n * 4}, {rewards, n * 8}, {dlogp, t * 4}, {status, 4}, {workspace, need}};
  const Range ins[] = {{logp, t * 4}, {ref_logp, t * 4}, {mask, t}, {cu_seqlens_padded, (n_slots + 1LL) * 4},
                       {pairs, n * 8}};
  if (!apart(outs, ins)) return THD_ERR_ALIAS;
  thdcp::PreferenceArgs a{};
  a.logp = logp;
  a.ref_logp = ref_logp;
  a.mask = mask;
  a.cu = cu_seqlens_padded;
  a.pairs = pairs;
  a.n_slots = n_slots;
  a.n_pairs = n_pairs;
  a.total = static_cast<int32_t>(total_tokens);
  a.beta = beta;
  a.smoothing = label_smoothing;
  a.scale = scale;
  a.loss = loss;
  a.rewards = rewards;
  a.dlogp = dlogp;
  a.status = status;
  a.ws_code = static_cast<int32_t*>(workspace);
  a.ws_sums = reinterpret_cast<double*>(static_cast<char*>(workspace) + 8);
  return launched(thdcp::launch_preference(a, as_stream(stream)));
}

}  // extern "C"
