// Internal declarations of the loss operators on packed streams.  Not part
// of the public ABI (that is include/thd_loss.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "thd_internal.h"
#include "thd_loss.h"

namespace thdcp {

// Rows of logits, and of their gradient where a call writes one.
struct LogitRows {
  const void* in;
  void* out;             // gradient rows, or null
  int64_t in_stride;     // elements between two rows
  int64_t out_stride;
  int32_t rows;
  int32_t vocab;
  int32_t dtype;         // THD_BF16, THD_FP16 or THD_FP32
};

// Which loss a gradient kernel computes.
enum LossKind : int { kLossLogp, kLossPolicy, kLossDistill };

// Per-row inputs and outputs of every loss; a call fills the members of its
// own loss and leaves the others null.
struct LossArgs {
  const uint8_t* mask;       // [rows], null: every row counts
  const int64_t* labels;     // [rows]
  const float* weights;      // [rows], null: 1
  // log-probabilities and their gradient
  const float* lse_in;       // [rows]
  const float* dlogp;        // [rows]
  float* lse;                // [rows]
  float* logp;               // [rows]
  // policy loss
  const float* old_logp;     // [rows]
  const float* ref_logp;     // [rows] or null
  const float* advantages;   // [rows]
  double ln_low, ln_high;    // logarithms of the clip's ends
  float low, high;           // the clip's ends
  float kl_coef;
  // distillation
  const void* teacher;       // [rows][k] teacher logits
  const void* teacher_ids;   // [rows][k] columns, int32 or int64
  int64_t teacher_stride;    // elements between two rows of both
  int32_t teacher_dtype;
  int32_t ids64;             // 1: teacher_ids are int64
  int32_t k;
  float temperature, inv_temperature;
  // outputs
  float* loss;               // [rows]
  int32_t* status;           // or null
  int32_t scan;              // 1: a workgroup of its own writes it (scan_status)
};

// Targets a call may have for one workgroup to look through them all: 64
// threads take about 10 us for as many, beside rows that take as long.
constexpr int64_t kScanTargets = 8192;

// Row parts of the two-pass form: every part's running maximum and sum, then
// the logits of the row's targets (its label, or the teacher's columns).
struct LossParts {
  int32_t parts;             // 1: the one-pass form, no workspace
  int32_t turns;             // turns of 256 words in a part
  int32_t chunk_shift;       // parts per chunk of an XCD's order, as a power of two
  float2* stats;             // [rows][parts] (maximum, sum of exponentials)
  float* targets;            // [rows][k]
};

// How a row is cut so that few rows still fill the chip; one part where one
// workgroup per row is the faster form.
LossParts logp_parts(int32_t rows, int32_t vocab, int32_t dtype);
LossParts loss_parts(int32_t rows, int32_t vocab, int32_t dtype);

// Compute units of the current device (256 where it does not say).
int32_t compute_units();

hipError_t launch_status_init(int32_t* status, hipStream_t stream);
hipError_t launch_token_logprobs(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream);
hipError_t launch_logp_backward(const LogitRows& r, const LossArgs& a, hipStream_t stream);
hipError_t launch_policy_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream);
hipError_t launch_distill_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream);
hipError_t launch_policy_parts(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream);
hipError_t launch_distill_parts(const LogitRows& r, const LossArgs& a, const LossParts& p, hipStream_t stream);

// Preference loss (thd_preference.hip).
struct PreferenceArgs {
  const float* logp;
  const float* ref_logp;     // or null
  const uint8_t* mask;       // or null
  const int32_t* cu;         // [n_slots + 1]
  const int32_t* pairs;      // [n_pairs][2]
  int32_t n_slots, n_pairs, total;
  double beta, smoothing, scale;
  float* loss;               // [n_pairs]
  float* rewards;            // [n_pairs][2]
  float* dlogp;              // [total]
  int32_t* status;
  int32_t* ws_code;          // boundary check's code, for the second launch
  double* ws_sums;           // [tiles + n_slots], entry tile + slot
};
int32_t preference_tiles(int32_t total);
hipError_t launch_preference(const PreferenceArgs& a, hipStream_t stream);

}  // namespace thdcp
