// Distillation from a teacher's top logits, one workgroup per row (kernel:
// thd_loss_rows.h).
#include "thd_loss_rows.h"

namespace thdcp {

hipError_t launch_distill_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  return launch_rows_dtype<kLossDistill>(r, a, stream);
}

}  // namespace thdcp
