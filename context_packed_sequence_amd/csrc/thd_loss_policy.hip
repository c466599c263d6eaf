// Policy loss, one workgroup per row (kernel: thd_loss_rows.h).
#include "thd_loss_rows.h"

namespace thdcp {

hipError_t launch_policy_rows(const LogitRows& r, const LossArgs& a, hipStream_t stream) {
  return launch_rows_dtype<kLossPolicy>(r, a, stream);
}

}  // namespace thdcp
