// xent_few.hip -- the cross-entropy kernels for heads applied to few rows, for
// gfx950.
#include "xent_device.h"

namespace sdc {
int32_t launch_logit_lse_few(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_lse<kDeep>(h, a, s);
}
int32_t launch_logit_dz_few(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_dz<kDeep>(h, a, s);
}
}  // namespace sdc
