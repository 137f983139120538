// xent_any.hip -- the cross-entropy kernels for heads whose weights' rows lie anywhere,
// for gfx950.
#include "xent_device.h"

namespace sdc {
int32_t launch_logit_lse_any(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_lse<kAny>(h, a, s);
}
int32_t launch_gradient_any(const HeadLaunch& h, const LogitArgs& a, const ProductArgs& x, hipStream_t s) {
  return launch_gradient<kAny>(h, a, x, s);
}
}  // namespace sdc
