// xent_any.hip -- the cross-entropy kernels for heads whose weights' rows lie anywhere,
// for gfx950.
#include "xent_device.h"

namespace sdc {
int32_t launch_logit_lse_any(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_lse<kAny>(h, a, s);
}
int32_t launch_logit_dz_any(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_dz<kAny>(h, a, s);
}
int32_t launch_products_any(const HeadLaunch& h, const ProductArgs& x, hipStream_t s) {
  return launch_products<kAny>(h, x, s);
}
}  // namespace sdc
