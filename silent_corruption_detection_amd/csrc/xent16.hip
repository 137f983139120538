// xent16.hip -- the cross-entropy kernels for heads whose weights' rows lie at 16-byte boundaries,
// for gfx950.
#include "xent_device.h"

namespace sdc {
int32_t launch_logit_lse16(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_lse<kAt16>(h, a, s);
}
int32_t launch_logit_dz16(const HeadLaunch& h, const LogitArgs& a, hipStream_t s) {
  return launch_logit_dz<kAt16>(h, a, s);
}
int32_t launch_products16(const HeadLaunch& h, const ProductArgs& x, hipStream_t s) {
  return launch_products<kAt16>(h, x, s);
}
}  // namespace sdc
