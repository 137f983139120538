// ffn_any.hip -- the gated feed-forward kernels for weights whose rows lie anywhere,
// for gfx950.
#include "ffn_device.h"

namespace sdc {
int32_t launch_ffn_any(const FfnLaunch& l, const FfnArgs& a, hipStream_t s) { return launch_ffn<kAny>(l, a, s); }
int32_t launch_ffn_products_any(const FfnLaunch& l, const FfnProductArgs& a, hipStream_t s) {
  return launch_ffn_products<kAny>(l, a, s);
}
}  // namespace sdc
