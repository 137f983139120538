// ffn16.hip -- the gated feed-forward kernels for weights whose rows lie at 16-byte boundaries,
// for gfx950.
#include "ffn_device.h"

namespace sdc {
int32_t launch_ffn16(const FfnLaunch& l, const FfnArgs& a, hipStream_t s) { return launch_ffn<kAt16>(l, a, s); }
int32_t launch_ffn_products16(const FfnLaunch& l, const FfnProductArgs& a, hipStream_t s) {
  return launch_ffn_products<kAt16>(l, a, s);
}
}  // namespace sdc
