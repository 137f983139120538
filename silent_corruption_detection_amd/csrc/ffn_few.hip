// ffn_few.hip -- the gated feed-forward kernels for few rows of x, for gfx950.
#include "ffn_device.h"

namespace sdc {
int32_t launch_ffn_few(const FfnLaunch& l, const FfnArgs& a, hipStream_t s) { return launch_ffn<kDeep>(l, a, s); }
}  // namespace sdc
