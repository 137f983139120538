// adamw32.hip -- the AdamW kernels with fp32 states, for gfx950.
#include "adamw_device.h"

namespace sdc {
int32_t launch_adamw32(uint32_t cls, const AdamwArgs& a, hipStream_t s) {
  return launch_adamw_state<0>(cls, a, s);
}
}  // namespace sdc
