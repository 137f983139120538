// adamw8.hip -- the AdamW kernels with 8-bit states, for gfx950.
#include "adamw_device.h"

namespace sdc {
int32_t launch_adamw8(uint32_t cls, const AdamwArgs& a, hipStream_t s) {
  return launch_adamw_state<1>(cls, a, s);
}
}  // namespace sdc
