// ssm_linattn_bf16.hip -- the linear-attention chunk kernel in bf16.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_core_bf16(const LinCore &a, int mode, bool reverse, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool wide = linattn_slice(true, a.k.d, a.v.d) == 128;
  if (a.k.d <= 64)
    return wide ? lin::launch_core_m<uint16_t, 64, 2>(a, mode, reverse, s)
                : lin::launch_core_m<uint16_t, 64, 1>(a, mode, reverse, s);
  if (a.k.d <= 128)
    return wide ? lin::launch_core_m<uint16_t, 128, 2>(a, mode, reverse, s)
                : lin::launch_core_m<uint16_t, 128, 1>(a, mode, reverse, s);
  return lin::launch_core_m<uint16_t, 256, 1>(a, mode, reverse, s);
}

}  // namespace ssm
