// ssm_linattn_f32.hip -- the linear-attention chunk kernel in fp32.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_core_f32(const LinCore &a, int mode, bool reverse, void *stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.k.d <= 64) return lin::launch_core_m<float, 64, 1>(a, mode, reverse, s);
  if (a.k.d <= 128) return lin::launch_core_m<float, 128, 1>(a, mode, reverse, s);
  return lin::launch_core_m<float, 256, 1>(a, mode, reverse, s);
}

}  // namespace ssm
