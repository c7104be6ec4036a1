// ssm_linattn_f32.hip -- the linear-attention chunk kernel in fp32.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_core_f32(const LinCore &a, int mode, bool reverse, void *stream) {
  return lin::launch_core<float>(a, mode, reverse, stream);
}

}  // namespace ssm
