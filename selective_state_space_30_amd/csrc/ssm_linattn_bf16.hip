// ssm_linattn_bf16.hip -- the linear-attention chunk kernel in bf16.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_core_bf16(const LinCore &a, int mode, bool reverse, void *stream) {
  return lin::launch_core<uint16_t>(a, mode, reverse, stream);
}

}  // namespace ssm
