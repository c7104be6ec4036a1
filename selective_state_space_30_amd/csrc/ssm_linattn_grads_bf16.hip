// ssm_linattn_grads_bf16.hip -- the linear-attention chunk kernel in bf16: gradients.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_grads_bf16(const LinCore &dq, const LinCore &dk, const LinCore &dv,
                              const LinPairs *pairs, void *stream) {
  return lin::launch_grads<uint16_t>(dq, dk, dv, pairs, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
