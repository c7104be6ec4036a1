// ssm_linattn_grads_f32.hip -- the linear-attention chunk kernel in fp32: gradients.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_grads_f32(const LinCore &dq, const LinCore &dk, const LinCore &dv,
                              const LinPairs *pairs, void *stream) {
  return lin::launch_grads<float>(dq, dk, dv, pairs, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
