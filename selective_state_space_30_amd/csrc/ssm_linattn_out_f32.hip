// ssm_linattn_out_f32.hip -- the linear-attention chunk kernel in fp32: forward output and segment state passes.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_out_f32(const LinCore &a, void *stream) {
  return lin::launch_out<float>(a, static_cast<hipStream_t>(stream));
}

int launch_linattn_states_f32(const LinCore &a, const LinCore *back, void *stream) {
  return lin::launch_states<float>(a, back, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
