// ssm_linattn_out_bf16.hip -- the linear-attention chunk kernel in bf16: forward output and segment state passes.
#include "ssm_linattn_core.h"

namespace ssm {

int launch_linattn_out_bf16(const LinCore &a, void *stream) {
  return lin::launch_out<uint16_t>(a, static_cast<hipStream_t>(stream));
}

int launch_linattn_states_bf16(const LinCore &a, const LinCore *back, void *stream) {
  return lin::launch_states<uint16_t>(a, back, static_cast<hipStream_t>(stream));
}

}  // namespace ssm
