// layer_ssm_bwd_bf16.hip -- the state space scan's gradient for bfloat16 inputs (layer_ssm_bwd.h).
#include "layer_ssm_bwd.h"

namespace layer {
namespace ssm_bwd {

void launch_bf16(const SsmParams& p, const BwdSpace& ws, hipStream_t st) { launch_kernel<uint16_t>(p, ws, st); }

}  // namespace ssm_bwd
}  // namespace layer
