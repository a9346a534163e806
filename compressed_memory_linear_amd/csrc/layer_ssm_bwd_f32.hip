// layer_ssm_bwd_f32.hip -- the state space scan's gradient for fp32 inputs (layer_ssm_bwd.h).
#include "layer_ssm_bwd.h"

namespace layer {
namespace ssm_bwd {

void launch_f32(const SsmParams& p, const BwdSpace& ws, hipStream_t st) { launch_kernel<float>(p, ws, st); }

}  // namespace ssm_bwd
}  // namespace layer
