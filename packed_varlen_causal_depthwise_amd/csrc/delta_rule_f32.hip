// The gated delta rule's kernels for FP32 tensors.
#include "delta_rule_step.h"

namespace kdaconv {

template void launch_rule_step<kRuleF32, kRuleF32>(const RuleParams&, int, hipStream_t);

}  // namespace kdaconv
