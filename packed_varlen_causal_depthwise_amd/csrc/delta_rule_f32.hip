// The gated delta rule's kernels for FP32 tensors.
#include "delta_rule_chunk.h"
#include "delta_rule_step.h"

namespace kdaconv {

template void launch_rule_step<kRuleF32, kRuleF32>(const RuleParams&, int, hipStream_t);
template void launch_rule_chunks<kRuleF32, kRuleF32>(const ChunkParams&, int, hipStream_t);

}  // namespace kdaconv
