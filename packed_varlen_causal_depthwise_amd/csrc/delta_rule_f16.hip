// The gated delta rule's kernels for f16 tensors, with f16 and FP32 gates.
#include "delta_rule_chunk.h"
#include "delta_rule_step.h"

namespace kdaconv {

template void launch_rule_step<kRuleF16, kRuleF16>(const RuleParams&, int, hipStream_t);
template void launch_rule_step<kRuleF16, kRuleF32>(const RuleParams&, int, hipStream_t);
template void launch_rule_chunks<kRuleF16, kRuleF16>(const ChunkParams&, int, hipStream_t);
template void launch_rule_chunks<kRuleF16, kRuleF32>(const ChunkParams&, int, hipStream_t);

}  // namespace kdaconv
