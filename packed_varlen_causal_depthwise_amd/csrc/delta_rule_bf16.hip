// The gated delta rule's kernels for bf16 tensors, with bf16 and FP32 gates.
#include "delta_rule_chunk.h"
#include "delta_rule_step.h"

namespace kdaconv {

template void launch_rule_step<kRuleBF16, kRuleBF16>(const RuleParams&, int, hipStream_t);
template void launch_rule_step<kRuleBF16, kRuleF32>(const RuleParams&, int, hipStream_t);
template void launch_rule_chunks<kRuleBF16, kRuleBF16>(const ChunkParams&, int, hipStream_t);
template void launch_rule_chunks<kRuleBF16, kRuleF32>(const ChunkParams&, int, hipStream_t);

}  // namespace kdaconv
