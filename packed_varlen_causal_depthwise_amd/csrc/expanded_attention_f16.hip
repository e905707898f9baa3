// Expanded attention for f16 tensors.
#include "expanded_attention_device.h"

namespace kdaconv {

template void launch_expanded<kRuleF16, 64, 32, 4>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 64, 32, 8>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 64, 64, 4>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 64, 64, 8>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 128, 32, 4>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 128, 32, 8>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 128, 64, 4>(const ExpandParams&, hipStream_t);
template void launch_expanded<kRuleF16, 128, 64, 8>(const ExpandParams&, hipStream_t);

}  // namespace kdaconv
