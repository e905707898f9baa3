// Absorbed latent attention for bf16 queries and latents of up to 256 channels.
#include "latent_attention_device.h"

namespace kdaconv {

template void launch_attend<kRuleBF16, 256, 1, false>(const AttendParams&, hipStream_t);
template void launch_attend<kRuleBF16, 256, 1, true>(const AttendParams&, hipStream_t);
template void launch_attend<kRuleBF16, 256, 2, false>(const AttendParams&, hipStream_t);
template void launch_attend<kRuleBF16, 256, 2, true>(const AttendParams&, hipStream_t);
template void launch_attend<kRuleBF16, 256, 4, false>(const AttendParams&, hipStream_t);
template void launch_attend<kRuleBF16, 256, 4, true>(const AttendParams&, hipStream_t);

}  // namespace kdaconv
