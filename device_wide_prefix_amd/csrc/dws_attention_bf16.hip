// Attention over cached keys and values, bf16.
#include "dws_attention_kernel.hpp"

namespace dws {

hipError_t launch_attention_bf16(const AttentionParams& p, hipStream_t stream) { return launch_type<bf16_t>(p, stream); }

}  // namespace dws
