// Attention over cached keys and values, f16.
#include "dws_attention_kernel.hpp"

namespace dws {

hipError_t launch_attention_f16(const AttentionParams& p, hipStream_t stream) { return launch_type<f16_t>(p, stream); }

}  // namespace dws
