// Attention over cached keys and values, f32.
#include "dws_attention_kernel.hpp"

namespace dws {

hipError_t launch_attention_f32(const AttentionParams& p, hipStream_t stream) { return launch_type<float>(p, stream); }

}  // namespace dws
