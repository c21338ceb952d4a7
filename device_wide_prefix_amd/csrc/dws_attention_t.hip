#include "dws_attention_kernel_t.hpp"
namespace dws { hipError_t launch_attention_bf16(const AttentionParams& p, hipStream_t stream) { k_attention<bf16_t,128,4,true><<<1,256,0,stream>>>(p); return hipSuccess; } }
