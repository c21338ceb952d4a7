// The chunked gated delta rule for bf16 inputs.
#include "dws_delta_kernel.hpp"

namespace dws {

hipError_t launch_delta_forward_bf16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    return precise ? forward_type<bf16_t, kPrecise<bf16_t>>(p, k, stream) : forward_type<bf16_t, 1>(p, k, stream);
}

hipError_t launch_delta_backward_bf16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    return backward_type<bf16_t>(p, k, precise, stream);
}

}  // namespace dws
