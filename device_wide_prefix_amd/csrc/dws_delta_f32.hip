// The chunked gated delta rule for f32 inputs.
#include "dws_delta_kernel.hpp"

namespace dws {

hipError_t launch_delta_forward_f32(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    (void)precise;      // fp32 operands are exact
    return forward_type<float, 1>(p, k, stream);
}

hipError_t launch_delta_backward_f32(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    return backward_type<float>(p, k, precise, stream);
}

}  // namespace dws
