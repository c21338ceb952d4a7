// The chunked gated delta rule for f16 inputs.
#include "dws_delta_kernel.hpp"

namespace dws {

hipError_t launch_delta_forward_f16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    return precise ? forward_type<f16_t, kPrecise<f16_t>>(p, k, stream) : forward_type<f16_t, 1>(p, k, stream);
}

hipError_t launch_delta_backward_f16(const DeltaParams& p, const DeltaPack& k, bool precise, hipStream_t stream)
{
    return backward_type<f16_t>(p, k, precise, stream);
}

}  // namespace dws
